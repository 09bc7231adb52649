// Attention over a paged KV cache held in 4 bits, for many query rows per kv
// head (runs of new tokens): 128 rows a CTA on tcgen05.
//
// A tile of 64 keys is expanded to fp16 operands in shared memory once for all
// 128 rows, K and V alike: a key's row of 128 bytes (64 dims), word j of its codes
// as 16 bytes j, so that Q's dims and the output's stand in the same order (4j,
// HD/2 + 4j, 4j + 1, ...).  For S = Q K^T K is K-major, for O = P V the same layout
// of V is MN-major: nothing is transposed.  What the operands hold depends on what
// the type has to keep:
//  * bf16: the values s c + z rounded to fp16 (off by 2^-11 at most, as Q and P), times a power of
//    two that follows K's largest value in the tile and V's largest so far (each
//    key's own, where they differ much);
//  * fp16, fp32: the codes, which are exact (odd nibbles at 16 times their value);
//    scales and offsets enter per key around the products, as for few rows.
// S goes to TMEM; two threads a row (32 keys each) turn it into P, in TMEM too,
// which is the first operand of O = P V; the O of a tile is added to the row's
// registers, rounded.
//
// Bound by the instructions around the products: for a tile the 128 rows' exp2
// alone take an SM 512 cycles, the products of heads of 64 some 250, and a tile
// takes 1740 of an SM that two CTAs share.  While S of a tile and O of the one
// before are computed the next tile is expanded; one block-wide barrier a tile.
// Measured: 4 runs of 512 tokens on up to 4096, 32 heads of 64 over 8 kv heads,
// bf16: 228 us (220 TFLOP/s); the codes of its cache fit L2.  Splits of the keys
// over a cluster join as for few rows.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4.cuh"
#include "kv4_codes.cuh"
#include "kv4_host.h"
#include "op_util.cuh"
#include "ptx.cuh"

namespace wpk {
namespace {

constexpr int kM = kPrefillRows;  // query rows of a CTA
constexpr int kTile = 64;      // keys of a tile
constexpr int kThreadsP = 256;
constexpr int kSplits = 8;
constexpr int kRing = 4;       // tiles in staging
constexpr uint32_t kLeastK = 15;  // K's exponents: both 2^(141 - field) and its inverse are normal numbers

template <typename T, int HD>
struct PGeo {
  using P = Keep<T>;
  static constexpr int kWords = HD / 8;                       // of a row's codes
  static constexpr int kQBytes = kM * HD * 2;                 // one of Q's parts
  static constexpr int kKBytes = kTile * HD * 2, kVBytes = HD * kTile * 2;
  // operands, 1024-byte aligned: K twice and V three times, since a tile is
  // expanded while the one before is multiplied
  static constexpr int kQ = 0, kQl = kQ + kQBytes, kK = kQl + (P::kQLow ? kQBytes : 0), kV = kK + 2 * kKBytes;
  static constexpr int kOps = kV + 3 * kVBytes;
  static constexpr int kCodes = kTile * HD / 2;               // staging: K's codes, V's, their scales
  static constexpr int kStage = 2 * kCodes + kTile * 8;
  static constexpr int kScales = kOps + kRing * kStage;       // what a tile's scales become, 1 KB each
  static constexpr int kRed = kScales + kRing * kTile * 16;   // [2][kM] floats: both threads of a row
  static constexpr int kFactors = kRed + 2 * kM * 4;          // values: what K's keys were divided by, V's exponents
  static constexpr int kBytes = kFactors + (P::kBf16 ? kRing * 2 * kTile * 4 : 0);
  // after the keys: O [kM][HD], offsets, sums
  static constexpr int kJoin = kM * (HD + 2) * 4;
  static constexpr int kSmem = (kBytes > kJoin ? kBytes : kJoin) + 1024;  // and what aligns it
  static constexpr int kS = 0, kP = 64, kO = 128, kCols = 256;  // TMEM: S, P (32 columns, 32 of what it lost), O
  static constexpr int kPerSm = HD == 64 ? 2 : 1;
  static constexpr bool kValues = P::kBf16;                   // operands hold values, not codes
};

struct Tile {  // what its scales say
  uint32_t have;           // runs of 16 keys that have a place
  uint32_t k_exp, v_exp;   // biased exponents: K's largest value here; V's largest scale (codes, see v_key_exp) or value so far
  bool k_spread;           // values: K's exponents differ by more than kSpread, each key has its own
  bool spread;             // V's exponents differ by more than kSpread
  int bad;                 // values: the first key whose V is NaN
};

// Four values as they are in memory (zeros where there are none).
template <typename T>
struct Raw4 {
  uint2 r;
  __device__ __forceinline__ void load(bool on, const T* p) {
    r = on ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
  }
  __device__ __forceinline__ void to(float* f) const { load4(reinterpret_cast<const T*>(&r), f); }
};
template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void load(bool on, const float* p) {
    r = on ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void to(float* f) const { f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w; }
};

struct PrefillArgs {
  int64_t q_tok, q_head, o_tok, o_head;
  const float* rope;
  int group, max_new, row_blocks, split;
  float scale_log2;
};

// Waits for a phase of a barrier; false where it has not ended after a second, nor
// when looked at once more (a context that was switched out comes back late).
// Nothing but a lost copy or product takes so long: the block then starts nothing
// more and its rows answer NaN.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (globaltimer() - t0 < 1000000000ull)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_try_wait(bar, parity);
}

// 32 columns of a thread's TMEM lane at two addresses each, waited for together.
__device__ __forceinline__ void tmem_ld32_two(uint32_t at_a, float* a, uint32_t at_b, float* b) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(a[0]), "=f"(a[1]), "=f"(a[2]), "=f"(a[3]), "=f"(a[4]), "=f"(a[5]), "=f"(a[6]), "=f"(a[7]), "=f"(a[8]), "=f"(a[9]), "=f"(a[10]), "=f"(a[11]), "=f"(a[12]), "=f"(a[13]), "=f"(a[14]), "=f"(a[15]), "=f"(a[16]), "=f"(a[17]), "=f"(a[18]), "=f"(a[19]), "=f"(a[20]), "=f"(a[21]), "=f"(a[22]), "=f"(a[23]), "=f"(a[24]), "=f"(a[25]), "=f"(a[26]), "=f"(a[27]), "=f"(a[28]), "=f"(a[29]), "=f"(a[30]), "=f"(a[31]),
        "=f"(b[0]), "=f"(b[1]), "=f"(b[2]), "=f"(b[3]), "=f"(b[4]), "=f"(b[5]), "=f"(b[6]), "=f"(b[7]), "=f"(b[8]), "=f"(b[9]), "=f"(b[10]), "=f"(b[11]), "=f"(b[12]), "=f"(b[13]), "=f"(b[14]), "=f"(b[15]), "=f"(b[16]), "=f"(b[17]), "=f"(b[18]), "=f"(b[19]), "=f"(b[20]), "=f"(b[21]), "=f"(b[22]), "=f"(b[23]), "=f"(b[24]), "=f"(b[25]), "=f"(b[26]), "=f"(b[27]), "=f"(b[28]), "=f"(b[29]), "=f"(b[30]), "=f"(b[31])
      : "r"(at_a), "r"(at_b)
      : "memory");
}

__device__ __forceinline__ void bar_pair(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// What a tile takes besides where its keys' exponents are spread, for a thread's 32
// keys.  Out of line, on a copy of x: within the loop over tiles their code costs the
// tiles that do without it 4 us of 234.
struct Logits {
  float x[32];
};
// K's keys have been divided by f each.
__device__ __noinline__ void multiply_keys(Logits* at, const float* f) {
#pragma unroll 4
  for (int i = 0; i < 32; ++i) at->x[i] *= f[i];
}
// The largest logit with its key's V exponent (rounded up); scales of V, two keys each.
__device__ __noinline__ float largest_product(const Logits* at, float k_tile, const float4* scales) {
  float top = -INFINITY;
#pragma unroll 4
  for (int i = 0; i < 16; ++i)
    top = max3(top, __fadd_ru(at->x[2 * i] * k_tile, (float)((int)v_key_exp(scales[i].x, scales[i].z) - 127)),
               __fadd_ru(at->x[2 * i + 1] * k_tile, (float)((int)v_key_exp(scales[i].y, scales[i].w) - 127)));
  return top;
}
// Values: the largest of the weights' logarithms with their keys' exponents.
__device__ __noinline__ float largest_weight(const Logits* at, float k_tile, float off, const float* v_own) {
  float most = -1024.f;
#pragma unroll 4
  for (int i = 0; i < 32; ++i) most = fmaxf(most, __fadd_ru(fmaf(at->x[i], k_tile, -off), v_own[i]));
  return most;
}
// The weights' sum; x becomes the logarithms of P, which are times 2^(their keys' exponents - v_exp).
__device__ __noinline__ float sum_weights(Logits* at, float k_tile, float off, const float* v_own, int v_exp) {
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < 32; ++i) {
    const float d = fmaf(at->x[i], k_tile, -off);
    sum += ex2(d);
    at->x[i] = d + (v_own[i] - (float)v_exp);
  }
  return sum;
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreadsP, PGeo<T, HD>::kPerSm)
    kv4_prefill_kernel(const Kv4Dev c, const T* __restrict__ q, T* __restrict__ out, const PrefillArgs a) {
  using G = PGeo<T, HD>;
  using P = Keep<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 + kRing];  // S ready, O ready, codes of a tile here
  __shared__ Tile tiles[2 * kRing];  // a tile is copied before the one four earlier is done with
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_lost[2];  // a wait before the barrier of an even (odd) tile has not ended
  uint8_t* smem = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int hw = warp >> 2;                    // half of the keys (S columns), and of the dims (O columns)
  const int r = 32 * (warp & 3) + lane;        // the row: TMEM lane
  const int rank = blockIdx.x % a.split;
  int item = blockIdx.x / a.split;
  const int rb = a.row_blocks - 1 - item % a.row_blocks;  // the rows that see most come first
  item /= a.row_blocks;
  const int head = item % c.n_kv, b = item / c.n_kv;
  if (b >= kv4_sequences(c)) return;  // as for every CTA of the cluster
  const int pos0 = c.pos[b];
  int q0, n_new;
  kv4_new(c, b, &q0, &n_new);
  const int64_t rows = (int64_t)min(n_new, a.max_new) * a.group, r0 = (int64_t)rb * kM;
  if (r0 >= rows) return;

  const int64_t cap = (int64_t)c.max_blocks * c.page_tokens;
  const int64_t my_row = r0 + r;
  const int my_new = my_row < rows ? (int)((uint32_t)my_row / (uint32_t)a.group) : 0;
  const int my_head = my_row < rows ? head * a.group + (int)((uint32_t)my_row % (uint32_t)a.group) : 0;
  const int64_t my_pos = (int64_t)pos0 + my_new;
  const bool placed = my_row < rows && pos0 >= 0 && my_pos < c.rope_positions;
  const int last = placed ? (int)(my_pos < cap ? my_pos : cap - 1) : -1;  // the row's last key
  const int64_t lo_pos = pos0 + r0 / a.group, hi_pos = pos0 + (min(r0 + kM, rows) - 1) / a.group;
  const int n_keys = pos0 < 0 ? 0 : (int)min(hi_pos + 1, cap);
  const int all_see = (int)min(lo_pos + 1, cap);  // keys below it are seen by every row that has a position
  const int n_tiles = n_keys ? (n_keys - 1) / kTile + 1 : 0;
  const int n_mine = n_tiles > rank ? (n_tiles - rank + a.split - 1) / a.split : 0;  // every split-th tile

  if (tid == 0) {
    s_lost[0] = s_lost[1] = 0;
    for (int i = 0; i < 2 + kRing; ++i) mbar_init(&bars[i], i < 2 ? 1 : 4);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, G::kCols);
    tmem_relinquish();
  }

  // Each warp has a task of its own besides: warps 0 and 1 issue S and O, 2 and 3
  // prepare K's and V's scales, 4 to 7 copy K's codes, V's, K's scales and V's.  A
  // copy takes the runs of 16 keys that lie in one page: lane 0 (to 3, with pages
  // that end in the tile) starts it.
  const int32_t* table = c.table + (int64_t)b * c.max_blocks;
  const int codes = c.page_tokens * (HD / 2), kind = warp & 3;
  const int unit = kind < 2 ? HD / 2 : 4;  // bytes of a key
  int block = -1;                          // of the next copy's run, looked up a tile ahead
  auto look_up = [&](int j) {
    const int64_t key = (int64_t)(rank + (int64_t)j * a.split) * kTile + 16 * (lane & 3);
    block = j < n_mine && key < n_keys ? table[kv4_slot(c, (int)key)] : -1;
  };
  auto copy = [&](int j) {  // the CTA's j-th tile
    if (j >= n_mine) return;
    const uint32_t have = __ballot_sync(0xFFFFFFFFu, block >= 0 && block < c.n_blocks) & 15u;
    uint64_t* bar = &bars[2 + (j & (kRing - 1))];
    if (lane == 0) {
      if (kind == 0) tiles[j & (2 * kRing - 1)].have = have;
      mbar_arrive_expect_tx(bar, __popc(have) * 16 * unit);
    }
    __syncwarp();
    if (lane < 4 && (have >> lane & 1u)) {
      const int key = (rank + j * a.split) * kTile + 16 * lane, row = key - kv4_slot(c, key) * c.page_tokens;
      if (lane == 0 || row == 0) {  // the run's page starts here
        const int runs = min(min(4 - lane, (c.page_tokens - row) >> 4), (n_keys - key + 15) >> 4);
        bulk_g2s(smem + G::kOps + (j & (kRing - 1)) * G::kStage + (kind >> 1) * (2 * G::kCodes) +
                     ((kind & 1) * kTile + 16 * lane) * unit,
                 kv4_page(c, block, head) + (kind >> 1) * (2 * codes) + ((kind & 1) * c.page_tokens + row) * unit,
                 runs * 16 * unit, bar);
      }
    }
  };
  // `turn`: the tile whose barrier comes next (-1: the one before the first tile).
  // Flags are read behind their barrier, while waits behind it set the other one.
  auto await = [&](uint64_t* bar, int phase, int turn) {
    if (!wait_bounded(bar, phase & 1)) s_lost[turn & 1] = 1;
  };
  auto arrived = [&](int j, int turn) { await(&bars[2 + (j & (kRing - 1))], j / kRing, turn); };

  // What the operands and the softmax need of a tile's scales, two keys a lane, of
  // K (e = 0) or V; zeros for keys without a place.
  uint32_t run_exp = kLeastExp, run_least = 255;  // (the least: of this lane's keys with a range)
  auto prepare = [&](int j, int e, int turn) {
    if (j >= n_mine) return;
    arrived(j, turn);
    const int slot = j & (kRing - 1), key0 = (rank + j * a.split) * kTile;
    Tile& tile = tiles[j & (2 * kRing - 1)];
    uint2 w = *reinterpret_cast<const uint2*>(smem + G::kOps + slot * G::kStage + 2 * G::kCodes + e * (4 * kTile) +
                                              8 * lane);
    const bool there = (tile.have >> (lane >> 3)) & 1u;
    if (!there || key0 + 2 * lane >= n_keys) w.x = 0;
    if (!there || key0 + 2 * lane + 1 >= n_keys) w.y = 0;
    const float sa = __uint_as_float(w.x << 16), sb = __uint_as_float(w.y << 16);
    float za = __uint_as_float(w.x & 0xFFFF0000u), zb = __uint_as_float(w.y & 0xFFFF0000u);
    if constexpr (G::kValues) {
      // the largest size of the values, a NaN left out
      const float ra = fmaxf(fmaxf(0.f, fabsf(za)), fabsf(fmaf(15.f, sa, za)));
      const float rb = fmaxf(fmaxf(0.f, fabsf(zb)), fabsf(fmaf(15.f, sb, zb)));
      uint32_t ea = min(__float_as_uint(ra) >> 23, 254u), eb = min(__float_as_uint(rb) >> 23, 254u);
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(ea, eb));
      if (e == 0) {
        // K's product is taken tile by tile, so it has a power of two for each; keys
        // that differ by more than kSpread have one each, which S's columns take back
        run_exp = max(top, kLeastK);
        const bool spread =
            __any_sync(0xFFFFFFFFu, (ra > 0.f && ea + kSpread < run_exp) || (rb > 0.f && eb + kSpread < run_exp));
        ea = spread ? max(ea, kLeastK) : run_exp;
        eb = spread ? max(eb, kLeastK) : run_exp;
        if (spread)
          reinterpret_cast<float2*>(smem + G::kFactors + slot * (2 * kTile * 4))[lane] =
              make_float2(__uint_as_float((ea - 14u) << 23), __uint_as_float((eb - 14u) << 23));
        if (lane == 0) tile.k_spread = spread;
      } else {
        // V's follows the largest value so far; where the exponents so far differ by
        // more than kSpread, each key has its own, which the weights take back
        run_exp = max(run_exp, top);
        run_least = min(run_least, min(ra > 0.f ? ea : 255u, rb > 0.f ? eb : 255u));
        const bool spread = __any_sync(0xFFFFFFFFu, run_least + kSpread < run_exp);
        if (lane == 0) tile.spread = spread;
        ea = spread ? max(ea, kLeastExp) : run_exp;
        eb = spread ? max(eb, kLeastExp) : run_exp;
        if (spread)
          reinterpret_cast<float2*>(smem + G::kFactors + slot * (2 * kTile * 4) + kTile * 4)[lane] =
              make_float2((float)ea, (float)eb);
      }
      // the largest value to 2^14..2^15
      const float fa = __uint_as_float((268u - ea) << 23), fb = __uint_as_float((268u - eb) << 23);
      if (e) {  // a NaN must not reach rows that do not see it
        const int bad = (int)__reduce_min_sync(0xFFFFFFFFu, za != za ? 2 * lane : zb != zb ? 2 * lane + 1 : INT_MAX);
        if (lane == 0) tile.bad = bad;
        if (za != za) za = 0.f;
        if (zb != zb) zb = 0.f;
      }
      auto twice = [](float x) {
        const __half2 h = __float2half2_rn(x);
        return *reinterpret_cast<const uint32_t*>(&h);
      };
      reinterpret_cast<uint4*>(smem + G::kScales + slot * (kTile * 16))[32 * e + lane] =
          make_uint4(twice(sa * fa), twice(za * fa), twice(sb * fb), twice(zb * fb));
    } else {
      const bool centre = e ? P::kCentreV : P::kCentreK;
      const float ya = centre ? fmaf(8.f, sa, za) : za, yb = centre ? fmaf(8.f, sb, zb) : zb;
      reinterpret_cast<float4*>(smem + G::kScales + slot * (kTile * 16))[32 * e + lane] = make_float4(sa, sb, ya, yb);
      if (e) {
        const uint32_t ea = v_key_exp(sa, ya), eb = v_key_exp(sb, yb);
        run_exp = max(run_exp, __reduce_max_sync(0xFFFFFFFFu, max(ea, eb)));
        run_least = min(run_least, min(sa != 0.f ? ea : 255u, sb != 0.f ? eb : 255u));
        const bool spread = __any_sync(0xFFFFFFFFu, run_least + kSpread < run_exp);
        if (lane == 0) tile.spread = spread;
      }
      if (lane == 0) tile.bad = INT_MAX;
    }
    if (lane == 0) (e ? tile.v_exp : tile.k_exp) = run_exp;
  };

  // The first tiles' places and Q's values are under way together.
  int first[kRing] = {};
  if (warp >= 4) {
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
      look_up(j);
      first[j] = block;
    }
  }
  constexpr int kU = G::kWords / 2;  // units of Q's row that the thread takes
  Raw4<T> raw[kU][2];
  const T* q_row = q + (int64_t)(q0 + my_new) * a.q_tok + my_head * a.q_head + 4 * hw * kU;
#pragma unroll
  for (int i = 0; i < kU; ++i) {
    raw[i][0].load(placed, q_row + 4 * i);
    raw[i][1].load(placed, q_row + HD / 2 + 4 * i);
  }
  __syncthreads();  // the barriers are there for everyone
  if (warp >= 4) {
#pragma unroll
    for (int j = 0; j < kRing; ++j) {
      block = first[j];
      copy(j);
    }
    look_up(kRing);
  }

  // Q: the thread's half of the row's units, times scale log2(e) and the power of
  // two that brings the row's largest value to 2^13..2^14
  float* red = reinterpret_cast<float*>(smem + G::kRed);
  float k_mul, z_mul;  // a logit is k_mul (s S + z z_mul)
  {
    float x[kU][8];  // dims 4u .. 4u + 3, then HD / 2 + 4u ..
    float top = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = hw * kU + i;
      raw[i][0].to(x[i]);
      raw[i][1].to(x[i] + 4);
      if (placed) {
        if (a.rope) {
          const float* cs = a.rope + (my_pos * (HD / 2) + 4 * u) * 2;
          float t[8];
          load4(cs, t);
          load4(cs + 4, t + 4);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = x[i][e], hi = x[i][4 + e];
            x[i][e] = lo * t[2 * e] - hi * t[2 * e + 1];
            x[i][4 + e] = hi * t[2 * e] + lo * t[2 * e + 1];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[i][e] *= a.scale_log2;
          top = fmaxf(top, fabsf(x[i][e]));
          sum += x[i][e];
        }
      }
    }
    red[hw * kM + r] = sum;
    __syncthreads();
    sum = red[r] + red[kM + r];
    __syncthreads();
    red[hw * kM + r] = top;
    __syncthreads();
    const uint32_t e8 = max(27u, __float_as_uint(fmaxf(red[r], red[kM + r])) >> 23);
    const float mul = __uint_as_float(e8 < 255u ? (267u - e8) << 23 : 0x3F800000u);
    constexpr float kCode = G::kValues || P::kCentreK ? 1.f : 16777216.f;
    k_mul = kCode / mul;
    z_mul = sum * mul * (1.f / kCode);
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = hw * kU + i;
      uint32_t hi[4], lo[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {  // nibbles n and n + 4
        const float m = !G::kValues && (n & 1) ? mul * 0.0625f : mul;
        const float y0 = x[i][n] * m, y1 = x[i][4 + n] * m;
        hi[n] = pack_f16(y0, y1);
        const float2 back = unpack_f16(hi[n]);
        lo[n] = pack_f16(y0 - back.x, y1 - back.y);
      }
      const uint32_t off = (u >> 3) * (kM * 128) + r * 128 + (((u & 7) ^ (r & 7)) << 4);
      *reinterpret_cast<uint4*>(smem + G::kQ + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      if (P::kQLow) *reinterpret_cast<uint4*>(smem + G::kQl + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp >> 1 == 1)
    for (int j = 0; j < 2; ++j) prepare(j, warp & 1, -1);
  __syncthreads();
  const uint32_t tmem = s_tmem, mine = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t smem0 = smem_u32(smem);

  float m = -INFINITY, off = 0.f;  // as for few rows; the same in both threads of a row
  F2 l2 = pair(0.f, 0.f), py2 = l2;
  float o[HD / 2];  // of the row: columns hw HD / 2 .., dims hw HD / 4 .. and those HD / 2 further, in turn
#pragma unroll
  for (int i = 0; i < HD / 2; ++i) o[i] = 0.f;
  int v_exp = (int)kLeastExp;  // values: O stands at 2^(141 - v_exp)
  auto add_part = [&](int i, const float* v) {  // 32 columns of a tile's O
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 t = split(add2(pair(o[i + e], o[i + e + 1]), pair(v[e], v[e + 1])));
      o[i + e] = t.x;
      o[i + e + 1] = t.y;
    }
  };
  // adds a tile's O but for its last 32 columns, whose address it gives
  auto add_o = [&](int j) -> uint32_t {
    await(&bars[1], j, j + 1);
    tc_fence_after();
    if (HD == 128) {
      float v[32];
      tmem_ld16x2(mine + G::kO + hw * (HD / 2), v);
      add_part(0, v);
    }
    return mine + G::kO + hw * (HD / 2) + HD / 2 - 32;
  };
  // K's and V's words of a key to 16-byte units of its rows, two or four a thread
  auto expand = [&](int j) {
    arrived(j, j - 1);
    const int slot = j & (kRing - 1);
    const uint8_t* stage = smem + G::kOps + slot * G::kStage;
    const int key = tid >> 2, part = tid & 3;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint8_t* rows_of = smem + (kv ? G::kV + j % 3 * G::kVBytes : G::kK + (j & 1) * G::kKBytes) + key * 128;
      __half2 s1{}, s16{}, z1{};
      if constexpr (G::kValues) {
        const uint2 w = reinterpret_cast<const uint2*>(smem + G::kScales + slot * (kTile * 16))[kTile * kv + key];
        s1 = *reinterpret_cast<const __half2*>(&w.x);
        z1 = *reinterpret_cast<const __half2*>(&w.y);
        s16 = __hmul2(s1, __float2half2_rn(0.0625f));
      }
      auto even = [&](uint32_t x) -> uint32_t {
        if constexpr (G::kValues) {
          const uint32_t y = centred_even<0>(x);
          const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&y), s1, z1);
          return *reinterpret_cast<const uint32_t*>(&v);
        } else {
          return kv ? codes_even<P::kCentreV>(x) : codes_even<P::kCentreK>(x);
        }
      };
      auto odd = [&](uint32_t x) -> uint32_t {
        if constexpr (G::kValues) {
          const uint32_t y = centred_odd<0>(x);
          const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&y), s16, z1);
          return *reinterpret_cast<const uint32_t*>(&v);
        } else {
          return kv ? codes_odd<P::kCentreV>(x) : codes_odd<P::kCentreK>(x);
        }
      };
#pragma unroll
      for (int i = 0; i < G::kWords / 8; ++i) {
        const uint2 w =
            *reinterpret_cast<const uint2*>(stage + kv * G::kCodes + key * (HD / 2) + i * 32 + part * 8);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = e ? w.y : w.x, y = x >> 8;
          *reinterpret_cast<uint4*>(rows_of + i * (kTile * 128) + (((2 * part + e) ^ (key & 7)) << 4)) =
              make_uint4(even(x), odd(x), even(y), odd(y));
        }
      }
    }
    fence_proxy_async_smem();  // the products read these generic-proxy writes
  };
  auto issue_s = [&](int j) {
    constexpr uint32_t idesc = idesc_f16(kM, kTile, false);
#pragma unroll
    for (int kk = 0; kk < HD / 16; ++kk) {
      const uint64_t kd =
          sdesc_k_sw128(smem0 + G::kK + (j & 1) * G::kKBytes + (kk >> 2) * (kTile * 128) + (kk & 3) * 32);
      const uint32_t qa = (kk >> 2) * (kM * 128) + (kk & 3) * 32;
      umma_f16(tmem + G::kS, sdesc_k_sw128(smem0 + G::kQ + qa), kd, idesc, kk > 0);
      if (P::kQLow) umma_f16(tmem + G::kS, sdesc_k_sw128(smem0 + G::kQl + qa), kd, idesc, 1u);
    }
    umma_commit(&bars[0]);
  };
  auto issue_o = [&](int j) {
    constexpr uint32_t idesc = idesc_f16(kM, HD, false) | 1u << 16;  // V is MN-major
#pragma unroll
    for (int kk = 0; kk < kTile / 16; ++kk) {
      // 16 keys: two groups of 8 rows; the next 64 dims are a leading offset away
      const uint64_t vd = sdesc_k_sw128(smem0 + G::kV + j % 3 * G::kVBytes + kk * 2048) +
                          ((uint64_t)(kTile * 128 / 16 - 1) << 16);
      umma_f16_ta(tmem + G::kO, tmem + G::kP + 8 * kk, vd, idesc, kk > 0);
      if (P::kPLow) umma_f16_ta(tmem + G::kO, tmem + G::kP + 32 + 8 * kk, vd, idesc, 1u);
    }
    umma_commit(&bars[1]);
  };

  if (n_mine) {
    expand(0);
    __syncthreads();
    if (tid == 0) issue_s(0);
    if (warp >= 4) {
      if (!s_lost[1]) copy(kRing);
      look_up(kRing + 1);
    }
    if (warp >> 1 == 1) prepare(2, warp & 1, 0);
  }
  int j = 0;
#pragma unroll 1
  for (; j < n_mine; ++j) {
    const int lost = s_lost[(j + 1) & 1];
    // While S of this tile and O of the one before are computed, the next tile is
    // expanded.
    const int key0 = (rank + j * a.split) * kTile;
    if (j + 1 < n_mine) expand(j + 1);
    if (lost) break;
    const uint32_t rest = j ? add_o(j - 1) : 0u;
    const Tile tile = tiles[j & (2 * kRing - 1)];
    const float4* scales = reinterpret_cast<const float4*>(smem + G::kScales + (j & (kRing - 1)) * (kTile * 16));
    await(&bars[0], j, j);
    tc_fence_after();

    // the row's logits of 32 keys, k_tile times them in units of log2
    float x[32];
    if (j) {
      float v[32];
      tmem_ld32_two(mine + G::kS + 32 * hw, x, rest, v);
      add_part(HD / 2 - 32, v);
    } else {
      tmem_ld16x2(mine + G::kS + 32 * hw, x);
    }
    float k_tile = k_mul;
    if constexpr (G::kValues) {
      if (tile.k_spread) {
        Logits copy;
        for (int i = 0; i < 32; ++i) copy.x[i] = x[i];
        multiply_keys(&copy, reinterpret_cast<const float*>(smem + G::kFactors + (j & (kRing - 1)) * (2 * kTile * 4)) +
                                 32 * hw);
        for (int i = 0; i < 32; ++i) x[i] = copy.x[i];
      } else {
        // > 0, so that a logit of -infinity stays one
        k_tile = fmaxf(k_mul * __uint_as_float((tile.k_exp - 14u) << 23), __uint_as_float(1u));
      }
    }
    float top = -INFINITY;
    if constexpr (!G::kValues) {
      const F2 z2 = pair(z_mul, z_mul);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 ks = scales[16 * hw + i];
        const float2 t = split(fma2(pair(ks.x, ks.y), pair(x[2 * i], x[2 * i + 1]), mul2(pair(ks.z, ks.w), z2)));
        x[2 * i] = t.x;
        x[2 * i + 1] = t.y;
      }
    }
    const bool part = tile.have != 15u || key0 > all_see - kTile;
    if (part) {  // scores without a place, or behind the row's last key
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((tile.have >> (2 * hw + (i >> 4))) & 1u) || key0 + 32 * hw + i > last) x[i] = -INFINITY;
    }
    // (sums rounded up, so that P does not pass its range however large the logits are)
    if (G::kValues || !tile.spread) {
#pragma unroll
      for (int i = 0; i < 32; i += 2) top = max3(top, x[i], x[i + 1]);
      top *= k_tile;
      if (!G::kValues) top = __fadd_ru(top, (float)((int)tile.v_exp - 127));
    } else {
      Logits copy;
      for (int i = 0; i < 32; ++i) copy.x[i] = x[i];
      top = largest_product(&copy, k_tile, scales + 32 + 16 * hw);
    }
    red[hw * kM + r] = top;
    bar_pair(1 + (warp & 3));  // the other half of the rows is the other warp's of the four
    const float m_new = fmaxf(m, fmaxf(top, red[(hw ^ 1) * kM + r]));
    const float* v_own = reinterpret_cast<const float*>(smem + G::kFactors + (j & (kRing - 1)) * (2 * kTile * 4)) +
                         kTile + 32 * hw;  // values: V's exponents, where they are spread
    const bool spread = G::kValues && tile.spread;
    if (m_new != m || spread || (G::kValues && (int)tile.v_exp != v_exp)) {
      // P reaches 2^15, as a weight or times its key's V scale
      const float off_new = __fsub_ru(m_new == -INFINITY ? 0.f : m_new, G::kValues ? 15.f : 14.f);
      const float fade = m == -INFINITY ? 0.f : ex2(off - off_new);
      float o_fade = fade;
      if constexpr (G::kValues) {
        int v_new = (int)tile.v_exp;
        if (spread) {
          // The row's own exponent: P is the weight times 2^(its key's exponent - v_new),
          // at most 2^15.  Down with the fading of what O holds, so that O only shrinks.
          Logits copy;
          for (int i = 0; i < 32; ++i) copy.x[i] = x[i];
          float most = largest_weight(&copy, k_tile, off_new, v_own);
          bar_pair(1 + (warp & 3));  // the other has read this row's largest logit
          red[hw * kM + r] = most;
          bar_pair(1 + (warp & 3));
          most = fmaxf(most, red[(hw ^ 1) * kM + r]);
          v_new = max((int)ceilf(most) - 15, (int)kLeastExp);
          if (m != -INFINITY) v_new = max(v_new, v_exp - (int)fminf(off_new - off, 512.f));
        }
        // operands that are values shrink as the exponent grows
        o_fade = m == -INFINITY ? 0.f : ex2((off - off_new) + (float)(v_exp - v_new));
        v_exp = v_new;
      }
      const F2 f2 = pair(fade, fade), o2 = pair(o_fade, o_fade);
      l2 = mul2(l2, f2);  // a NaN stays
      if (!G::kValues) py2 = mul2(py2, f2);
#pragma unroll
      for (int i = 0; i < HD / 2; i += 2) {
        const float2 t = split(mul2(pair(o[i], o[i + 1]), o2));
        o[i] = t.x;
        o[i + 1] = t.y;
      }
      m = m_new;
      off = off_new;
    }
    F2 down = pair(-off, -off), k2 = pair(k_tile, k_tile), l_own = l2;
    if (spread) {
      Logits copy;
      for (int i = 0; i < 32; ++i) copy.x[i] = x[i];
      l_own = add2(l2, pair(sum_weights(&copy, k_tile, off, v_own, v_exp), 0.f));
      for (int i = 0; i < 32; ++i) x[i] = copy.x[i];
      k2 = pair(1.f, 1.f);
      down = pair(0.f, 0.f);
    }
#pragma unroll
    for (int g = 0; g < 2; ++g) {  // 16 keys: 8 columns of P
      uint32_t hi[8], lo[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int n = 8 * g + i;
        const float2 d = split(fma2(pair(x[2 * n], x[2 * n + 1]), k2, down));
        const float2 pf = make_float2(ex2(d.x), ex2(d.y));
        const F2 p = pair(pf.x, pf.y);
        l2 = add2(l2, p);
        if constexpr (G::kValues) {
          hi[i] = pack_f16(pf.x, pf.y);
          continue;
        }
        const float4 vs = scales[32 + 16 * hw + n];
        // a key that the row does not see must not count, even with an offset of NaN
        const F2 y = part ? pair(x[2 * n] == -INFINITY ? 0.f : vs.z, x[2 * n + 1] == -INFINITY ? 0.f : vs.w)
                          : pair(vs.z, vs.w);
        py2 = fma2(p, y, py2);
        const float2 w = split(mul2(p, pair(vs.x, vs.y)));
        hi[i] = pack_f16(w.x, w.y);
        if (P::kPLow) {
          const float2 back = unpack_f16(hi[i]);
          lo[i] = pack_f16(w.x - back.x, w.y - back.y);
        }
      }
      tmem_st8(mine + G::kP + 16 * hw + 8 * g, hi);
      if (P::kPLow) tmem_st8(mine + G::kP + 32 + 16 * hw + 8 * g, lo);
    }
    if (spread) l2 = l_own;
    if (tile.bad <= last - key0) l2 = pair(NAN, NAN);  // `last` is -1 for rows without a key
    tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp >= 4) {
      if (!s_lost[j & 1]) copy(j + 1 + kRing);  // where the tile was that is expanded now
      look_up(j + 2 + kRing);
    } else if (warp >= 2)
      prepare(j + 3, warp & 1, j + 1);
    else if (lane == 0) {
      if (warp == 1)
        issue_o(j);
      else if (j + 1 < n_mine)
        issue_s(j + 1);
    }
    __syncwarp();
  }
  if (j < n_mine) {  // given up: what was started (copies of the next tiles, S, the O before) ends before its memory is left
    for (int i = j; i < min(n_mine, j + kRing); ++i) arrived(i, j);
    await(&bars[0], j, j);
    if (j) await(&bars[1], j - 1, j);
  } else if (n_mine) {
    float v[32];
    tmem_ld16x2(add_o(n_mine - 1), v);
    add_part(HD / 2 - 32, v);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, G::kCols);
  // a thread of each half holds its dims of the row; the sums come together
  {
    const float2 lp = split(l2), pp = split(py2);
    red[hw * kM + r] = lp.x + lp.y;
    __syncthreads();
    const float l = red[r] + red[kM + r];
    __syncthreads();
    red[hw * kM + r] = pp.x + pp.y;
    __syncthreads();
    const float py = red[r] + red[kM + r];
    __syncthreads();
    // codes: odd nibbles stand 16 times as high, raw ones at 2^-24; values at
    // 2^14 / 2^v_exp, their weights at 2^15
    constexpr float even = P::kCentreV ? 1.f : 16777216.f;
    const float back = __uint_as_float((uint32_t)(v_exp - 29) << 23);
#pragma unroll
    for (int i = 0; i < HD / 2; ++i)
      o[i] = G::kValues ? o[i] * back : fmaf(o[i], i >> 1 & 1 ? even * 0.0625f : even, py);
    const float sum = G::kValues ? l * 0x1p-15f : l;
    const float none = s_lost[0] || s_lost[1] ? NAN : 0.f;
    float* join = reinterpret_cast<float*>(smem);  // [kM][HD + 2]
    if (a.split == 1) {
      if (my_row < rows) {
        // a row that saw no key, or has no rotation, answers zeros
        const float inv = sum == 0.f || !placed ? 0.f : 1.0f / sum;
        T* dst = out + (int64_t)(q0 + my_new) * a.o_tok + my_head * a.o_head;
#pragma unroll
        for (int i = 0; i < HD / 2; i += 8) {
          float y[2][4];
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e & 1][e >> 1] = (inv == 0.f ? 0.f : o[i + e] * inv) + none;
          store4(dst + hw * (HD / 4) + i / 2, y[0]);
          store4(dst + HD / 2 + hw * (HD / 4) + i / 2, y[1]);
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < HD / 2; ++i)
      join[r * (HD + 2) + (i & 1) * (HD / 2) + hw * (HD / 4) + (i >> 1)] = o[i] + none;
    if (hw == 0) {
      join[r * (HD + 2) + HD] = m == -INFINITY ? -INFINITY : off;
      join[r * (HD + 2) + HD + 1] = sum;
    }
    cluster_barrier();
    // each CTA joins every split-th row, 4 dims a thread
    constexpr int kPer = HD / 4;
#pragma unroll 1
    for (int e = tid; e < kM / a.split * kPer; e += kThreadsP) {
      const int jr = e / kPer * a.split + rank, d = e % kPer * 4;
      float best = -INFINITY, all = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
      for (int s = 0; s < a.split; ++s)
        best = fmaxf(best, __uint_as_float(cluster_load32(cluster_address(join + jr * (HD + 2) + HD, s))));
      for (int s = 0; s < a.split; ++s) {
        const uint32_t at = cluster_address(join + jr * (HD + 2), s);
        const float ms = __uint_as_float(cluster_load32(at + HD * 4));
        const float w = ms == best ? 1.f : ex2(ms - best);
        all = fmaf(w, __uint_as_float(cluster_load32(at + HD * 4 + 4)), all);
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = fmaf(w, __uint_as_float(cluster_load32(at + (d + i) * 4)), y[i]);
      }
      if (r0 + jr < rows) {
        const uint32_t fresh = (uint32_t)(r0 + jr) / (uint32_t)a.group, h = (uint32_t)(r0 + jr) % (uint32_t)a.group;
        const bool zero = all == 0.f || (int64_t)pos0 + fresh >= c.rope_positions;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = zero ? 0.f : y[i] / all;
        store4(out + (int64_t)(q0 + (int)fresh) * a.o_tok + (head * a.group + (int)h) * a.o_head + d, y);
      }
    }
    cluster_barrier();  // no CTA leaves while another reads its part
  }
}

template <typename T, int HD>
cudaError_t launch(const Kv4Dev& d, const Kv4Tensor& q, const Kv4Tensor& o, PrefillArgs a, int64_t items,
                   cudaStream_t s) {
  using G = PGeo<T, HD>;
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(kv4_prefill_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::kSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  }
  // CTAs that share a block's keys: while the GPU (148 SMs) is not full, and once
  // more between one wave and two, where sequences of other lengths leave the last
  // wave half empty (512 blocks of 3000 keys on average: 250 us whole, 228 in two,
  // 296 in four, since a CTA's start costs as much as 4 tiles; 8 blocks of 4096 keys
  // in 8 parts each 28 us, in 16 4 us more)
  const int64_t tiles = ((int64_t)d.max_blocks * d.page_tokens + kTile - 1) / kTile, wave = 148 * G::kPerSm;
  a.split = 1;
  while (a.split < kSplits && tiles >= a.split * 8 &&
         (items * a.split * 2 <= wave || (items * a.split > wave && items * a.split < 2 * wave)))
    a.split *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * a.split));
  cfg.blockDim = dim3(kThreadsP);
  cfg.dynamicSmemBytes = G::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_prefill_kernel<T, HD>, d, static_cast<const T*>(q.p),
                            static_cast<T*>(const_cast<void*>(o.p)), a);
}

}  // namespace

cudaError_t kv4_prefill_launch(const Kv4Dev& d, int head_dim, int max_new, const Kv4Tensor& q, int group, int dtype,
                               const float* rope, float scale_log2, const Kv4Tensor& out, cudaStream_t s) {
  PrefillArgs a{};
  a.q_tok = q.token, a.q_head = q.head, a.o_tok = out.token, a.o_head = out.head;
  a.rope = rope;
  a.group = group;
  a.max_new = max_new;
  a.scale_log2 = scale_log2;
  a.row_blocks = (int)(((int64_t)max_new * group + kM - 1) / kM);
  const int64_t items = (int64_t)a.row_blocks * d.n_kv * d.batch;
  const bool wide = head_dim == 128;
  if (dtype == WPK_F32)
    return wide ? launch<float, 128>(d, q, out, a, items, s) : launch<float, 64>(d, q, out, a, items, s);
  if (dtype == WPK_BF16)
    return wide ? launch<__nv_bfloat16, 128>(d, q, out, a, items, s)
                : launch<__nv_bfloat16, 64>(d, q, out, a, items, s);
  return wide ? launch<__half, 128>(d, q, out, a, items, s) : launch<__half, 64>(d, q, out, a, items, s);
}

}  // namespace wpk
