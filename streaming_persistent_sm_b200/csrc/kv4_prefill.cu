// Attention over a paged KV cache held in 4 bits, for many query rows per kv
// head (runs of new tokens): 128 rows a CTA on tcgen05.
//
// A tile of 64 keys is expanded to fp16 operands in shared memory once for all
// 128 rows, K and V alike: a key's row of 128 bytes (64 dims), word j of its codes
// as 16 bytes j, so that Q's dims and the output's stand in the same order (4j,
// HD/2 + 4j, 4j + 1, ...).  For S = Q K^T K is K-major, for O = P V the same layout
// of V is MN-major: nothing is transposed.  What the operands hold depends on what
// the type has to keep:
//  * bf16: the values s c + z rounded to fp16 (2^-12, as Q and P), times a power of
//    two that follows the largest value so far;
//  * fp16, fp32: the codes, which are exact (odd nibbles at 16 times their value);
//    scales and offsets enter per key around the products, as for few rows.
// S goes to TMEM; two threads a row (32 keys each) turn it into P, in TMEM too,
// which is the first operand of O = P V; the O of a tile is added to the row's
// registers, rounded.
//
// Bound by the arithmetic around the products: for a tile the 128 rows' exp2
// alone take an SM 512 cycles, the products of heads of 64 some 250.  While a
// tile's O is computed the next one is expanded, and two CTAs share an SM.
// Splits of the keys over a cluster join as for few rows.
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

constexpr int kM = 128;        // query rows of a CTA
constexpr int kTile = 64;      // keys of a tile
constexpr int kThreadsP = 256;
constexpr int kSplits = 8;

template <typename T, int HD>
struct PGeo {
  using P = Keep<T>;
  static constexpr int kWords = HD / 8;                       // of a row's codes
  static constexpr int kQBytes = kM * HD * 2;                 // one of Q's parts
  static constexpr int kKBytes = kTile * HD * 2, kVBytes = HD * kTile * 2;
  static constexpr int kQ = 0, kQl = kQ + kQBytes, kK = kQl + (P::kQLow ? kQBytes : 0), kV = kK + 2 * kKBytes;
  static constexpr int kOps = kV + 2 * kVBytes;               // operands: 1024-byte aligned
  static constexpr int kCodes = kTile * HD / 2;               // staging: K's codes, V's, the scales
  static constexpr int kStage = 2 * kCodes + kTile * 8;
  static constexpr int kScales = kOps + 2 * kStage;           // the tile's scales as floats
  static constexpr int kRed = kScales + kTile * 16;           // [2][kM] floats: both threads of a row
  static constexpr int kBytes = kRed + 2 * kM * 4;
  // after the keys: O [kM][HD], offsets, sums
  static constexpr int kJoin = kM * (HD + 2) * 4;
  static constexpr int kSmem = (kBytes > kJoin ? kBytes : kJoin) + 1024;  // and what aligns it
  static constexpr int kS = 0, kO = 64, kCols = HD == 64 ? 128 : 256;  // TMEM: S (P over it), O
  static constexpr int kPerSm = HD == 64 ? 2 : 1;
  static constexpr bool kValues = P::kBf16;                   // operands hold values, not codes
};

struct PrefillArgs {
  int64_t q_tok, q_head, o_tok, o_head;
  const float* rope;
  int group, max_new, row_blocks, split;
  float scale_log2;
};

// Waits for a phase of the products' barrier; false after a second (nothing but
// a lost product would take so long): the rows then answer NaN.
__device__ __forceinline__ bool wait_products(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 63) == 0 && globaltimer() - t0 > 1000000000ull) return false;
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(kThreadsP, PGeo<T, HD>::kPerSm)
    kv4_prefill_kernel(const Kv4Dev c, const T* __restrict__ q, T* __restrict__ out, const PrefillArgs a) {
  using G = PGeo<T, HD>;
  using P = Keep<T>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2];  // S ready, O ready
  __shared__ uint32_t s_tmem, s_vexp[2];
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
  const int n_tiles = (n_keys + kTile - 1) / kTile;

  if (tid == 0) {
    mbar_init(&bars[0], 1);
    mbar_init(&bars[1], 1);
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&s_tmem, G::kCols);
    tmem_relinquish();
  }

  // Copies of a tile: a thread takes one 16-byte piece of K's codes and one of
  // V's (heads of 64: half of the threads), the last warp the scales as well.
  constexpr int kPieces = kTile * HD / 2 / 16;  // of K, and of V: 128 or 256
  const int32_t* table = c.table + (int64_t)b * c.max_blocks;
  const int codes = c.page_tokens * (HD / 2);
  const int p_key = tid / (HD / 32), p_at = tid % (HD / 32) * 16;  // the piece's key in the tile, byte in its row
  const int s_lane = tid - (kThreadsP - 32);                       // the last warp copies the scales, 4 keys a lane
  const int s_key = 4 * (s_lane & 15);
  auto page_of = [&](int tile, int key_in) -> int {
    const int64_t key = (int64_t)tile * kTile + key_in;
    return key < n_keys ? table[kv4_slot(c, (int)key)] : -1;
  };
  auto copy = [&](int tile, int block, int s_block, uint8_t* stage) {
    if (tid < kPieces && block >= 0 && block < c.n_blocks) {
      const int key = tile * kTile + p_key, row = key - kv4_slot(c, key) * c.page_tokens;
      const uint8_t* src = kv4_page(c, block, head) + row * (HD / 2) + p_at;
      cp16(stage + p_key * (HD / 2) + p_at, src);
      cp16(stage + G::kCodes + p_key * (HD / 2) + p_at, src + codes);
    }
    if (s_lane >= 0 && s_block >= 0 && s_block < c.n_blocks) {
      const int key = tile * kTile + s_key, row = key - kv4_slot(c, key) * c.page_tokens;
      cp16(stage + 2 * G::kCodes + s_lane * 16,
           kv4_page(c, s_block, head) + 2 * codes + ((s_lane >> 4) * c.page_tokens + row) * 4);
    }
    cp_commit();
  };
  int block = tid < kPieces ? page_of(rank, p_key) : -1, s_block = s_lane >= 0 ? page_of(rank, s_key) : -1;
  // Runs of 16 keys that have a place, of the tile to come: each warp's first
  // lanes look them up for themselves.
  auto runs_of = [&](int tile) -> uint32_t {
    int id = -1;
    if (lane < 4) id = page_of(tile, 16 * lane);
    return __ballot_sync(0xFFFFFFFFu, id >= 0 && id < c.n_blocks) & 15u;
  };
  copy(rank, block, s_block, smem + G::kOps);
  uint32_t have_next = runs_of(rank);
  if (tid < kPieces) block = page_of(rank + a.split, p_key);
  if (s_lane >= 0) s_block = page_of(rank + a.split, s_key);

  // Q: the thread's half of the row's units, times scale log2(e) and the power of
  // two that brings the row's largest value to 2^13..2^14
  float* red = reinterpret_cast<float*>(smem + G::kRed);
  float k_mul, z_mul;  // a logit is k_mul (s S + z z_mul)
  {
    constexpr int kU = G::kWords / 2;  // units of the thread
    float x[kU][8];                    // dims 4u .. 4u + 3, then HD / 2 + 4u ..
    float top = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int u = hw * kU + i;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[i][e] = 0.f;
      if (placed) {
        const T* p = q + (int64_t)(q0 + my_new) * a.q_tok + my_head * a.q_head + 4 * u;
        load4(p, x[i]);
        load4(p + HD / 2, x[i] + 4);
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
  const uint32_t tmem = s_tmem, mine = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
  const uint32_t smem0 = smem_u32(smem);

  float m = -INFINITY, off = 0.f;  // as for few rows; the same in both threads of a row
  F2 l2 = pair(0.f, 0.f), py2 = l2;
  float o[HD / 2];  // of the row: columns hw HD / 2 .., dims hw HD / 4 .. and those HD / 2 further, in turn
#pragma unroll
  for (int i = 0; i < HD / 2; ++i) o[i] = 0.f;
  // biased exponents: V's largest scale (codes: P carries V's scales, times a
  // power of two that makes it fit) or value, K's largest value
  uint32_t v_exp = 41, k_exp = 41;
  bool ok = true;
  int n_done = 0;  // tiles before this one
  // adds the O of the tile before, which was computed meanwhile
  auto add_o = [&]() {
    ok = ok && wait_products(&bars[1], (n_done - 1) & 1);
    tc_fence_after();
#pragma unroll
    for (int i = 0; i < HD / 2; i += 32) {
      float v[32];
      tmem_ld16x2(mine + G::kO + hw * (HD / 2) + i, v);
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const float2 t = split(add2(pair(o[i + e], o[i + e + 1]), pair(v[e], v[e + 1])));
        o[i + e] = t.x;
        o[i + e + 1] = t.y;
      }
    }
    tc_fence_before();
  };
#pragma unroll 1
  for (int tile = rank; tile < n_tiles; tile += a.split, ++n_done) {
    const int buf = n_done & 1, key0 = tile * kTile;
    const uint32_t have = have_next;
    cp_wait<0>();
    __syncthreads();  // the tile's codes are here; every thread is done with the other staging buffer
    copy(tile + a.split, block, s_block, smem + G::kOps + (buf ^ 1) * G::kStage);
    have_next = runs_of(tile + a.split);
    if (tid < kPieces) block = page_of(tile + 2 * a.split, p_key);
    if (s_lane >= 0) s_block = page_of(tile + 2 * a.split, s_key);

    const uint8_t* stage = smem + G::kOps + buf * G::kStage;
    const uint32_t* sz = reinterpret_cast<const uint32_t*>(stage + 2 * G::kCodes);  // K's [kTile], V's
    float4* scales = reinterpret_cast<float4*>(smem + G::kScales);  // codes: K's [32], V's [32], two keys each
    uint32_t v_new = v_exp;
    int bad = INT_MAX;  // values: the first key whose V is NaN
    __half2 vs2[2], vz2[2];  // values: scale and offset of this thread's key, of K and V
    if constexpr (G::kValues) {
      const uint2 kw = *reinterpret_cast<const uint2*>(sz + 2 * lane);
      const uint2 vw = *reinterpret_cast<const uint2*>(sz + kTile + 2 * lane);
      const bool there = (have >> (lane >> 3)) & 1u;
      const bool ta = there && key0 + 2 * lane < n_keys, tb = there && key0 + 2 * lane + 1 < n_keys;
      auto reach = [](uint32_t w) {  // the row's largest size; 0 if it is NaN
        const float s = __uint_as_float(w << 16), z = __uint_as_float(w & 0xFFFF0000u);
        return fmaxf(fmaxf(0.f, fabsf(z)), fabsf(fmaf(15.f, s, z)));
      };
      const float kt = fmaxf(ta ? reach(kw.x) : 0.f, tb ? reach(kw.y) : 0.f);
      const float vt = fmaxf(ta ? reach(vw.x) : 0.f, tb ? reach(vw.y) : 0.f);
      k_exp = max(k_exp, min(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(kt)) >> 23, 254u));
      v_new = max(v_new, min(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(vt)) >> 23, 254u));
      const bool na = ta && (vw.x & 0x7FFF0000u) > 0x7F800000u, nb = tb && (vw.y & 0x7FFF0000u) > 0x7F800000u;
      if (__any_sync(0xFFFFFFFFu, na || nb))
        bad = (int)__reduce_min_sync(0xFFFFFFFFu, na ? 2 * lane : nb ? 2 * lane + 1 : INT_MAX);
      // the thread's own key, values at 2^14..2^15 for the largest
      const int key = tid >> 2;
      const bool mine_there = ((have >> (key >> 4)) & 1u) && key0 + key < n_keys;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w = mine_there ? sz[e * kTile + key] : 0u;
        const float f = __uint_as_float((268u - (e ? v_new : k_exp)) << 23);
        float z = __uint_as_float(w & 0xFFFF0000u);
        if (e && z != z) z = 0.f;  // its NaN must not reach rows that do not see it
        vs2[e] = __float2half2_rn(__uint_as_float(w << 16) * f);
        vz2[e] = __float2half2_rn(z * f);
      }
    } else if (warp == 0 || warp == 4) {
      // the scales as floats, two keys a lane; zeros for keys without a place
      const uint32_t* half_sz = sz + (hw ? kTile : 0);
      const bool there = (have >> (lane >> 3)) & 1u;
      const uint32_t wa = there && key0 + 2 * lane < n_keys ? half_sz[2 * lane] : 0u;
      const uint32_t wb = there && key0 + 2 * lane + 1 < n_keys ? half_sz[2 * lane + 1] : 0u;
      const bool centre = hw ? P::kCentreV : P::kCentreK;
      const float sa = __uint_as_float(wa << 16), sb = __uint_as_float(wb << 16);
      const float za = __uint_as_float(wa & 0xFFFF0000u), zb = __uint_as_float(wb & 0xFFFF0000u);
      scales[32 * hw + lane] =
          make_float4(sa, sb, centre ? fmaf(8.f, sa, za) : za, centre ? fmaf(8.f, sb, zb) : zb);
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, max(wa << 16, wb << 16));
      if (hw && lane == 0) s_vexp[buf] = min(top >> 23, 254u);
    }
    // K and V: words of a key to 16-byte units of its rows, two or four a thread
    {
      const int key = tid >> 2, part = tid & 3;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        uint8_t* rows_of = smem + (kv ? G::kV + buf * G::kVBytes : G::kK + buf * G::kKBytes) + key * 128;
        auto even = [&](uint32_t x) -> uint32_t {
          if constexpr (G::kValues) {
            const uint32_t y = centred_even<0>(x);
            const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&y), vs2[kv], vz2[kv]);
            return *reinterpret_cast<const uint32_t*>(&v);
          } else {
            return kv ? codes_even<P::kCentreV>(x) : codes_even<P::kCentreK>(x);
          }
        };
        const __half2 s16 = G::kValues ? __hmul2(vs2[kv], __float2half2_rn(0.0625f)) : __half2{};
        auto odd = [&](uint32_t x) -> uint32_t {
          if constexpr (G::kValues) {
            const uint32_t y = centred_odd<0>(x);
            const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&y), s16, vz2[kv]);
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
    }
    if (n_done && tid == 0) ok = ok && wait_products(&bars[1], (n_done - 1) & 1);  // S lies over the tile before's P
    fence_proxy_async_smem();  // the products read these generic-proxy writes
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_f16(kM, kTile, false);
#pragma unroll
      for (int kk = 0; kk < HD / 16; ++kk) {
        const uint64_t kd = sdesc_k_sw128(smem0 + G::kK + buf * G::kKBytes + (kk >> 2) * (kTile * 128) + (kk & 3) * 32);
        const uint32_t qa = (kk >> 2) * (kM * 128) + (kk & 3) * 32;
        umma_f16(tmem + G::kS, sdesc_k_sw128(smem0 + G::kQ + qa), kd, idesc, kk > 0);
        if (P::kQLow) umma_f16(tmem + G::kS, sdesc_k_sw128(smem0 + G::kQl + qa), kd, idesc, 1u);
      }
      umma_commit(&bars[0]);
    }
    if (n_done) add_o();
    ok = ok && wait_products(&bars[0], n_done & 1);
    tc_fence_after();

    // the row's logits of 32 keys, k_tile times them in units of log2
    float x[32];
    tmem_ld16x2(mine + G::kS + 32 * hw, x);
    const float k_tile = G::kValues ? k_mul * __uint_as_float((k_exp - 14u) << 23) : k_mul;
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
    const bool part = have != 15u || key0 + kTile > all_see;
    if (part) {  // scores without a place, or behind the row's last key
#pragma unroll
      for (int i = 0; i < 32; ++i)
        if (!((have >> (2 * hw + (i >> 4))) & 1u) || key0 + 32 * hw + i > last) x[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 32; i += 2) top = max3(top, x[i], x[i + 1]);
    red[hw * kM + r] = top;
    tc_fence_before();
    __syncthreads();  // and every S is read: P may lie over it
    tc_fence_after();
    const float m_new = fmaxf(m, fmaxf(top, red[(hw ^ 1) * kM + r]) * k_tile);
    if constexpr (!G::kValues) v_new = max(v_exp, s_vexp[buf]);
    if (m_new != m || v_new != v_exp) {
      // P reaches 2^15: as a weight, or times V's largest scale
      const float off_new = (m_new == -INFINITY ? 0.f : m_new) - (G::kValues ? 15.f : (float)(141 - (int)v_new));
      const float fade = m == -INFINITY ? 0.f : ex2(off - off_new);
      // operands that are values shrink as the largest one grows
      const float o_fade = G::kValues ? fade * __uint_as_float(max(127 - (int)(v_new - v_exp), 0) << 23) : fade;
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
      v_exp = v_new;
    }
    if (bad <= last - key0) l2 = pair(NAN, NAN);  // `last` is -1 for rows without a key
    const F2 down = pair(-off, -off), k2 = pair(k_tile, k_tile);
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
      tmem_st8(mine + G::kS + 16 * hw + 8 * g, hi);
      if (P::kPLow) tmem_st8(mine + G::kS + 32 + 16 * hw + 8 * g, lo);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    if (tid == 0) {
      tc_fence_after();
      constexpr uint32_t idesc = idesc_f16(kM, HD, false) | 1u << 16;  // V is MN-major
#pragma unroll
      for (int kk = 0; kk < kTile / 16; ++kk) {
        // 16 keys: two groups of 8 rows; the next 64 dims are a leading offset away
        const uint64_t vd = sdesc_k_sw128(smem0 + G::kV + buf * G::kVBytes + kk * 2048) +
                            ((uint64_t)(kTile * 128 / 16 - 1) << 16);
        umma_f16_ta(tmem + G::kO, tmem + G::kS + 8 * kk, vd, idesc, kk > 0);
        if (P::kPLow) umma_f16_ta(tmem + G::kO, tmem + G::kS + 32 + 8 * kk, vd, idesc, 1u);
      }
      umma_commit(&bars[1]);
    }
  }
  if (n_done) add_o();
  cp_wait<0>();  // before this memory holds other things
  ok = __syncthreads_and(ok);
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
    const float back = __uint_as_float(v_exp - 29u << 23);
#pragma unroll
    for (int i = 0; i < HD / 2; ++i)
      o[i] = G::kValues ? o[i] * back : fmaf(o[i], i >> 1 & 1 ? even * 0.0625f : even, py);
    const float sum = G::kValues ? l * 0x1p-15f : l;
    const float none = ok ? 0.f : NAN;
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
      join[r * (HD + 2) + HD] = m == -INFINITY ? -INFINITY : G::kValues ? m : off;
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
  // CTAs that share a block's keys, while the GPU (148 SMs) is not full and each
  // has some tiles
  const int64_t tiles = ((int64_t)d.max_blocks * d.page_tokens + kTile - 1) / kTile;
  a.split = 1;
  while (a.split < kSplits && items * a.split * 2 <= 148 * G::kPerSm && tiles >= a.split * 8) a.split *= 2;
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
  if (items > INT_MAX / kSplits) return cudaErrorInvalidValue;
  const bool wide = head_dim == 128;
  if (dtype == WPK_F32)
    return wide ? launch<float, 128>(d, q, out, a, items, s) : launch<float, 64>(d, q, out, a, items, s);
  if (dtype == WPK_BF16)
    return wide ? launch<__nv_bfloat16, 128>(d, q, out, a, items, s)
                : launch<__nv_bfloat16, 64>(d, q, out, a, items, s);
  return wide ? launch<__half, 128>(d, q, out, a, items, s) : launch<__half, 64>(d, q, out, a, items, s);
}

}  // namespace wpk
