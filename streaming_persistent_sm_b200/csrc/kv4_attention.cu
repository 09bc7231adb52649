// Attention over a paged KV cache held in 4 bits, for few query rows per kv
// head (single tokens).
//
// A row x of the cache is s c + z with c in 0..15, or s d + y with d = c - 8 and
// y = z + 8 s, so
//   q . k = s (sum_i q_i c_i) + z (sum_i q_i),
//   sum_t p_t v_t = sum_t (p_t s_t) d_t + sum_t p_t y_t:
// the matrix products run on the codes themselves, and scales and offsets enter
// per token around them.  A code needs hardly any conversion: a nibble alone in
// the low mantissa bits of an fp16 is the number c 2^-24 (c 2^-20 for the next
// nibble), exactly, so one AND makes an operand of two codes; with the bits of
// 1024 above it, it is 1024 + c (1024 + 16 c), and a subtraction leaves d.  V
// takes the centred codes: a sum over thousands of tokens all of one sign would
// lose what the centred one keeps (1.2e-3 against 2e-4 at 131072 tokens, fp16, before
// each step had sums of its own).
//
// One warp takes 64 keys at a time for up to 8 query rows: S = Q K^T as
// m16n8k16 products (rows 0-7 Q rounded to fp16, rows 8-15 what the rounding
// left, so Q has 22 bits), one online softmax over its keys, and O^T = V^T P^T
// with the P of S's registers as the second operand, unmoved.  With so few rows
// the tensor pipe is idle most of the time and the cache's bytes are the bound;
// 128-row tcgen05 tiles would pad 8 rows to 128.
//
// The keys of a (sequence, kv head, 8 rows) are split over the warps of a
// cluster of CTAs, which join their partial softmaxes through distributed shared
// memory: one launch, no workspace, no atomics, so the result does not depend
// on timing.  Each warp streams its pages through its own ring of shared-memory
// stages with 16-byte asynchronous copies; nothing spins.
//
// Bound by the instructions around the products, some 680 a warp's step, and for
// little work by latency.  Measured: 32 sequences of up to 8192 keys, 32 heads of 64
// over 8 kv heads, bf16: 42 us (2.8 TB/s of cache); one of 131072, 64 heads of 128
// over 8, fp16: 95 us (1.5 TB/s); one of 624: 7.6 us.
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

constexpr int kRows = 8;    // query rows of a CTA (the N of the P V product)
constexpr int kKeys = 64;   // keys of a warp's step
constexpr int kMaxSplit = 16;

// The tcgen05 kernel's calls: from 64 query rows a (sequence, kv head) on, where
// this kernel would have much to do (blocks of 8 rows times the keys that a table
// names).  Measured (us, this kernel / that one, bf16, heads of 64, 8 kv heads):
// 16 sequences of 4096 keys: 48 rows 66 / 78, 64 rows 75 / 78, 128 rows 144 / 81;
// of 512 keys: 64 rows 20 / 23, 96 rows 27 / 23, 128 rows 34 / 24; one of 4096:
// 128 rows 17 / 28.  fp16 and fp32 meet at 64 to 80 rows, heads of 128 at 48 to 56.
constexpr int kManyRows = 64;
constexpr int64_t kManyWork = 1 << 20;
bool many_rows(const Kv4Dev& d, int64_t rows) {
  return rows >= kManyRows && (double)((rows + 7) / 8 * d.n_kv) * d.batch >=
                                  (double)(kManyWork / ((int64_t)d.max_blocks * d.page_tokens));
}


// A CTA of WARPS warps: 4, of which an SM holds four (three at head_dim 128), or
// 12, one to an SM, where 16 CTAs a cluster would not fill the GPU otherwise.
template <int HD, int WARPS>
struct Geo {
  static constexpr int kPerSm = WARPS == 12 ? 1 : HD == 64 ? 4 : 3;
  static constexpr int kStages = HD == 64 && WARPS == 12 ? 3 : 2;
  static constexpr int kRowBytes = HD / 2;
  static constexpr int kStageBytes = kKeys * (2 * kRowBytes + 8);  // K codes, V codes, K (s, z), V (s, z)
  static constexpr int kWarpBytes = kStages * kStageBytes + kKeys * 16;  // and the step's scales as floats
  static constexpr int kRing = WARPS * kWarpBytes;
  // after the keys: every warp's rows (O, then m, l and the sum of p y), then the CTA's
  static constexpr int kWarpPart = kRows * (HD + 3);  // floats
  static constexpr int kCtaPart = kRows * (HD + 2);
  static constexpr int kJoin = (WARPS * kWarpPart + kCtaPart) * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

struct AttnArgs {
  int64_t q_tok, q_head, o_tok, o_head;
  const float* rope;
  int group, max_new, row_blocks, split;  // split: CTAs of a cluster
  float scale_log2;                       // scale * log2(e)
};

// d += a b: a 16 x 16 (fp16, rows), b 16 x 8 (fp16, columns), d fp32.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// In a warp, lane = 4 g + t.  S's columns 2t and 2t + 1 of the n-th group of 8
// keys are its keys t and 7 - t: with this order neither the K rows (8 at a
// time) nor the V words (4 rows x 8 words) of a step meet in a bank.
template <typename T, int HD, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, Geo<HD, WARPS>::kPerSm)
    kv4_attention_kernel(const Kv4Dev c, const T* __restrict__ q, T* __restrict__ out, const AttnArgs a) {
  using G = Geo<HD, WARPS>;
  using P = Keep<T>;
  constexpr int WPL = HD / 32;  // words of a K row that a lane multiplies
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % a.split;
  int item = blockIdx.x / a.split;
  const int rb = item % a.row_blocks;
  item /= a.row_blocks;
  const int head = item % c.n_kv, b = item / c.n_kv;
  if (b >= kv4_sequences(c)) return;  // as for every CTA of the cluster

  // This warp's first step's keys, four runs of 16 inside a page each (one run of
  // 64 where pages hold whole steps).  Lane i < runs keeps run i's place in the
  // table from step to step.  The first page ids are asked for before it is known
  // how many keys there are.
  const int stride = a.split * WARPS, first = rank * WARPS + warp;
  const bool whole = c.page_tokens % kKeys == 0;
  const int32_t* table = c.table + (int64_t)b * c.max_blocks;
  const int ahead = stride * kKeys, skip_slots = ahead / c.page_tokens, skip_rows = ahead % c.page_tokens;
  int64_t key = (int64_t)first * kKeys + 16 * lane;
  int slot = (int)(key / c.page_tokens), row = (int)(key % c.page_tokens);
  auto ask = [&]() {  // the id of the page of the run
    return lane < (whole ? 1 : 4) && slot < c.max_blocks ? table[slot] : -1;
  };
  int block = ask();

  const int pos0 = c.pos[b];
  int q0, n_new;
  kv4_new(c, b, &q0, &n_new);
  const int64_t rows = (int64_t)min(n_new, a.max_new) * a.group;
  const int64_t r0 = (int64_t)rb * kRows;
  if (r0 >= rows) return;

  // the rows' positions and the keys [0, n_keys) that any of them sees
  const int64_t cap = (int64_t)c.max_blocks * c.page_tokens;
  const int64_t my_row = r0 + g;
  const int my_new = my_row < rows ? (int)((uint32_t)my_row / (uint32_t)a.group) : 0;
  const int64_t my_pos = (int64_t)pos0 + my_new;
  const bool placed = my_row < rows && pos0 >= 0 && my_pos < c.rope_positions;
  const int last = placed ? (int)(my_pos < cap ? my_pos : cap - 1) : -1;  // the row's last key
  const int64_t lo_pos = pos0 + r0 / a.group, hi_pos = pos0 + (min(r0 + kRows, rows) - 1) / a.group;
  const int n_keys = pos0 < 0 ? 0 : (int)min(hi_pos + 1, cap);
  const int all_see = (int)min(lo_pos + 1, cap);  // keys below it are seen by every row that has a position
  const int n_steps = n_keys ? (n_keys - 1) / kKeys + 1 : 0;
  const int codes = c.page_tokens * G::kRowBytes;

  uint8_t* ring = smem + warp * G::kWarpBytes;
  float4* scales = reinterpret_cast<float4*>(ring + G::kStages * G::kStageBytes);
  // Copies the step's keys to `stage`, as far as they have a place, moves on to
  // the warp's next step, and says which runs came (4 bits).
  auto issue = [&](uint8_t* stage) -> uint32_t {
    const bool here = block >= 0 && block < c.n_blocks && key < n_keys;
    const uint32_t came = __ballot_sync(0xFFFFFFFFu, here) & 15u;
    const unsigned long long base = here ? reinterpret_cast<unsigned long long>(kv4_page(c, block, head)) : 0;
    const int j = lane & 15, of_v = lane >> 4;  // 16 lanes copy K's (s, z), 16 V's: four keys each
    uint8_t* sz = stage + 2 * kKeys * G::kRowBytes + lane * 16;
    uint32_t held;
    if (whole) {
      const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, base, 0));
      const int at = __shfl_sync(0xFFFFFFFFu, row, 0);
      held = came & 1 ? 15u : 0;
      if (page) {
        const uint8_t* src = page + at * G::kRowBytes + lane * 16;
        uint8_t* dst = stage + lane * 16;
#pragma unroll
        for (int o = 0; o < kKeys * G::kRowBytes; o += 512) {
          cp16(dst + o, src + o);
          cp16(dst + kKeys * G::kRowBytes + o, src + codes + o);
        }
        cp16(sz, page + 2 * codes + (of_v * c.page_tokens + at + 4 * j) * 4);
      }
    } else {
      held = came;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, base, i));
        const int at = __shfl_sync(0xFFFFFFFFu, row, i);
        if (!page) continue;
        const uint8_t* src = page + at * G::kRowBytes + lane * 16;
        uint8_t* dst = stage + i * 16 * G::kRowBytes + lane * 16;
#pragma unroll
        for (int o = 0; o < 16 * G::kRowBytes; o += 512) {
          cp16(dst + o, src + o);
          cp16(dst + kKeys * G::kRowBytes + o, src + codes + o);
        }
      }
      const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, base, j >> 2));
      const int at = __shfl_sync(0xFFFFFFFFu, row, j >> 2);
      if (page) cp16(sz, page + 2 * codes + (of_v * c.page_tokens + at + 4 * (j & 3)) * 4);
    }
    cp_commit();
    key += ahead;
    slot += skip_slots;
    row += skip_rows;
    if (row >= c.page_tokens) {
      row -= c.page_tokens;
      ++slot;
    }
    block = ask();
    return held;
  };
  uint32_t held = 0;  // 4 bits a stage: runs that came
#pragma unroll
  for (int s = 0; s < G::kStages - 1; ++s) held |= issue(ring + s * G::kStageBytes) << (4 * s);

  // Q: lane (g, t) holds dims 4 WPL t .. + 4 WPL of both halves of row g, times
  // scale log2(e) and a power of two that brings the row's largest value to
  // 2^13..2^14, each row by its own; k_mul takes it back
  uint32_t qa[2 * WPL][4];
  float k_mul, logit_z;
  {
    float lo[4 * WPL], hi[4 * WPL];
#pragma unroll
    for (int i = 0; i < 4 * WPL; ++i) lo[i] = hi[i] = 0.f;
    if (placed) {
      const T* p = q + (int64_t)(q0 + my_new) * a.q_tok +
                   (head * a.group + (int)((uint32_t)my_row % (uint32_t)a.group)) * a.q_head + 4 * WPL * t;
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        load4(p + 4 * i, lo + 4 * i);
        load4(p + HD / 2 + 4 * i, hi + 4 * i);
      }
      if (a.rope) {
        const float* r = a.rope + (my_pos * (HD / 2) + 4 * WPL * t) * 2;
#pragma unroll
        for (int i = 0; i < 2 * WPL; ++i) {
          float cs[4];
          load4(r + 4 * i, cs);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float x = lo[2 * i + e], y = hi[2 * i + e];
            lo[2 * i + e] = x * cs[2 * e] - y * cs[2 * e + 1];
            hi[2 * i + e] = y * cs[2 * e] + x * cs[2 * e + 1];
          }
        }
      }
    }
    float top = 0.f, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4 * WPL; ++i) {
      lo[i] *= a.scale_log2;
      hi[i] *= a.scale_log2;
      top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
      sum += lo[i] + hi[i];
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
    logit_z = sum;
    // exponent fields: the power of two is 2^(140 - e), within fp32 (rows of no
    // finite value, or below 2^-100, as they are)
    const uint32_t e = max(__float_as_uint(top) >> 23, 27u);
    const float mul = __uint_as_float(e < 255u ? (267u - e) << 23 : 0x3F800000u);
    k_mul = (P::kCentreK ? 1.f : 16777216.f) / mul;
#pragma unroll
    for (int k = 0; k < 2 * WPL; ++k) {
#pragma unroll
      for (int odd = 0; odd < 2; ++odd) {  // odd nibbles stand 16 times as high
        const int i = 4 * (k >> 1) + 2 * (k & 1) + odd;
        const float m = odd ? mul * 0.0625f : mul;
        const float x = lo[i] * m, y = hi[i] * m;
        const uint32_t h = pack_f16(x, y);
        const float2 back = unpack_f16(h);
        qa[k][2 * odd] = h;
        qa[k][2 * odd + 1] = P::kQLow ? pack_f16(x - back.x, y - back.y) : 0u;
      }
    }
  }

  // Running sums of the online softmax, all of them 2^-off times the true ones:
  // off = m - 14, where m is at least a key's logit and its V's exponent together
  // (v_key_exp, kSpread), for all keys so far.  So P s, which the second product
  // takes in fp16, stays below 2^15 whatever the scales, and P y within fp32.
  float m = -INFINITY, off = 0.f;  // of row g
  F2 l2 = pair(0.f, 0.f), py2 = l2;  // l and the sum of p y, of this lane's keys only, in two halves
  float o[2 * WPL][4];               // rows 2t, 2t + 1: dims 4g + .. of both halves
#pragma unroll
  for (int i = 0; i < 2 * WPL; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  uint32_t v_most = kLeastExp, v_least = 255;  // V's exponents so far (the least: of this lane's keys with a range)
  int cur = 0;
#pragma unroll 1
  for (int step = first; step < n_steps; step += stride) {
    cp_wait<G::kStages - 2>();
    __syncwarp();
    {  // every lane is done with the previous step's stage: refill it
      const int to = cur == 0 ? G::kStages - 1 : cur - 1;
      held = (held & ~(15u << (4 * to))) | issue(ring + to * G::kStageBytes) << (4 * to);
    }
    const uint8_t* stage = ring + cur * G::kStageBytes;
    const uint32_t have = (held >> (4 * cur)) & 15u;
    cur = cur + 1 == G::kStages ? 0 : cur + 1;
    const int key0 = step * kKeys;

    // the step's scales as floats: lane 4 n + t's keys are 8 n + t and 8 n + 7 - t,
    // as S's columns have them; zeros for keys without a place (whatever the stage
    // held)
    bool spread;
    {
      const uint32_t* ksz = reinterpret_cast<const uint32_t*>(stage + 2 * kKeys * G::kRowBytes);
      const int ja = 8 * g + t, jb = 8 * g + 7 - t;
      const bool there = (have >> (g >> 1)) & 1u;
      const bool in_a = there && key0 + ja < n_keys, in_b = there && key0 + jb < n_keys;
      const uint32_t ka = in_a ? ksz[ja] : 0u, kb = in_b ? ksz[jb] : 0u;
      const uint32_t va = in_a ? ksz[kKeys + ja] : 0u, vb = in_b ? ksz[kKeys + jb] : 0u;
      auto s_of = [](uint32_t w) { return __uint_as_float(w << 16); };
      auto z_of = [](uint32_t w, bool centre) {
        const float z = __uint_as_float(w & 0xFFFF0000u);
        return centre ? fmaf(8.f, __uint_as_float(w << 16), z) : z;
      };
      scales[lane] = make_float4(s_of(ka), s_of(kb), z_of(ka, P::kCentreK), z_of(kb, P::kCentreK));
      const float4 vs = make_float4(s_of(va), s_of(vb), z_of(va, P::kCentreV), z_of(vb, P::kCentreV));
      scales[32 + lane] = vs;
      const uint32_t ea = v_key_exp(vs.x, vs.z), eb = v_key_exp(vs.y, vs.w);
      v_most = max(v_most, __reduce_max_sync(0xFFFFFFFFu, max(ea, eb)));
      v_least = min(v_least, min(vs.x != 0.f ? ea : 255u, vs.y != 0.f ? eb : 255u));
      spread = __any_sync(0xFFFFFFFFu, v_least + kSpread < v_most);
    }
    __syncwarp();

    // S, and the logits in units of log2
    float x[16];
    const F2 z2 = pair(logit_z, logit_z), k2 = pair(k_mul, k_mul);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      float s[4] = {0.f, 0.f, 0.f, 0.f};
      const int at = 8 * n + (g & 1 ? 7 - (g >> 1) : g >> 1);
      uint32_t w[WPL];
      if (WPL == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(stage + at * G::kRowBytes + t * 8);
        w[0] = v.x, w[1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + at * G::kRowBytes + t * 16);
        w[0] = v.x, w[1] = v.y, w[WPL - 2] = v.z, w[WPL - 1] = v.w;
      }
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        const uint32_t h = w[i] >> 8;
        const uint32_t k0 = P::kCentreK ? centred_even(w[i]) : w[i] & kEven;
        const uint32_t k1 = P::kCentreK ? centred_odd(w[i]) : w[i] & kOdd;
        const uint32_t k2 = P::kCentreK ? centred_even(h) : h & kEven, k3 = P::kCentreK ? centred_odd(h) : h & kOdd;
        mma16816(s, qa[2 * i][0], qa[2 * i][1], qa[2 * i][2], qa[2 * i][3], k0, k1);
        mma16816(s, qa[2 * i + 1][0], qa[2 * i + 1][1], qa[2 * i + 1][2], qa[2 * i + 1][3], k2, k3);
      }
      const float4 ks = scales[4 * n + t];
      F2 dot = pair(s[0], s[1]);
      if (P::kQLow) dot = add2(dot, pair(s[2], s[3]));
      const float2 xs = split(fma2(pair(ks.x, ks.y), mul2(dot, k2), mul2(pair(ks.z, ks.w), z2)));
      x[2 * n] = xs.x;
      x[2 * n + 1] = xs.y;
    }
    const bool part = have != 15u || key0 > all_see - kKeys;
    if (part) {  // scores without a place, or behind the row's last key
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (!((have >> (n >> 1)) & 1u) || key0 + 8 * n + (e ? 7 - t : t) > last) x[2 * n + e] = -INFINITY;
    }

    // softmax of row g over the step's keys
    float top;  // (sums rounded up, so that P does not pass its range however large the logits are)
    if (!spread) {
      top = max3(x[0], x[1], x[2]);
#pragma unroll
      for (int i = 3; i < 15; i += 2) top = max3(top, x[i], x[i + 1]);
      top = __fadd_ru(fmaxf(top, x[15]), (float)((int)v_most - 127));
    } else {
      top = -INFINITY;
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float4 vs = scales[32 + 4 * n + t];
        top = max3(top, __fadd_ru(x[2 * n], (float)((int)v_key_exp(vs.x, vs.z) - 127)),
                   __fadd_ru(x[2 * n + 1], (float)((int)v_key_exp(vs.y, vs.w) - 127)));
      }
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const float m_new = fmaxf(m, top);
    if (__any_sync(0xFFFFFFFFu, m_new != m)) {
      const float off_new = __fsub_ru(m_new == -INFINITY ? 0.f : m_new, 14.f);
      const float fade = m == -INFINITY ? 0.f : ex2(off - off_new);
      l2 = mul2(l2, pair(fade, fade));  // a NaN stays
      py2 = mul2(py2, pair(fade, fade));
      const float f0 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t), f1 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i) {
        o[i][0] *= f0, o[i][2] *= f0;
        o[i][1] *= f1, o[i][3] *= f1;
      }
      m = m_new;
      off = off_new;
    }
    const F2 down = pair(-off, -off);
    if (!part) {
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float4 vs = scales[32 + 4 * n + t];
        const float2 d = split(add2(pair(x[2 * n], x[2 * n + 1]), down));
        const F2 p = pair(ex2(d.x), ex2(d.y));
        l2 = add2(l2, p);
        py2 = fma2(p, pair(vs.z, vs.w), py2);
        const float2 w = split(mul2(p, pair(vs.x, vs.y)));
        x[2 * n] = w.x;
        x[2 * n + 1] = w.y;
      }
    } else {  // a key that the row does not see must not count, even with an offset of NaN
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        const float4 vs = scales[32 + 4 * n + t];
        const float pa = ex2(x[2 * n] - off), pb = ex2(x[2 * n + 1] - off);
        l2 = add2(l2, pair(pa, pb));
        py2 = fma2(pair(pa, pb), pair(x[2 * n] == -INFINITY ? 0.f : vs.z, x[2 * n + 1] == -INFINITY ? 0.f : vs.w), py2);
        x[2 * n] = pa * vs.x;
        x[2 * n + 1] = pb * vs.y;
      }
    }

    // O^T += V^T P^T, 16 keys at a time
    float own[2 * WPL][4];
#pragma unroll
    for (int i = 0; i < 2 * WPL; ++i) own[i][0] = own[i][1] = own[i][2] = own[i][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t b0 = pack_f16(x[4 * k], x[4 * k + 1]), b1 = pack_f16(x[4 * k + 2], x[4 * k + 3]);
      uint32_t d0 = 0, d1 = 0;
      if (P::kPLow) {
        const float2 r0 = unpack_f16(b0), r1 = unpack_f16(b1);
        d0 = pack_f16(x[4 * k] - r0.x, x[4 * k + 1] - r0.y);
        d1 = pack_f16(x[4 * k + 2] - r1.x, x[4 * k + 3] - r1.y);
      }
      const uint8_t* v = stage + kKeys * G::kRowBytes + 16 * k * G::kRowBytes;
      const uint32_t* v0 = reinterpret_cast<const uint32_t*>(v + t * G::kRowBytes);
      const uint32_t* v1 = reinterpret_cast<const uint32_t*>(v + (7 - t) * G::kRowBytes);
      const uint32_t* v2 = reinterpret_cast<const uint32_t*>(v + (8 + t) * G::kRowBytes);
      const uint32_t* v3 = reinterpret_cast<const uint32_t*>(v + (15 - t) * G::kRowBytes);
      uint32_t w[WPL / 2][4];
      if (WPL == 2) {
        w[0][0] = v0[g], w[0][1] = v1[g], w[0][2] = v2[g], w[0][3] = v3[g];
      } else {
        // rows of 16 words: half of the lanes take their second word first, so
        // that the four rows of a load do not meet in a bank
        const int f = g + 8 * (t >> 1), h = f ^ 8;
        uint32_t u[4] = {v0[f], v1[f], v2[f], v3[f]};
        uint32_t y[4] = {v0[h], v1[h], v2[h], v3[h]};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[0][i] = t < 2 ? u[i] : y[i];
          w[WPL / 2 - 1][i] = t < 2 ? y[i] : u[i];
        }
      }
#pragma unroll
      for (int i = 0; i < WPL / 2; ++i) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t a01 = __byte_perm(w[i][0], w[i][1], half ? 0x7632 : 0x5410);
          uint32_t a23 = __byte_perm(w[i][2], w[i][3], half ? 0x7632 : 0x5410);
#pragma unroll
          for (int pair = 0; pair < 2; ++pair) {
            float(&d)[4] = own[4 * i + 2 * half + pair];
            const uint32_t e0 = P::kCentreV ? centred_even(a01) : a01 & kEven;
            const uint32_t e1 = P::kCentreV ? centred_odd(a01) : a01 & kOdd;
            const uint32_t e2 = P::kCentreV ? centred_even(a23) : a23 & kEven;
            const uint32_t e3 = P::kCentreV ? centred_odd(a23) : a23 & kOdd;
            mma16816(d, e0, e1, e2, e3, b0, b1);
            if (P::kPLow) mma16816(d, e0, e1, e2, e3, d0, d1);
            a01 >>= 8;
            a23 >>= 8;
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 2 * WPL; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const float2 r = split(add2(pair(o[i][e], o[i][e + 1]), pair(own[i][e], own[i][e + 1])));
        o[i][e] = r.x;
        o[i][e + 1] = r.y;
      }
  }
  cp_wait<0>();
  const float2 lp = split(l2), pp = split(py2);
  float l = lp.x + lp.y, py = pp.x + pp.y;
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    py += __shfl_xor_sync(0xFFFFFFFFu, py, d);
  }

  // join the warps, then the cluster's CTAs
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
  {
    float* mine = part + warp * G::kWarpPart;
    const float even = P::kCentreV ? 1.f : 16777216.f;  // raw codes stand at 2^-24
#pragma unroll
    for (int i = 0; i < 2 * WPL; ++i) {
      // o[i]: word g + 8 (i / 4) of the row, its half (i / 2) % 2, nibble pair i % 2
      const int dim = 4 * (g + 8 * (i >> 2)) + (HD / 2) * ((i >> 1) & 1) + 2 * (i & 1);
      float* r = mine + 2 * t * HD + dim;
      r[0] = o[i][0] * even;
      r[HD] = o[i][1] * even;
      r[1] = o[i][2] * (even * 0.0625f);
      r[HD + 1] = o[i][3] * (even * 0.0625f);
    }
    if (t == 0) {
      mine[kRows * HD + g] = m == -INFINITY ? -INFINITY : off;
      mine[kRows * HD + kRows + g] = l;
      mine[kRows * HD + 2 * kRows + g] = py;
    }
  }
  __syncthreads();
  // a row that saw no key, or has no rotation, answers zeros
  auto store = [&](int e, float sum, float all) {
    const int rw = e / HD;
    if (r0 + rw >= rows) return;
    const uint32_t fresh = (uint32_t)(r0 + rw) / (uint32_t)a.group, h = (uint32_t)(r0 + rw) % (uint32_t)a.group;
    const float y = all == 0.f || (int64_t)pos0 + fresh >= c.rope_positions ? 0.f : sum / all;
    T* dst = out + (int64_t)(q0 + (int)fresh) * a.o_tok + (head * a.group + (int)h) * a.o_head + e % HD;
    if constexpr (P::kFp32)
      *dst = y;
    else if constexpr (P::kBf16)
      *dst = __float2bfloat16_rn(y);
    else
      *dst = __float2half_rn(y);
  };
  float* cta = part + WARPS * G::kWarpPart;  // O [row][HD], then the offsets, then l
#pragma unroll 1
  for (int e = threadIdx.x; e < kRows * HD; e += WARPS * 32) {
    const int rw = e / HD;
    float top = -INFINITY, sum = 0.f, all = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, part[w * G::kWarpPart + kRows * HD + rw]);
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float* p = part + w * G::kWarpPart;
      const float mw = p[kRows * HD + rw];
      const float f = mw == top ? 1.f : ex2(mw - top);  // no key yet anywhere: sums of zeros
      sum = fmaf(f, p[e] + p[kRows * HD + 2 * kRows + rw], sum);
      all = fmaf(f, p[kRows * HD + kRows + rw], all);
    }
    if (a.split == 1) {
      store(e, sum, all);
      continue;
    }
    cta[e] = sum;
    if (e % HD == 0) {
      cta[kRows * HD + rw] = top;
      cta[kRows * HD + kRows + rw] = all;
    }
  }
  if (a.split == 1) return;
  cluster_barrier();
#pragma unroll 1
  for (int e = rank * WARPS * 32 + threadIdx.x; e < kRows * HD; e += a.split * WARPS * 32) {
    const int rw = e / HD;
    float top = -INFINITY, sum = 0.f, all = 0.f;
#pragma unroll 4
    for (int r = 0; r < a.split; ++r)
      top = fmaxf(top, __uint_as_float(cluster_load32(cluster_address(cta + kRows * HD + rw, r))));
#pragma unroll 4
    for (int r = 0; r < a.split; ++r) {
      const float mr = __uint_as_float(cluster_load32(cluster_address(cta + kRows * HD + rw, r)));
      const float lr = __uint_as_float(cluster_load32(cluster_address(cta + kRows * HD + kRows + rw, r)));
      const float po = __uint_as_float(cluster_load32(cluster_address(cta + e, r)));
      const float f = mr == top ? 1.f : ex2(mr - top);
      sum = fmaf(f, po, sum);
      all = fmaf(f, lr, all);
    }
    store(e, sum, all);
  }
  cluster_barrier();  // no CTA leaves while another reads its part
}

// Per device, once: the kernel's shared-memory limit and cluster size.
template <typename T, int HD, int WARPS>
cudaError_t prepare() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
  const void* fn = reinterpret_cast<const void*>(&kv4_attention_kernel<T, HD, WARPS>);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<HD, WARPS>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

template <typename T, int HD, int WARPS>
cudaError_t launch(const Kv4Dev& d, const Kv4Tensor& q, const Kv4Tensor& o, const AttnArgs& a, int64_t items,
                   cudaStream_t s) {
  cudaError_t e = prepare<T, HD, WARPS>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * a.split));
  cfg.blockDim = dim3(WARPS * 32);
  cfg.dynamicSmemBytes = Geo<HD, WARPS>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = a.split > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<T, HD, WARPS>, d, static_cast<const T*>(q.p),
                            static_cast<T*>(const_cast<void*>(o.p)), a);
}

// CTAs that share a row block's keys: enough to fill the GPU (148 SMs), no more
// than leave a warp two steps of 64 keys.
template <typename T, int HD>
cudaError_t choose(const Kv4Dev& d, const Kv4Tensor& q, const Kv4Tensor& o, AttnArgs a, int64_t items,
                   cudaStream_t s) {
  const int64_t steps = ((int64_t)d.max_blocks * d.page_tokens + kKeys - 1) / kKeys;
  auto split = [&](int64_t ctas, int warps) {
    int n = 1;
    while (n < kMaxSplit && items * n * 2 <= ctas && steps >= (int64_t)n * 2 * warps * 2) n *= 2;
    return n;
  };
  // 16 CTAs of 4 warps for each: would they leave more than half of the GPU idle?
  const bool wide = items * kMaxSplit * 2 < 148 * Geo<HD, 4>::kPerSm && steps >= kMaxSplit * 12 * 2;
  a.split = wide ? split(148, 12) : split(148 * Geo<HD, 4>::kPerSm, 4);
  return wide ? launch<T, HD, 12>(d, q, o, a, items, s) : launch<T, HD, 4>(d, q, o, a, items, s);
}

}  // namespace

int kv4_attention_launch(const Kv4Dev& d, int head_dim, int max_new, const Kv4Tensor& q, int n_heads, int dtype,
                         const float* rope, float scale, const Kv4Tensor& out, cudaStream_t s) {
  if (d.total == 0 || max_new == 0) return WPK_OK;
  AttnArgs a{};
  a.q_tok = q.token, a.q_head = q.head, a.o_tok = out.token, a.o_head = out.head;
  a.rope = rope;
  a.group = n_heads / d.n_kv;
  a.max_new = std::min(max_new, d.total);
  if (!d.indptr) a.max_new = std::min(a.max_new, d.each);
  a.scale_log2 = (scale == 0.f ? 1.0f / sqrtf((float)head_dim) : scale) * 1.4426950408889634f;
  // blocks of rows of the kernel that takes the call; row numbers fit 32 bits
  const int64_t rows = (int64_t)a.max_new * a.group;
  const char* too_many = "too many query rows for one call (a closer max_new asks for fewer)";
  if (rows > INT_MAX - kPrefillRows) return op_fail(WPK_ERR_SHAPE, too_many);
  const bool many = many_rows(d, rows);
  const int block = many ? kPrefillRows : kRows;
  const int64_t row_blocks = (rows + block - 1) / block, blocks = row_blocks * d.n_kv;
  if (blocks > INT_MAX / kMaxSplit / d.batch) return op_fail(WPK_ERR_SHAPE, too_many);
  const int64_t items = blocks * d.batch;
  a.row_blocks = (int)row_blocks;
  cudaError_t e;
  const bool wide = head_dim == 128;
  if (many)
    e = kv4_prefill_launch(d, head_dim, a.max_new, q, a.group, dtype, rope, a.scale_log2, out, s);
  else if (dtype == WPK_F32)
    e = wide ? choose<float, 128>(d, q, out, a, items, s) : choose<float, 64>(d, q, out, a, items, s);
  else if (dtype == WPK_BF16)
    e = wide ? choose<__nv_bfloat16, 128>(d, q, out, a, items, s) : choose<__nv_bfloat16, 64>(d, q, out, a, items, s);
  else
    e = wide ? choose<__half, 128>(d, q, out, a, items, s) : choose<__half, 64>(d, q, out, a, items, s);
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof msg, "wpk_kv4_attention: %s", cudaGetErrorString(e));
    cudaGetLastError();
    return op_fail(WPK_ERR_CUDA, msg);
  }
  return WPK_OK;
}

}  // namespace wpk
