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
// lose what the centred one keeps (1.2e-3 against 2e-4 at 131072 tokens, fp16).
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
#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "kv4.cuh"
#include "kv4_host.h"
#include "op_util.cuh"
#include "ptx.cuh"

namespace cg = cooperative_groups;

namespace wpk {
namespace {

constexpr int kRows = 8;    // query rows of a CTA (the N of the P V product)
constexpr int kKeys = 64;   // keys of a warp's step

template <int HD>
struct Geo {
  static constexpr int kWarps = 8;
  static constexpr int kStages = 3;
  static constexpr int kRowBytes = HD / 2;
  static constexpr int kStageBytes = kKeys * (2 * kRowBytes + 8);  // K codes, V codes, K (s, z), V (s, z)
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  // after the keys: every warp's rows (O, then m, l and the sum of p z), then the CTA's
  static constexpr int kWarpPart = kRows * (HD + 3);  // floats
  static constexpr int kCtaPart = kRows * (HD + 2);
  static constexpr int kJoin = (kWarps * kWarpPart + kCtaPart) * 4;
  static constexpr int kSmem = kRing > kJoin ? kRing : kJoin;
};

struct AttnArgs {
  int64_t q_tok, q_head, o_tok, o_head;
  const float* rope;
  int group, max_new, row_blocks, split;  // split: CTAs of a cluster
  float scale_log2;                       // scale * log2(e)
};

__device__ __forceinline__ void cp16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_f16(uint32_t u) {
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// d += a b: a 16 x 16 (fp16, rows), b 16 x 8 (fp16, columns), d fp32.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;

// The codes less 8 of two even nibbles, and of two odd ones times 16.
__device__ __forceinline__ uint32_t centred_even(uint32_t w) {
  const uint32_t u = (w & kEven) | 0x64006400u, eight = 0x64086408u;  // 1032
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&eight));
  return *reinterpret_cast<const uint32_t*>(&d);
}
__device__ __forceinline__ uint32_t centred_odd(uint32_t w) {
  const uint32_t u = (w & kOdd) | 0x64006400u, eight = 0x64806480u;  // 1024 + 16 * 8
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&eight));
  return *reinterpret_cast<const uint32_t*>(&d);
}

// In a warp, lane = 4 g + t.  S's columns 2t and 2t + 1 of the n-th group of 8
// keys are its keys t and 7 - t: with this order neither the K rows (8 at a
// time) nor the V words (4 rows x 8 words) of a step meet in a bank.
template <typename T, int HD>
__global__ void __launch_bounds__(Geo<HD>::kWarps * 32)
    kv4_attention_kernel(const Kv4Dev c, const T* __restrict__ q, T* __restrict__ out, const AttnArgs a) {
  using G = Geo<HD>;
  constexpr int WPL = HD / 32;          // words of a K row that a lane multiplies
  // P keeps 22 bits (two products) for fp32 and fp16 tensors.  For bf16 ones its
  // 11 bits are enough: they add 4e-4 to the output's own rounding of 1.7e-3
  // (relative, of random values), but would double fp16's 2e-4.
  constexpr bool kFull = !std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x % a.split;
  int item = blockIdx.x / a.split;
  const int rb = item % a.row_blocks;
  item /= a.row_blocks;
  const int head = item % c.n_kv, b = item / c.n_kv;
  if (b >= kv4_sequences(c)) return;  // as for every CTA of the cluster
  int q0, n_new;
  kv4_new(c, b, &q0, &n_new);
  const int64_t rows = (int64_t)min(n_new, a.max_new) * a.group;
  const int64_t r0 = (int64_t)rb * kRows;
  if (r0 >= rows) return;

  // the rows' positions and the keys [0, n_keys) that any of them sees
  const int pos0 = c.pos[b];
  const int64_t cap = (int64_t)c.max_blocks * c.page_tokens;
  const int64_t my_row = r0 + g;
  const int my_new = my_row < rows ? (int)(my_row / a.group) : 0;
  const int64_t my_pos = (int64_t)pos0 + my_new;
  const bool placed = my_row < rows && pos0 >= 0 && my_pos < c.rope_positions;
  const int last = placed ? (int)(my_pos < cap ? my_pos : cap - 1) : -1;  // the row's last key
  const int64_t lo_pos = pos0 + r0 / a.group, hi_pos = pos0 + (min(r0 + kRows, rows) - 1) / a.group;
  const int n_keys = pos0 < 0 ? 0 : (int)min(hi_pos + 1, cap);
  const int all_see = (int)min(lo_pos + 1, cap);  // keys below it are seen by every row that has a position

  // Q: lane (g, t) holds dims 4 WPL t .. + 4 WPL of both halves of row g,
  // scaled by a power of two that brings the row's largest value to 2^13..2^14
  uint32_t qa[2 * WPL][4];
  float logit_mul, logit_z;
  {
    float lo[4 * WPL], hi[4 * WPL];
#pragma unroll
    for (int i = 0; i < 4 * WPL; ++i) lo[i] = hi[i] = 0.f;
    if (placed) {
      const T* p = q + (int64_t)(q0 + my_new) * a.q_tok + (head * a.group + (int)(my_row % a.group)) * a.q_head +
                   4 * WPL * t;
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
      top = fmaxf(top, fmaxf(fabsf(lo[i]), fabsf(hi[i])));
      sum += lo[i] + hi[i];
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    const int up = top > 0.f && top < INFINITY ? min(13 - ilogbf(top), 120) : 0;
    const float mul = scalbnf(1.f, up);
    logit_mul = scalbnf(a.scale_log2, (kFull ? 0 : 24) - up);
    logit_z = a.scale_log2 * sum;
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
        qa[k][2 * odd + 1] = pack_f16(x - back.x, y - back.y);
      }
    }
  }

  uint8_t* ring = smem + warp * (G::kStages * G::kStageBytes);
  const int n_steps = (n_keys + kKeys - 1) / kKeys, stride = a.split * G::kWarps;
  const int32_t* table = c.table + (int64_t)b * c.max_blocks;
  const int codes = c.page_tokens * G::kRowBytes;

  // A step's keys come in four runs of 16, each inside one page.  Lane i < 4
  // looks run i up (a step ahead of the copies): its rows' place, or NULL.
  struct Run {
    const uint8_t* page;
    int row;
  };
  auto look_up = [&](int step) {
    Run r{nullptr, 0};
    const int64_t key = (int64_t)step * kKeys + 16 * lane;
    if (lane < 4 && step < n_steps && key < n_keys) {
      const int slot = (int)key / c.page_tokens;
      const int block = table[slot];
      r.row = (int)key - slot * c.page_tokens;
      if (block >= 0 && block < c.n_blocks) r.page = kv4_page(c, block, head);
    }
    return r;
  };
  auto issue = [&](const Run& mine, uint8_t* stage) {
    const unsigned long long base = reinterpret_cast<unsigned long long>(mine.page);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, base, i));
      const int row = __shfl_sync(0xFFFFFFFFu, mine.row, i);
      if (!page) continue;
      const uint8_t* src = page + row * G::kRowBytes + lane * 16;
      uint8_t* dst = stage + i * 16 * G::kRowBytes + lane * 16;
#pragma unroll
      for (int o = 0; o < 16 * G::kRowBytes; o += 512) {
        cp16(dst + o, src + o);
        cp16(dst + kKeys * G::kRowBytes + o, src + codes + o);
      }
    }
    // 16 lanes copy K's (s, z), 16 V's: four keys each
    const int j = lane & 15, of_v = lane >> 4;
    const uint8_t* page = reinterpret_cast<const uint8_t*>(__shfl_sync(0xFFFFFFFFu, base, j >> 2));
    const int row = __shfl_sync(0xFFFFFFFFu, mine.row, j >> 2);
    if (page)
      cp16(stage + 2 * kKeys * G::kRowBytes + lane * 16,
           page + 2 * codes + (of_v * c.page_tokens + row + 4 * (j & 3)) * 4);
  };

  float m = -INFINITY, l = 0.f, pz = 0.f;  // of row g (pz: of p y); l and pz of this lane's keys only
  float o[2 * WPL][4];                     // rows 2t, 2t + 1: dims 4g + .. of both halves (word g, word g + 8)
#pragma unroll
  for (int i = 0; i < 2 * WPL; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  // exponent field of the largest V scale so far: P s is kept times 2^14 over
  // that scale's power of two, so that it stays inside fp16 whatever the scales
  // (a scale below 2^-113 counts as 2^-113)
  uint32_t v_exp = 14;

  int step = rank * G::kWarps + warp;
  uint32_t held = 0;  // 4 bits a stage: runs that have a place
  Run next = look_up(step);
#pragma unroll
  for (int s = 0; s < G::kStages - 1; ++s) {
    held |= (__ballot_sync(0xFFFFFFFFu, next.page != nullptr) & 15u) << (4 * s);
    issue(next, ring + s * G::kStageBytes);
    cp_commit();
    next = look_up(step + (s + 1) * stride);
  }
  int cur = 0;
  for (; step < n_steps; step += stride) {
    cp_wait<G::kStages - 2>();
    __syncwarp();
    {  // every lane is done with the previous step's stage: refill it
      const int to = cur == 0 ? G::kStages - 1 : cur - 1;
      held = (held & ~(15u << (4 * to))) | ((__ballot_sync(0xFFFFFFFFu, next.page != nullptr) & 15u) << (4 * to));
      issue(next, ring + to * G::kStageBytes);
      cp_commit();
      next = look_up(step + G::kStages * stride);
    }
    const uint8_t* stage = ring + cur * G::kStageBytes;
    const uint32_t have = (held >> (4 * cur)) & 15u;
    cur = cur + 1 == G::kStages ? 0 : cur + 1;
    const int key0 = step * kKeys;

    // S
    float s[8][4];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
      const int key = 8 * n + (g & 1 ? 7 - (g >> 1) : g >> 1);
      uint32_t w[WPL];
      if (WPL == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(stage + key * G::kRowBytes + t * 8);
        w[0] = v.x, w[1] = v.y;
      } else {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + key * G::kRowBytes + t * 16);
        w[0] = v.x, w[1] = v.y, w[WPL - 2] = v.z, w[WPL - 1] = v.w;
      }
#pragma unroll
      for (int i = 0; i < WPL; ++i) {
        const uint32_t h = w[i] >> 8;
        const uint32_t k0 = kFull ? centred_even(w[i]) : w[i] & kEven, k1 = kFull ? centred_odd(w[i]) : w[i] & kOdd;
        const uint32_t k2 = kFull ? centred_even(h) : h & kEven, k3 = kFull ? centred_odd(h) : h & kOdd;
        mma16816(s[n], qa[2 * i][0], qa[2 * i][1], qa[2 * i][2], qa[2 * i][3], k0, k1);
        mma16816(s[n], qa[2 * i + 1][0], qa[2 * i + 1][1], qa[2 * i + 1][2], qa[2 * i + 1][3], k2, k3);
      }
    }
    const uint32_t* ksz = reinterpret_cast<const uint32_t*>(stage + 2 * kKeys * G::kRowBytes);
    const uint32_t* vsz = ksz + kKeys;
    float x[16];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t sz = ksz[8 * n + (e ? 7 - t : t)];
        const float ks = __uint_as_float(sz << 16);
        const float kz = fmaf(kFull ? 8.f : 0.f, ks, __uint_as_float(sz & 0xFFFF0000u));
        x[2 * n + e] = fmaf(ks, (s[n][e] + s[n][2 + e]) * logit_mul, kz * logit_z);
      }
    float vs[16], vz[16];
#pragma unroll
    for (int n = 0; n < 8; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t sz = vsz[8 * n + (e ? 7 - t : t)];
        vs[2 * n + e] = __uint_as_float(sz << 16);
        vz[2 * n + e] = fmaf(8.f, vs[2 * n + e], __uint_as_float(sz & 0xFFFF0000u));
      }
    if (have != 15u || key0 + kKeys > all_see) {
      // keys without a place, or behind a row's last one: their score is left
      // out, and whatever their rows hold (or the stage held) reads as zero
#pragma unroll
      for (int n = 0; n < 8; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int key = key0 + 8 * n + (e ? 7 - t : t);
          const bool there = (have >> (n >> 1)) & 1u;
          if (!there || key >= n_keys) vs[2 * n + e] = vz[2 * n + e] = 0.f;
          if (!there || key > last) {
            x[2 * n + e] = -INFINITY;
            vz[2 * n + e] = 0.f;
          }
        }
    }

    // softmax of row g over the step's keys, and the running normalisers
    float top = x[0];
    uint32_t s_top = __float_as_uint(vs[0]);
#pragma unroll
    for (int i = 1; i < 16; ++i) {
      top = fmaxf(top, x[i]);
      s_top = max(s_top, __float_as_uint(vs[i]));
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    const uint32_t e_new = max(v_exp, min(__reduce_max_sync(0xFFFFFFFFu, s_top) >> 23, 254u));
    const float m_new = fmaxf(m, top);
    const bool moved = m_new != m || e_new != v_exp;
    const float m_use = m_new == -INFINITY ? 0.f : m_new;
    if (__any_sync(0xFFFFFFFFu, moved)) {
      const float fade = ex2(m - m_use);
      l *= fade;
      pz *= fade;
      const float drop = scalbnf(1.f, max((int)v_exp - (int)e_new, -126));
      const float f0 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t) * drop;
      const float f1 = __shfl_sync(0xFFFFFFFFu, fade, 8 * t + 4) * drop;
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i) {
        o[i][0] *= f0, o[i][2] *= f0;
        o[i][1] *= f1, o[i][3] *= f1;
      }
      m = m_new;
      v_exp = e_new;
    }
    const float unit = __uint_as_float((268u - v_exp) << 23);  // 2^(14 - exponent)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float p = ex2(x[i] - m_use);
      l += p;
      pz = fmaf(p, vz[i], pz);
      x[i] = p * (vs[i] * unit);
    }

    // O^T += V^T P^T, 16 keys at a time.  The tensor pipe cuts off what its sums
    // cannot hold: where 22 bits are kept, a step's sum is its own and joins the
    // running one in a rounded addition.
    float step_o[2 * WPL][4];
    if (kFull) {
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i) step_o[i][0] = step_o[i][1] = step_o[i][2] = step_o[i][3] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t b0 = pack_f16(x[4 * k], x[4 * k + 1]), b1 = pack_f16(x[4 * k + 2], x[4 * k + 3]);
      uint32_t d0 = 0, d1 = 0;
      if (kFull) {
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
        const int first = g + 8 * (t >> 1), second = first ^ 8;
        uint32_t u[4] = {v0[first], v1[first], v2[first], v3[first]};
        uint32_t y[4] = {v0[second], v1[second], v2[second], v3[second]};
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
            float(&d)[4] = kFull ? step_o[4 * i + 2 * half + pair] : o[4 * i + 2 * half + pair];
            const uint32_t e0 = centred_even(a01), e1 = centred_odd(a01), e2 = centred_even(a23), e3 = centred_odd(a23);
            mma16816(d, e0, e1, e2, e3, b0, b1);
            if (kFull) mma16816(d, e0, e1, e2, e3, d0, d1);
            a01 >>= 8;
            a23 >>= 8;
          }
        }
      }
    }
    if (kFull) {
#pragma unroll
      for (int i = 0; i < 2 * WPL; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += step_o[i][e];
    }
  }
  cp_wait<0>();
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l += __shfl_xor_sync(0xFFFFFFFFu, l, d);
    pz += __shfl_xor_sync(0xFFFFFFFFu, pz, d);
  }

  // join the warps, then the cluster's CTAs
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
  {
    float* mine = part + warp * G::kWarpPart;
    const float even = scalbnf(1.f, (int)v_exp - 127 - 14);  // one over the power of two that P s carries
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
      mine[kRows * HD + g] = m;
      mine[kRows * HD + kRows + g] = l;
      mine[kRows * HD + 2 * kRows + g] = pz;
    }
  }
  __syncthreads();
  float* cta = part + G::kWarps * G::kWarpPart;  // O [row][HD], then m, then l
  for (int e = threadIdx.x; e < kRows * HD; e += G::kWarps * 32) {
    const int row = e / HD;
    float top = -INFINITY, sum = 0.f, all = 0.f;
#pragma unroll
    for (int w = 0; w < G::kWarps; ++w) top = fmaxf(top, part[w * G::kWarpPart + kRows * HD + row]);
#pragma unroll
    for (int w = 0; w < G::kWarps; ++w) {
      const float* p = part + w * G::kWarpPart;
      const float mw = p[kRows * HD + row];
      const float f = mw == top ? 1.f : ex2(mw - top);  // no key yet anywhere: sums of zeros
      sum = fmaf(f, p[e] + p[kRows * HD + 2 * kRows + row], sum);
      all = fmaf(f, p[kRows * HD + kRows + row], all);
    }
    cta[e] = sum;
    if (e % HD == 0) {
      cta[kRows * HD + row] = top;
      cta[kRows * HD + kRows + row] = all;
    }
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster_barrier();
  for (int e = rank * G::kWarps * 32 + threadIdx.x; e < kRows * HD; e += a.split * G::kWarps * 32) {
    const int row = e / HD;
    float top = -INFINITY, sum = 0.f, all = 0.f;
    for (int r = 0; r < a.split; ++r) top = fmaxf(top, cluster.map_shared_rank(cta, r)[kRows * HD + row]);
    for (int r = 0; r < a.split; ++r) {
      const float* p = cluster.map_shared_rank(cta, r);
      const float mr = p[kRows * HD + row];
      const float f = mr == top ? 1.f : ex2(mr - top);
      sum = fmaf(f, p[e], sum);
      all = fmaf(f, p[kRows * HD + kRows + row], all);
    }
    if (r0 + row < rows) {
      const int64_t fresh = (r0 + row) / a.group;
      // a row that saw no key, or has no rotation, answers zeros
      const float y = all == 0.f || pos0 + fresh >= c.rope_positions ? 0.f : sum / all;
      T* dst = out + (q0 + fresh) * a.o_tok + (head * a.group + (int)((r0 + row) % a.group)) * a.o_head + e % HD;
      if constexpr (sizeof(T) == 4)
        *dst = y;
      else if constexpr (std::is_same<T, __half>::value)
        *dst = __float2half_rn(y);
      else
        *dst = __float2bfloat16_rn(y);
    }
  }
  cluster_barrier();  // no CTA leaves while another reads its part
}

// Per device, once: the kernel's shared-memory limit and cluster size.
template <typename T, int HD>
cudaError_t prepare() {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load(std::memory_order_acquire) >> dev & 1))) return e;
  const void* fn = reinterpret_cast<const void*>(&kv4_attention_kernel<T, HD>);
  e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, Geo<HD>::kSmem);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

template <typename T, int HD>
cudaError_t launch(const Kv4Dev& d, const Kv4Tensor& q, const Kv4Tensor& o, AttnArgs a, int64_t items,
                   cudaStream_t s) {
  cudaError_t e = prepare<T, HD>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(items * a.split));
  cfg.blockDim = dim3(Geo<HD>::kWarps * 32);
  cfg.dynamicSmemBytes = Geo<HD>::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.split;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kv4_attention_kernel<T, HD>, d, static_cast<const T*>(q.p),
                            static_cast<T*>(const_cast<void*>(o.p)), a);
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
  const int64_t row_blocks = ((int64_t)a.max_new * a.group + kRows - 1) / kRows;
  const int64_t items = row_blocks * d.n_kv * d.batch;
  if (items > INT_MAX / 16) return op_fail(WPK_ERR_SHAPE, "too many query rows for one call");
  a.row_blocks = (int)row_blocks;
  // CTAs that share a row block's keys: enough to fill the SMs (two CTAs each
  // at head_dim 64), and no more than have a step of 64 keys per warp
  const int64_t longest = ((int64_t)d.max_blocks * d.page_tokens + kKeys - 1) / kKeys;
  a.split = 1;
  while (a.split < 16 && items * a.split < 148 && longest > (int64_t)a.split * 8) a.split *= 2;
  cudaError_t e;
  const bool wide = head_dim == 128;
  if (dtype == WPK_F32)
    e = wide ? launch<float, 128>(d, q, out, a, items, s) : launch<float, 64>(d, q, out, a, items, s);
  else if (dtype == WPK_BF16)
    e = wide ? launch<__nv_bfloat16, 128>(d, q, out, a, items, s) : launch<__nv_bfloat16, 64>(d, q, out, a, items, s);
  else
    e = wide ? launch<__half, 128>(d, q, out, a, items, s) : launch<__half, 64>(d, q, out, a, items, s);
  if (e != cudaSuccess) {
    char msg[160];
    snprintf(msg, sizeof msg, "wpk_kv4_attention: %s", cudaGetErrorString(e));
    cudaGetLastError();
    return op_fail(WPK_ERR_CUDA, msg);
  }
  return WPK_OK;
}

}  // namespace wpk
