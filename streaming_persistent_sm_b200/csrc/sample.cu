// wpk_sample: the next token of each row of logits, by temperature, top-k,
// top-p and min-p, with given uniform numbers.
//
// A cluster of CTAs takes a row.  Each CTA reads its slice of the row once into
// shared memory and all further passes run there: one read of the logits is what
// the operator has to move.  What a row keeps is "the tokens up to this (logit,
// id)", and nearly always these are few.  So the tokens that can be kept are
// bounded by a distance from the largest logit - for top-k by the distance of
// the k-th best of the maxima of four tokens each, for top-p by where the masses
// summed up in buckets, rounded down, reach its share, for min-p by its logarithm
// - and sent to the first
// CTA, which sorts them and finishes the row alone (one warp of it where they are at
// most 128).
//
// A row whose bound holds more than kList tokens (a flat one) goes the longer
// way: the tokens fall into 2048 buckets by their distance, the counts (or
// masses) of the buckets, summed over the cluster, say in which one the border
// lies, and that one's tokens are sorted - after cutting its range of logits
// into 2048 again where it holds too many.
//
// A token's weight exp((z - zmax) / T) is computed in 64 bits and held as a
// whole multiple of 2^-45, so that sums do not depend on their order (shared
// atomics, clusters of any size) and decisions at a border are those of the
// definition.  B200 runs 64-bit arithmetic at half the 32-bit rate, and a weight
// takes some 20 operations; the bulk of a row, of weights below 2^-14, is
// computed in 32 bits with the exponent's rounding errors carried along: 2^-22
// of such a weight, 2^-36 of the largest.
#include <limits.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "op_util.cuh"

namespace wpk {
namespace {

constexpr int kSampThreads = 512;
constexpr int kSampWarps = kSampThreads / 32;
constexpr int kBins = 2048;
constexpr int kList = 2048;         // tokens that the first CTA sorts
constexpr int kRange = 64;          // top-k's first buckets reach 64 below the largest logit
constexpr int kMaxVocab = 1 << 18;  // 2^18 weights of at most 2^45 fit 63 bits
constexpr int kMaxCluster = 8;
constexpr int kTwoPerSm = 22016;  // tokens of a slice of which two fit an SM (113 KB each)
constexpr double kOne = 35184372088832.0;  // 2^45: a weight of 1
constexpr uint64_t kAll = ~0ull;           // a place behind every token

struct SampleArgs {
  const void* logits;
  int64_t stride;
  int vocab, slice, cluster;
  const float *uniform, *temperature, *top_p, *min_p;
  const int32_t* top_k;
  int32_t* tok;
  float* logprob;
  int32_t* kept;
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }

// Order of floats (no NaN, -0 as +0) as unsigned numbers, and back.
__device__ __forceinline__ uint32_t rank_bits(float z) {
  const uint32_t u = __float_as_uint(z);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_rank(uint32_t r) {
  return __uint_as_float((r & 0x80000000u) ? (r & 0x7FFFFFFFu) : ~r);
}
// The bucket at x (0 where x is none: the largest logit times an infinite 1 / T).
__device__ __forceinline__ int bucket(float x) { return x > 0.f ? (int)fminf(x, (float)(kBins - 1)) : 0; }
// A token's place in the ranking: smaller is better, equal logits by id.
__device__ __forceinline__ uint64_t place(float z, uint32_t id) { return ((uint64_t)(~rank_bits(z)) << 32) | id; }

// exp(t) for t <= 0, to a few units of 2^-53: t = n ln 2 + r, exp(r) as the
// fourth power of its Taylor sum at r / 4 (|r / 4| < 0.087: the first term left
// out, of degree 10, is below 2^-56).  Zero below -110, which is under every fp32 number.
__device__ __forceinline__ double exp_neg(double t) {
  if (!(t > -110.0)) return 0.0;
  const double shift = 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are the whole number
  const double s = t * 1.4426950408889634 + shift;
  const int n = __double2loint(s);
  const double k = s - shift;
  double r = fma(k, -0.69314718055994529, t);
  r = fma(k, -2.3190468138462996e-17, r);  // ln 2 less its double
  r *= 0.25;
  double p = 1.0 / 362880.0;
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  p *= p;
  p *= p;
  return __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
}

// 2^-kTail: weights below it are computed in 32 bits.
constexpr float kTail = 14.f;

struct Weigh {  // weights of a row's tokens
  float zmax, log2_t, log2_t_rest;  // log2(e) / T and what its float leaves
  double inv_t;
  __device__ __forceinline__ double weight(float z) const {
    return z > -INFINITY ? exp_neg(((double)z - (double)zmax) * inv_t) : 0.0;
  }
  // log2 of the weight, to 2^-20 or so: enough to choose a way
  __device__ __forceinline__ float log2_weight(float z) const { return (z - zmax) * log2_t; }
  __device__ __forceinline__ uint64_t heavy_mass(float z) const { return __double2ull_rn(weight(z) * kOne); }
  // The mass of a token of log2_weight t < -kTail.  The exponent is carried with
  // its rounding errors (of the distance and of the product) and split into a
  // whole number and a rest below 1/2, so the error is ex2's, 2^-22.
  __device__ __forceinline__ uint32_t tail_mass(float z, float t) const {
    if (!(t > -48.f)) return 0;
    const float d = z - zmax, back = d + zmax;
    const float lost = (z - back) + (zmax - (back - d));  // z - zmax - d
    const float n = rintf(t);
    const float rest = (t - n) + fmaf(d, log2_t, -t) + fmaf(d, log2_t_rest, lost * log2_t);
    float m;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(m) : "f"(rest));
    return __float2uint_rn(m * __int_as_float((int)n + (45 + 127) << 23));
  }
  __device__ __forceinline__ uint64_t mass(float z) const {
    const float t = log2_weight(z);
    return t < -kTail ? tail_mass(z, t) : z > -INFINITY ? heavy_mass(z) : 0;
  }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}
__device__ __forceinline__ uint64_t warp_min64(uint64_t v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = min(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ uint64_t warp_scan64(uint64_t v) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// Shared memory of a CTA, the slice's logits behind it.
constexpr int kLocal = kBins / 2;  // candidates that a CTA other than the first can send
struct SampleShared {
  union {
    uint64_t mass[kBins];
    uint64_t list[kList];  // the bins' masses are read before the list is filled
  };
  union {
    uint32_t count[kBins];
    uint64_t local[kLocal];  // the bins are read before the candidates are collected
  };
  uint64_t warp_a[kSampWarps], warp_b[kSampWarps];
  uint64_t word[2][4];  // what this CTA tells the others, in turn
  uint32_t part[3][kSampWarps];
  uint32_t list_n, local_n, local_at;
  int found;
};
static_assert(sizeof(SampleShared) % 16 == 0, "the slice behind it is aligned");

// Sums (or minima) of two values over the CTA, in every thread; warp_a keeps
// the warps' sums of the first.
template <bool kMin>
__device__ __forceinline__ void block_join(SampleShared& S, uint64_t* a, uint64_t* b) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t wa = kMin ? warp_min64(*a) : warp_sum64(*a), wb = kMin ? warp_min64(*b) : warp_sum64(*b);
  __syncthreads();
  if (lane == 0) {
    S.warp_a[warp] = wa;
    S.warp_b[warp] = wb;
  }
  __syncthreads();
  const uint64_t none = kMin ? kAll : 0, ja = lane < kSampWarps ? S.warp_a[lane] : none,
                 jb = lane < kSampWarps ? S.warp_b[lane] : none;
  *a = kMin ? warp_min64(ja) : warp_sum64(ja);
  *b = kMin ? warp_min64(jb) : warp_sum64(jb);
}

// Publishes this CTA's words (thread 0's) and meets the others; word(turn, i, r)
// then reads rank r's, until the next meeting but one.
__device__ __forceinline__ void meet(SampleShared& S, int& turn, uint64_t a, uint64_t b) {
  turn ^= 1;
  if (threadIdx.x == 0) {
    S.word[turn][0] = a;
    S.word[turn][1] = b;
  }
  cluster_barrier();
}
__device__ __forceinline__ uint64_t word(const SampleShared& S, int turn, int i, int rank) {
  return cluster_load64(cluster_address(&S.word[turn][i], rank));
}
// Lane r holds rank r's word (other lanes: `none`): one trip for all ranks.
__device__ __forceinline__ uint64_t words(const SampleShared& S, int turn, int i, int cluster, uint64_t none) {
  const int lane = threadIdx.x & 31;
  return lane < cluster ? word(S, turn, i, lane) : none;
}

// Adds a token to bin b (b < 0: none), called by whole warps.  One addition for
// the warp where all its tokens fall into one bin, as in rows of equal logits.
__device__ __forceinline__ void add_to_bin(SampleShared& S, int b, bool by_mass, uint64_t u) {
  const uint32_t in = __ballot_sync(0xFFFFFFFFu, b >= 0);
  if (in == 0) return;
  const int lead = __ffs(in) - 1;
  const int b0 = __shfl_sync(0xFFFFFFFFu, b, lead);
  const bool same = __all_sync(0xFFFFFFFFu, b < 0 || b == b0);
  if (same && __popc(in) > 4) {
    if (by_mass) u = warp_sum64(b >= 0 ? u : 0);
    if ((threadIdx.x & 31) == lead) {
      atomicAdd(&S.count[b0], (uint32_t)__popc(in));
      if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&S.mass[b0]), (unsigned long long)u);
    }
  } else if (b >= 0) {
    atomicAdd(&S.count[b], 1u);
    if (by_mass) atomicAdd(reinterpret_cast<unsigned long long*>(&S.mass[b]), (unsigned long long)u);
  }
}

// Exclusive sum of v over the threads before this one (v of whole CTAs).
__device__ __forceinline__ uint64_t block_before(SampleShared& S, uint64_t v) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t upto = warp_scan64(v);
  __syncthreads();
  if (lane == 31) S.warp_a[warp] = upto;
  __syncthreads();
  return upto - v + warp_sum64(lane < warp ? S.warp_a[lane] : 0);
}

// The same over one warp, or over the CTA.
template <bool kBlock>
__device__ __forceinline__ uint64_t sum_before(SampleShared& S, uint64_t v) {
  return kBlock ? block_before(S, v) : warp_scan64(v) - v;
}
template <bool kBlock>
__device__ __forceinline__ uint64_t sum_all(SampleShared& S, uint64_t v) {
  if (!kBlock) return warp_sum64(v);
  uint64_t same = 0;
  block_join<false>(S, &v, &same);
  return v;
}

constexpr int kEach = kList / kSampThreads;  // entries of the list that a thread holds
static_assert(kEach == 4, "sort_each holds four");

// Sorts `size` entries (a power of two, 128 or more), four in each of the first
// size / 4 threads, ascending, as a bitonic network: partners are in the thread,
// in the warp (shuffles), or, above 128 entries, in another warp (through the
// list).  Called by whole CTAs where size > 128.
__device__ __forceinline__ void sort_each(SampleShared& S, uint64_t (&v)[kEach], int size) {
  const int i0 = kEach * threadIdx.x;
#pragma unroll 1
  for (int s = 2; s <= size; s *= 2)
#pragma unroll 1
    for (int j = s / 2; j > 0; j /= 2) {
      if (j >= 32 * kEach) {
        __syncthreads();
        if (i0 < size) {
#pragma unroll
          for (int e = 0; e < kEach; ++e) S.list[i0 + e] = v[e];
        }
        __syncthreads();
        if (i0 < size) {
          const bool low = ((i0 & j) == 0) == ((i0 & s) == 0);
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            const uint64_t other = S.list[(i0 ^ j) + e];
            v[e] = low ? min(v[e], other) : max(v[e], other);
          }
        }
      } else if (j >= kEach) {
        const bool low = ((i0 & j) == 0) == ((i0 & s) == 0);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, v[e], j / kEach);
          v[e] = low ? min(v[e], other) : max(v[e], other);
        }
      } else {
        auto order = [&](int x, int y) {  // entries x < y of the thread
          const bool up = ((i0 + x) & s) == 0;
          const uint64_t a = min(v[x], v[y]), c = max(v[x], v[y]);
          v[x] = up ? a : c;
          v[y] = up ? c : a;
        };
        if (j == 2) {
          order(0, 2);
          order(1, 3);
        } else {
          order(0, 1);
          order(2, 3);
        }
      }
    }
}
__device__ __forceinline__ int sort_size(int n) {
  int size = 32 * kEach;
  while (size < n) size *= 2;
  return size;
}

struct Filters {
  int k;           // top-k's number, where it is on
  float p;         // top-p's share
  bool by_k, by_p;
  double floor_w;  // min-p, 0: off
  double u;
};

// The rest of a row on the first CTA, from its m candidates: a beginning of the
// ranking that holds all that can be kept.  all_mass: that of the whole row, for
// top-p without top-k.
template <bool kBlock>
__device__ __forceinline__ void finish(SampleShared& S, const SampleArgs& A, int b, const Weigh& W, const Filters& f,
                                       int m, uint64_t all_mass) {
  const int i0 = kEach * threadIdx.x;
  uint64_t v[kEach], w[kEach], sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) v[e] = i0 + e < m ? S.list[i0 + e] : kAll;
  sort_each(S, v, sort_size(m));
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    w[e] = i0 + e < m ? W.mass(from_rank(~(uint32_t)(v[e] >> 32))) : 0;
    sum += w[e];
  }
  // how many are kept: top-k's number, top-p's beginning of it, min-p's
  int keep = f.by_k ? min(m, f.k) : m;
  if (f.by_p) {
    if (f.by_k) {
      uint64_t in = 0;
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (i0 + e < keep) in += w[e];
      all_mass = sum_all<kBlock>(S, in);
    }
    const double want = ceil((double)f.p * (double)all_mass);
    const uint64_t target = want > 1.0 ? (uint64_t)want : (uint64_t)1;
    uint64_t left = sum_before<kBlock>(S, sum), short_of = 0;  // beginnings that fall short
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      left += w[e];
      short_of += i0 + e < keep && left < target;
    }
    keep = min(keep, (int)sum_all<kBlock>(S, short_of) + 1);
  }
  if (f.floor_w > 0.0) {
    uint64_t heavy = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      heavy += i0 + e < keep && W.weight(from_rank(~(uint32_t)(v[e] >> 32))) >= f.floor_w;
    keep = (int)sum_all<kBlock>(S, heavy);
  }
  // the kept ones in the order of ids, and the draw
  uint64_t in = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const bool on = i0 + e < keep;
    if (on) in += w[e];
    v[e] = on ? v[e] << 32 | v[e] >> 32 : kAll;
  }
  const uint64_t mass = sum_all<kBlock>(S, in);
  const uint64_t want = min((uint64_t)(f.u * (double)mass), mass - 1);
  sort_each(S, v, sort_size(keep));
  sum = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    w[e] = i0 + e < keep ? W.mass(from_rank(~(uint32_t)v[e])) : 0;
    sum += w[e];
  }
  uint64_t left = sum_before<kBlock>(S, sum);
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    if (left <= want && want < left + w[e]) {  // in one thread
      const double t = ((double)from_rank(~(uint32_t)v[e]) - (double)W.zmax) * W.inv_t;
      A.tok[b] = (int)(v[e] >> 32);
      if (A.logprob) A.logprob[b] = (float)(t - log((double)mass / kOne));
      if (A.kept) A.kept[b] = keep;
    }
    left += w[e];
  }
}

template <typename T>
__global__ void __launch_bounds__(kSampThreads, 2) wpk_sample_kernel(const SampleArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  SampleShared& S = *reinterpret_cast<SampleShared*>(smem);
  float* z = reinterpret_cast<float*>(smem + sizeof(SampleShared));
  const int cluster = A.cluster, rank = blockIdx.x % cluster, b = blockIdx.x / cluster;
  const int base = min(A.vocab, rank * A.slice), n = min(A.vocab - base, A.slice);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;

  // read the slice, padded with masked tokens to whole vectors of all lanes
  const int padded = (n + 127) & ~127;
  float top = -INFINITY;
  uint32_t finite = 0, bad = 0;
  {
    const T* src = static_cast<const T*>(A.logits) + b * A.stride + base;
    uint32_t count = 0, wrong = 0;
    auto take = [&](float x) {
      const float y = x + 0.f;  // -0 becomes +0
      top = fmaxf(top, y);
      wrong |= !(y < INFINITY);
      count += y > -INFINITY;
      return y;
    };
    if (reinterpret_cast<uintptr_t>(src) % (4 * sizeof(T)) == 0) {
#pragma unroll 4
      for (int i = 4 * threadIdx.x; i < (n & ~3); i += 4 * kSampThreads) {
        float x[4];
        load4(src + i, x);
        *reinterpret_cast<float4*>(z + i) = make_float4(take(x[0]), take(x[1]), take(x[2]), take(x[3]));
      }
      const int i = (n & ~3) + threadIdx.x;
      if (i < n) z[i] = take(to_float(src[i]));
    } else {
#pragma unroll 8
      for (int i = threadIdx.x; i < n; i += kSampThreads) z[i] = take(to_float(src[i]));
    }
    if (n + threadIdx.x < padded) z[n + threadIdx.x] = -INFINITY;
    finite = count;
    bad = wrong;
  }
  // the row's largest logit, its tokens that are not masked, whether any is NaN or +inf
  {
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, rank_bits(top)), c = __reduce_add_sync(0xFFFFFFFFu, finite),
                   w = __reduce_or_sync(0xFFFFFFFFu, bad);
    if (lane == 0) {
      S.part[0][warp] = m;
      S.part[1][warp] = c;
      S.part[2][warp] = w;
    }
    for (int i = threadIdx.x; i < kBins; i += kSampThreads) S.count[i] = 0;
    if (threadIdx.x == 0) S.list_n = S.local_n = 0;
    __syncthreads();
    const bool on = lane < kSampWarps;
    const uint32_t tm = __reduce_max_sync(0xFFFFFFFFu, on ? S.part[0][lane] : 0u),
                   tc = __reduce_add_sync(0xFFFFFFFFu, on ? S.part[1][lane] : 0u),
                   tw = __reduce_or_sync(0xFFFFFFFFu, on ? S.part[2][lane] : 0u);
    meet(S, turn, (uint64_t)tm << 32 | tc, tw);
    const uint64_t a = words(S, turn, 0, cluster, 0);
    finite = __reduce_add_sync(0xFFFFFFFFu, (uint32_t)a);
    top = from_rank(__reduce_max_sync(0xFFFFFFFFu, (uint32_t)(a >> 32)));
    bad = __reduce_or_sync(0xFFFFFFFFu, (uint32_t)words(S, turn, 1, cluster, 0));
  }
  Weigh W;
  W.zmax = top;
  // a warp's tokens, in the order of ids: whole vectors of all lanes
  const int per = ((padded + kSampWarps - 1) / kSampWarps + 127) & ~127;
  const int seg_lo = min(padded, warp * per), seg_hi = min(padded, seg_lo + per);
  const float temperature = A.temperature ? A.temperature[b] : 1.f;
  const bool none = bad != 0 || finite == 0;
  if (none || !(temperature > 0.f)) {  // as for every CTA of the cluster
    // the lowest id of the largest logit
    uint64_t id = kAll, same;
    for (int i = seg_lo + 4 * lane; i < seg_hi && !none; i += 128) {
      const float4 x = *reinterpret_cast<const float4*>(z + i);
      if (x.w == top) id = min(id, (uint64_t)(base + i + 3));
      if (x.z == top) id = min(id, (uint64_t)(base + i + 2));
      if (x.y == top) id = min(id, (uint64_t)(base + i + 1));
      if (x.x == top) id = min(id, (uint64_t)(base + i));
    }
    same = id;
    block_join<true>(S, &id, &same);
    meet(S, turn, id, 0);
    id = warp_min64(words(S, turn, 0, cluster, kAll));
    if (rank == 0 && threadIdx.x == 0) {
      A.tok[b] = none ? -1 : (int)id;
      if (A.logprob) A.logprob[b] = none ? NAN : 0.f;
      if (A.kept) A.kept[b] = none ? 0 : 1;
    }
    cluster_barrier();  // no CTA leaves while another may read its words
    return;
  }
  W.inv_t = 1.0 / (double)temperature;
  const double log2_t = 1.4426950408889634 * W.inv_t;
  W.log2_t = (float)log2_t;
  W.log2_t_rest = isfinite(W.log2_t) ? (float)(log2_t - (double)W.log2_t) : 0.f;
  Filters f;
  f.k = A.top_k ? A.top_k[b] : 0;
  f.p = A.top_p ? A.top_p[b] : 1.f;
  const float mp = A.min_p ? A.min_p[b] : 0.f;
  f.floor_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
  const float u_part = A.uniform[b];
  f.u = u_part > 0.f ? fmin((double)u_part, 1.0) : 0.0;
  f.by_k = f.k > 0 && (uint32_t)f.k < finite;
  f.by_p = f.p < 1.f;
  const bool by_k = f.by_k, by_p = f.by_p;
  const float p = f.p;
  const int k = f.k;
  const double floor_w = f.floor_w;
  const bool filtered = by_k || by_p || floor_w > 0.0;

  // The mass of all tokens: what a row without filters draws from, and top-p
  // alone is measured by.  For the latter, heavy tokens' weights in units of
  // 2^-13, rounded down, are summed up in buckets of their log2.
  constexpr float kSteps = kBins / kTail;
  uint64_t all_mass = 0;
  if (!filtered || (by_p && !by_k)) {
    uint64_t v = 0;
#pragma unroll 1
    for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
      const float4 x4 = *reinterpret_cast<const float4*>(z + i);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
      const float t_top = W.log2_weight(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])));
      if (t_top < -kTail) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v += W.tail_mass(x[e], W.log2_weight(x[e]));
      } else {
#pragma unroll 1
        for (int e = 0; e < 4; ++e) {
          const float xe = e == 0 ? x[0] : e == 1 ? x[1] : e == 2 ? x[2] : x[3];
          const uint64_t u = W.mass(xe);
          v += u;
          const float t = W.log2_weight(xe);
          if (filtered && !(t < -kTail) && xe > -INFINITY)
            atomicAdd(&S.count[bucket(-t * kSteps)], (uint32_t)(u >> 32));
        }
      }
    }
    v = warp_sum64(v);
    if (lane == 0) S.warp_a[warp] = v;
    __syncthreads();
    const uint64_t mine = warp_sum64(lane < kSampWarps ? S.warp_a[lane] : 0);
    meet(S, turn, mine, 0);
    const uint64_t a = words(S, turn, 0, cluster, 0);
    all_mass = warp_sum64(a);
    if (!filtered) {
      // the token at which the mass in the order of ids is first above its part
      const uint64_t want = min((uint64_t)(f.u * (double)all_mass), all_mass - 1);
      const uint64_t before = warp_sum64(lane < rank ? a : 0);
      if (want >= before && want - before < mine) {  // one CTA of the cluster,
        uint64_t rest = want - before;
        const uint64_t lower = warp_sum64(lane < warp ? S.warp_a[lane] : 0);
        if (rest >= lower && rest - lower < S.warp_a[warp]) {  // and one warp of it
          rest -= lower;
#pragma unroll 1
          for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
            uint64_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) u[e] = W.mass(z[i + e]);
            const uint64_t four = u[0] + u[1] + u[2] + u[3], upto = warp_scan64(four);
            if (__any_sync(0xFFFFFFFFu, upto > rest)) {
              uint64_t left = upto - four;
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if (left <= rest && rest < left + u[e]) {  // in one lane
                  const double t = ((double)z[i + e] - (double)W.zmax) * W.inv_t;
                  A.tok[b] = base + i + e;
                  if (A.logprob) A.logprob[b] = (float)(t - log((double)all_mass / kOne));
                  if (A.kept) A.kept[b] = (int)finite;
                }
                left += u[e];
              }
              break;
            }
            rest -= __shfl_sync(0xFFFFFFFFu, upto, 31);
          }
        }
      }
      cluster_barrier();  // no CTA leaves while another may read its words
      return;
    }
  }

  {
    // the candidates: tokens no further than `reach` from the largest logit
    float reach = INFINITY;
    if (by_k || by_p) {
      if (by_k) {
        // the k-th best of the maxima of four tokens each: at least k tokens are
        // no further.  Bucketed, so a bit further.
#pragma unroll 2
        for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
          const float4 x = *reinterpret_cast<const float4*>(z + i);
          const float d = (W.zmax - fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w))) * ((float)kBins / kRange);
          if (d < (float)kBins) atomicAdd(&S.count[(int)d], 1u);
        }
        cluster_barrier();
      }
      // rank 0 sums the CTAs' buckets and finds the one that reaches the target
      turn ^= 1;
      if (rank == 0) {
        const double want = ceil((double)p * (double)all_mass / 4294967296.0);
        const uint64_t target = by_k ? (uint64_t)k : want > 1.0 ? (uint64_t)want : 1;
        uint32_t c[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) c[e] = 0;
        for (int r = 0; r < cluster; ++r) {
          const uint32_t rc = cluster_address(&S.count[threadIdx.x * kEach], r);
#pragma unroll
          for (int e = 0; e < kEach; ++e) c[e] += cluster_load32(rc + 4 * e);
        }
        if (threadIdx.x == 0) S.word[turn][0] = kBins;  // not reached
        uint64_t left = block_before(S, (uint64_t)c[0] + c[1] + c[2] + c[3]);
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (left < target && target <= left + c[e]) S.word[turn][0] = threadIdx.x * kEach + e;
          left += c[e];
        }
      }
      cluster_barrier();
      const int bin = (int)word(S, turn, 0, 0);
      // the bucket's far edge, and what the bucketing rounds
      if (bin < kBins)
        reach = by_k ? (bin + 1) * ((float)kRange / kBins) * 1.00001f
                     : ((bin + 1) * (1.f / kSteps) * 1.00001f) / W.log2_t;
    }
    // (with top-k, only its tokens may be dropped by min-p afterwards)
    if (floor_w > 0.0 && !by_k) reach = fminf(reach, temperature * (0.01f - logf((float)floor_w)));
    // the first CTA's go straight into its list, another's together
#pragma unroll 2
    for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
      const float4 v = *reinterpret_cast<const float4*>(z + i);
      const float x[4] = {v.x, v.y, v.z, v.w};
      if (!(W.zmax - fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) <= reach)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (x[e] > -INFINITY && W.zmax - x[e] <= reach) {
          if (rank == 0) {
            const uint32_t at = atomicAdd(&S.list_n, 1u);
            if (at < kList) S.list[at] = place(x[e], base + i + e);
          } else {
            const uint32_t at = atomicAdd(&S.local_n, 1u);
            if (at < kLocal) S.local[at] = place(x[e], base + i + e);
          }
        }
    }
    if (rank != 0) {
      __syncthreads();
      const uint32_t n_local = S.local_n;
      if (n_local) {  // more than can be sent: as many as the list does not hold
        if (threadIdx.x == 0)
          S.local_at = cluster_add32(cluster_address(&S.list_n, 0), n_local <= kLocal ? n_local : kList + 1);
        __syncthreads();
        const uint32_t to = cluster_address(S.list, 0), at = S.local_at;
        if (n_local <= kLocal)
          for (uint32_t i = threadIdx.x; i < n_local; i += kSampThreads)
            if (at + i < kList) cluster_store64(to + 8 * (at + i), S.local[i]);
      }
    }
    cluster_barrier();
    const uint32_t listed = cluster_load32(cluster_address(&S.list_n, 0));
    cluster_arrive();  // this CTA has read the number
    if (listed <= kList) {
      if (rank == 0) {
        if (listed <= 32 * kEach) {
          if (warp == 0) finish<false>(S, A, b, W, f, (int)listed, all_mass);
        } else {
          finish<true>(S, A, b, W, f, (int)listed, all_mass);
        }
      }
      cluster_wait();
      return;
    }
    cluster_wait();
  }

  // The longer way.  Its buckets: the distance from zmax in steps of `range` /
  // 2048; everything beyond 40 T (a share of 4e-18 each) falls into the last
  // one.  The distance rounds, the product rounds and the cut keeps the order,
  // so bins are ordered.
  float range = 0.f;
  if (by_k || by_p) {
    uint64_t low = kAll, same;
#pragma unroll 2
    for (int i = seg_lo + lane; i < seg_hi; i += 32)
      if (z[i] > -INFINITY) low = min(low, (uint64_t)rank_bits(z[i]));
    same = low;
    block_join<true>(S, &low, &same);
    meet(S, turn, low, 0);
    low = warp_min64(words(S, turn, 0, cluster, kAll));
    range = fminf(W.zmax - from_rank((uint32_t)low), 40.f * temperature);
  }
  const float bins_per = range > 0.f ? kBins / range : 0.f;
  const int n32 = (n + 31) & ~31;

  // What is kept: tokens up to place `upto`, of weight floor_w at least.
  uint64_t upto = kAll, sum = 0, before = 0, mine = 0, kept = 0;
  // 0: top-k's border; 1: the mass of what it keeps, and top-p's border;
  // 2: the kept mass; 3: as 2, of the tokens of one logit (a tie at a border)
  float tie = 0.f;
  uint64_t target = 0;
  bool tied = false, tied_mass = false;
#pragma unroll 1
  for (int phase = 0; phase < 3;) {
    if (phase == 0 && !tied && !by_k) {
      phase = 1;
      continue;
    }
    if (phase == 1 && !tied && !by_p) {
      phase = 2;
      continue;
    }
    if (phase > 0 || tied) {
      // sums in the order of ids: masses of the kept tokens, or the tied tokens' number
      uint64_t v = 0, c = 0;
      const double least = phase == 2 ? floor_w : 0.0;
#pragma unroll 4
      for (int i = seg_lo + lane; i < seg_hi; i += 32) {
        const float zi = z[i];
        if (!(zi > -INFINITY) || (upto != kAll && place(zi, base + i) > upto)) continue;
        if (tied) {
          v += zi == tie;
          continue;
        }
        if (least > 0.0 && W.weight(zi) < least) continue;
        v += W.mass(zi);
        ++c;
      }
      block_join<false>(S, &v, &c);
      mine = v;
      meet(S, turn, v, c);
      const uint64_t a = words(S, turn, 0, cluster, 0);
      sum = warp_sum64(a);
      before = warp_sum64(lane < rank ? a : 0);
      kept = warp_sum64(words(S, turn, 1, cluster, 0));
      if (phase == 2 || tied) {
        // the first token, in the order of ids, at which the sum is above `want`
        uint64_t want;
        if (tied) {
          if (tied_mass) {  // that many of them reach the target
            const uint64_t each = max((uint64_t)W.mass(tie), (uint64_t)1);
            target = (target + each - 1) / each;
          }
          want = min(target, sum) - 1;
        } else {
          want = min((uint64_t)(f.u * (double)sum), sum - 1);
        }
        const bool here = want >= before && want - before < mine;
        if (here) {  // the whole CTA
          uint64_t rest = want - before;
          bool holds = true;  // this warp does: uniform in it
#pragma unroll 1
          for (int w = 0; w < warp; ++w) {
            const uint64_t a = S.warp_a[w];
            holds = holds && rest >= a;
            rest -= a;
          }
          holds = holds && rest < S.warp_a[warp];
          if (holds) {
#pragma unroll 1
            for (int i0 = seg_lo; i0 < seg_hi; i0 += 32) {
              const int i = i0 + lane;
              uint64_t a = 0;
              if (i < seg_hi) {
                const float zi = z[i];
                if (zi > -INFINITY && place(zi, base + i) <= upto) {
                  if (tied)
                    a = zi == tie;
                  else if (floor_w == 0.0 || W.weight(zi) >= floor_w)
                    a = W.mass(zi);
                }
              }
              const uint64_t scan = warp_scan64(a);
              const uint32_t over = __ballot_sync(0xFFFFFFFFu, scan > rest);
              if (over) {
                if (lane == 0) S.found = i0 + __ffs(over) - 1;
                break;
              }
              rest -= __shfl_sync(0xFFFFFFFFu, scan, 31);
            }
          }
          __syncthreads();
        }
        if (phase == 2) {
          if (here && threadIdx.x == 0) {
            const int at = S.found;
            const double t = ((double)z[at] - (double)W.zmax) * W.inv_t;
            A.tok[b] = base + at;
            if (A.logprob) A.logprob[b] = (float)(t - log((double)sum / kOne));
            if (A.kept) A.kept[b] = (int)kept;
          }
          break;
        }
        // a tie: the owner tells the place of the last token kept
        meet(S, turn, here ? place(tie, base + S.found) : kAll, 0);
        upto = warp_min64(words(S, turn, 0, cluster, kAll));
        tied = false;
        ++phase;
        continue;
      }
    }

    // the border: the place of the last token of the shortest beginning of the
    // ranking whose count (or mass) reaches `target`
    const bool by_mass = phase == 1;
    float reach = INFINITY;
    if (by_mass) {
      const double want = ceil((double)p * (double)sum);
      target = min(want > 1.0 ? (uint64_t)want : (uint64_t)1, sum);
      // as reach_p, of the mass that top-k leaves
      reach = temperature *
              (logf(2.f * A.vocab / (1.f - fmaxf(p, 0.f))) - logf((float)((double)sum / kOne)) + 0.1f);
    } else {
      target = (uint64_t)k;
    }
    int bin = -1;             // the bin that holds the border,
    uint32_t lo = 0, hi = 0;  // of the rank bits lo .. hi; hi = 0: of the buckets
#pragma unroll 1
    for (int round = 0;; ++round) {
      __syncthreads();
      for (int i = threadIdx.x; i < kBins; i += kSampThreads) {
        S.count[i] = 0;
        S.mass[i] = 0;
      }
      if (threadIdx.x == 0) S.list_n = 0;
      __syncthreads();
#pragma unroll 1
      for (int i = threadIdx.x; i < n32; i += kSampThreads) {
        int to = -1;
        uint64_t u = 0;
        const float zi = i < n ? z[i] : -INFINITY;
        if (zi > -INFINITY && W.zmax - zi <= reach && place(zi, base + i) <= upto) {
          const uint32_t bits = rank_bits(zi);
          if (hi == 0)
            to = bucket((W.zmax - zi) * bins_per);
          else if (bits >= lo && bits <= hi)
            to = (int)((uint64_t)(hi - bits) * kBins / ((uint64_t)(hi - lo) + 1));
          if (by_mass && to >= 0) u = W.mass(zi);
        }
        add_to_bin(S, to, by_mass, u);
      }
      // rank 0 sums the CTAs' bins and finds the one that reaches the target
      cluster_barrier();
      turn ^= 1;
      if (rank == 0) {
        constexpr int each = kBins / kSampThreads;
        uint64_t v[each], c[each], all = 0;
#pragma unroll
        for (int i = 0; i < each; ++i) v[i] = c[i] = 0;
#pragma unroll 1
        for (int r = 0; r < cluster; ++r) {
          const uint32_t rc = cluster_address(&S.count[threadIdx.x * each], r);
          const uint32_t rm = cluster_address(&S.mass[threadIdx.x * each], r);
#pragma unroll
          for (int i = 0; i < each; ++i) {
            c[i] += cluster_load32(rc + 4 * i);
            v[i] += cluster_load64(rm + 8 * i);
          }
        }
#pragma unroll
        for (int i = 0; i < each; ++i) {
          if (!by_mass) v[i] = c[i];
          all += v[i];
        }
        uint64_t left = block_before(S, all);
#pragma unroll
        for (int i = 0; i < each; ++i) {
          if (left < target && target <= left + v[i]) {
            S.word[turn][0] = left;
            S.word[turn][1] = threadIdx.x * each + i;
            S.word[turn][2] = c[i];
          }
          left += v[i];
        }
      }
      cluster_barrier();
      target -= word(S, turn, 0, 0);
      bin = (int)word(S, turn, 1, 0);
      const uint32_t tokens = (uint32_t)word(S, turn, 2, 0);

      // the rank bits of its tokens; each round leaves a 2048th of the range
      uint64_t least = kAll, most = kAll;
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += kSampThreads) {
        const float zi = z[i];
        if (!(zi > -INFINITY) || !(W.zmax - zi <= reach) || place(zi, base + i) > upto) continue;
        const uint32_t bits = rank_bits(zi);
        int to = -1;
        if (hi == 0)
          to = bucket((W.zmax - zi) * bins_per);
        else if (bits >= lo && bits <= hi)
          to = (int)((uint64_t)(hi - bits) * kBins / ((uint64_t)(hi - lo) + 1));
        if (to != bin) continue;
        least = min(least, (uint64_t)bits);
        most = min(most, (uint64_t)~bits);
        if (tokens <= kList) {  // few enough to be sorted: rank 0's list takes them
          const uint32_t at = cluster_add32(cluster_address(&S.list_n, 0), 1u);
          if (at < kList) cluster_store64(cluster_address(S.list, 0) + 8 * at, place(zi, base + i));
        }
      }
      if (tokens <= kList) {
        cluster_barrier();
        turn ^= 1;
        if (rank == 0) {
          uint64_t key[kEach], v[kEach], sum = 0;
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            const int i = kEach * threadIdx.x + e;
            key[e] = i < (int)tokens ? S.list[i] : kAll;
          }
          sort_each(S, key, sort_size((int)tokens));
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            v[e] = key[e] == kAll ? 0 : by_mass ? W.mass(from_rank(~(uint32_t)(key[e] >> 32))) : 1;
            sum += v[e];
          }
          uint64_t left = block_before(S, sum);
#pragma unroll
          for (int e = 0; e < kEach; ++e) {
            if (left < target && target <= left + v[e]) S.word[turn][0] = key[e];
            left += v[e];
          }
        }
        cluster_barrier();
        upto = word(S, turn, 0, 0);
        ++phase;
        break;
      }
      block_join<true>(S, &least, &most);
      meet(S, turn, least, most);
      least = warp_min64(words(S, turn, 0, cluster, kAll));
      most = warp_min64(words(S, turn, 1, cluster, kAll));
      lo = (uint32_t)least;
      hi = ~(uint32_t)most;
      if (lo == hi || round == 5) {  // one logit: so many of its tokens, in the order of ids
        tied = true;
        tied_mass = by_mass;
        tie = from_rank(hi);
        break;
      }
    }
  }
  cluster_barrier();  // no CTA leaves while another may read its words
}

template <typename T>
cudaError_t launch(const SampleArgs& a, int batch, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(done.load(std::memory_order_acquire) >> dev & 1)) {
    e = cudaFuncSetAttribute(wpk_sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)sizeof(SampleShared) + kMaxVocab / kMaxCluster * 4);
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)batch * a.cluster);
  cfg.blockDim = dim3(kSampThreads);
  cfg.dynamicSmemBytes = sizeof(SampleShared) + a.slice * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = a.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, wpk_sample_kernel<T>, a);
}

}  // namespace
}  // namespace wpk

using namespace wpk;

extern "C" int wpk_sample(const void* logits_dev, int dtype, int batch, int vocab, int64_t row_stride,
                          const float* uniform_dev, const float* temperature_dev, const int32_t* top_k_dev,
                          const float* top_p_dev, const float* min_p_dev, int32_t* out_tok_dev,
                          float* out_logprob_dev, int32_t* out_kept_dev, void* stream) {
  if (!logits_dev || !uniform_dev || !out_tok_dev)
    return op_fail(WPK_ERR_INVALID_ARG, "null logits, uniform numbers or tokens");
  if (dtype != WPK_F32 && dtype != WPK_BF16 && dtype != WPK_F16) return op_fail(WPK_ERR_INVALID_ARG, "bad dtype");
  if (batch < 0 || vocab <= 0) return op_fail(WPK_ERR_INVALID_ARG, "batch must be >= 0 and vocab positive");
  if (vocab > kMaxVocab) return op_fail(WPK_ERR_UNSUPPORTED, "vocab must be <= 262144");
  if (row_stride < vocab && batch > 1) return op_fail(WPK_ERR_INVALID_ARG, "row_stride must be >= vocab");
  if (batch > INT_MAX / kMaxCluster) return op_fail(WPK_ERR_SHAPE, "too many rows for one call");
  if ((uintptr_t)logits_dev % (dtype == WPK_F32 ? 4 : 2))
    return op_fail(WPK_ERR_INVALID_ARG, "logits must be aligned to an element");
  if (batch == 0) return WPK_OK;
  SampleArgs a{logits_dev, row_stride, vocab, 0, 1, uniform_dev, temperature_dev, top_p_dev, min_p_dev, top_k_dev,
               out_tok_dev, out_logprob_dev, out_kept_dev};
  // CTAs of a row: one up to 8192 tokens; else as many as let two slices live in
  // an SM's shared memory, and up to 8 while the rows leave SMs (148) idle
  if (vocab > 8192) {
    a.cluster = std::min(kMaxCluster, (vocab + kTwoPerSm - 1) / kTwoPerSm);
    while (a.cluster < kMaxCluster && batch * (a.cluster + 1) <= 148) ++a.cluster;
  }
  a.slice = ((vocab + a.cluster - 1) / a.cluster + 127) / 128 * 128;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == WPK_F32    ? launch<float>(a, batch, s)
                        : dtype == WPK_BF16 ? launch<__nv_bfloat16>(a, batch, s)
                                            : launch<__half>(a, batch, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return op_fail(WPK_ERR_CUDA, cudaGetErrorString(e));
  }
  return WPK_OK;
}
