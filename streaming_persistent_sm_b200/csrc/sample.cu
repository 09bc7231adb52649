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
// takes some 20 operations; the bulk of a row, of weights below 2^-24, is
// computed in 32 bits with the exponent's rounding errors carried along, 2^-22
// of such a weight, which is half of 2^-45.  (From 2^-14 down the same would save a
// fifth of a row's time, but 2^17 such tokens shift a border by a hundredth of a
// token: other draws than the definition's.)
//
// Measured, fp32 logits of 128256 (three inputs each): one row with top-p 11 to 23 us,
// 48 rows with all filters 31 to 66, 128 with most of the tokens masked in half of the
// rows 68 to 85 (0.8 to 1 TB/s of 66 MB); 32 rows of 2048: 6.7.  Latency bounds it: the
// barriers between a row's passes, the 64-bit weights under top-p, and for a large
// top-k or a flat row the one CTA that sorts.
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
  // pairs of terms, so that few depend on one another
  const double r2 = r * r, r4 = r2 * r2;
  const double p0 = 1.0 + r, p1 = fma(r, 1.0 / 6.0, 0.5), p2 = fma(r, 1.0 / 120.0, 1.0 / 24.0),
               p3 = fma(r, 1.0 / 5040.0, 1.0 / 720.0), p4 = fma(r, 1.0 / 362880.0, 1.0 / 40320.0);
  double p = fma(fma(r4, p4, fma(r2, p3, p2)), r4, fma(r2, p1, p0));
  p *= p;
  p *= p;
  return __hiloint2double(__double2hiint(p) + (n << 20), __double2loint(p));
}

// Weights below 2^-kTail are computed in 32 bits, to half of 2^-45: 2^-22 of such a
// weight.  See tail_mass for those below 2^-kFar.
constexpr float kTail = 24.f;
constexpr float kFar = 29.f;

struct Weigh {  // weights of a row's tokens
  float zmax, log2_t, log2_t_rest;  // log2(e) / T and what its float leaves
  double inv_t;
  __device__ __forceinline__ double weight(float z) const {
    return z > -INFINITY ? exp_neg(((double)z - (double)zmax) * inv_t) : 0.0;
  }
  // log2 of the weight, to 2^-20 or so: enough to choose a way
  __device__ __forceinline__ float log2_weight(float z) const { return (z - zmax) * log2_t; }
  __device__ __forceinline__ uint64_t heavy_mass(float z) const { return __double2ull_rn(weight(z) * kOne); }
  // The mass of a token of log2_weight t < -kTail.  Down to 2^-kFar the exponent
  // is carried with its rounding errors (of the distance and of the product) and
  // split into a whole number and a rest below 1/2, so the error is ex2's, 2^-22.
  // Below, t's own rounding (2^-18 of the weight) is less than 1/4 of 2^-45.
  __device__ __forceinline__ uint32_t tail_mass(float z, float t) const {
    float rest = t + 45.f, scale = 1.f, m;
    if (!(t < -kFar)) {
      const float d = z - zmax, back = d + zmax;
      const float lost = (z - back) + (zmax - (back - d));  // z - zmax - d
      const float n = rintf(t);
      rest = (t - n) + fmaf(d, log2_t, -t) + fmaf(d, log2_t_rest, lost * log2_t);
      scale = __int_as_float((int)n + (45 + 127) << 23);
    }
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(m) : "f"(rest));
    return __float2uint_rn(m * scale);
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
constexpr int kLocalBits = 10, kLocal = 1 << kLocalBits;
struct SampleShared {
  union {
    uint64_t mass[kBins];
    uint64_t list[kList];  // the bins' masses are read before the list is filled
  };
  union {
    uint32_t count[kBins];
    uint64_t local[kLocal];  // the first CTA's, once the buckets are read
  };
  uint64_t warp_a[kSampWarps], warp_b[kSampWarps];
  uint64_t word[2][4];  // what this CTA tells the others, in turn
  uint32_t part[3][kSampWarps];
  uint32_t list_n, local_n, local_at;  // entries of the list, of `local` (of the list, elsewhere than first)
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

constexpr int kEach = kList / kSampThreads;  // entries of the list that a thread holds

struct Filters {
  int k;           // top-k's number, where it is on
  float p;         // top-p's share
  bool by_k, by_p;
  double floor_w;  // min-p, 0: off
  double u;
};

// An answer, by one thread.
__device__ __forceinline__ void answer(const SampleArgs& A, int b, const Weigh& W, uint32_t id, float z, uint64_t mass,
                                       int kept) {
  A.tok[b] = (int)id;
  if (A.logprob) {
    const double t = ((double)z - (double)W.zmax) * W.inv_t;
    A.logprob[b] = (float)(t - log((double)mass / kOne));
  }
  if (A.kept) A.kept[b] = kept;
}
__device__ __forceinline__ float logit_of(uint64_t place) { return from_rank(~(uint32_t)(place >> 32)); }

// What a CTA does with few tokens: four lanes a token go through all of them
// and add up what comes before it - 128 * 128 comparisons, no order made.
constexpr int kFew = kSampThreads / 4;
__device__ __forceinline__ uint64_t four_sum(uint64_t v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 1);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 2);
}

// The draw among n <= kFew tokens: places in S.list, in S.local twice their mass
// and 1 where they are kept.
__device__ __forceinline__ void draw_few(const SampleShared& S, const SampleArgs& A, int b, const Weigh& W, double u,
                                         int n) {
  const int e = threadIdx.x >> 2;
  const uint64_t mine = e < n ? S.list[e] : 0, own = e < n ? S.local[e] : 0;
  uint64_t mass = 0, kept = 0, before = 0;
#pragma unroll 2
  for (int j = threadIdx.x & 3; j < n; j += 4) {
    const uint64_t w = (S.local[j] & 1) ? S.local[j] >> 1 : 0;
    mass += w;
    kept += S.local[j] & 1;
    if ((uint32_t)S.list[j] < (uint32_t)mine) before += w;
  }
  mass = four_sum(mass);
  kept = four_sum(kept);
  before = four_sum(before);
  const uint64_t want = min((uint64_t)(u * (double)mass), mass - 1);
  if ((threadIdx.x & 3) == 0 && (own & 1) && before <= want && want - before < own >> 1)
    answer(A, b, W, (uint32_t)mine, logit_of(mine), mass, (int)kept);
}

// The rest of a row from its n <= kFew candidates: a beginning of the ranking
// that holds all that can be kept.  all_mass: that of the whole row, for top-p
// without top-k.
__device__ __forceinline__ void finish_few(SampleShared& S, const SampleArgs& A, int b, const Weigh& W,
                                           const Filters& f, int n, uint64_t all_mass) {
  const int e = threadIdx.x >> 2;
  if (threadIdx.x < n) S.local[threadIdx.x] = W.mass(logit_of(S.list[threadIdx.x])) << 1;
  __syncthreads();
  const uint64_t mine = e < n ? S.list[e] : 0, own = e < n ? S.local[e] >> 1 : 0;
  uint64_t rank = 0, before = 0;
#pragma unroll 2
  for (int j = threadIdx.x & 3; j < n; j += 4)
    if (S.list[j] < mine) {
      ++rank;
      before += S.local[j] >> 1;
    }
  rank = four_sum(rank);
  before = four_sum(before);
  bool keep = !f.by_k || rank < (uint64_t)f.k;
  if (f.by_p) {
    if (f.by_k) {  // the mass that top-k leaves
      __syncthreads();
      if ((threadIdx.x & 3) == 0 && e < n) S.local[e] = own << 1 | keep;
      __syncthreads();
      all_mass = 0;
      for (int j = threadIdx.x & 3; j < n; j += 4)
        if (S.local[j] & 1) all_mass += S.local[j] >> 1;
      all_mass = four_sum(all_mass);
    }
    // kept while what comes before falls short of the share
    keep = keep && (before == 0 || (double)before < (double)f.p * (double)all_mass);
  }
  if (f.floor_w > 0.0) keep = keep && W.weight(logit_of(mine)) >= f.floor_w;
  __syncthreads();
  if ((threadIdx.x & 3) == 0 && e < n) S.local[e] = own << 1 | keep;
  __syncthreads();
  draw_few(S, A, b, W, f.u, n);
}

// Among the n <= kList keys of the list (whole CTAs) up to `upto`: the last one
// of the shortest beginning, in ascending order, whose number (or mass) reaches
// `target`, which all of them together do.  Keys are places, or ids with the
// rank bits' complement below them (by_id).  They fall into bins by their high
// word; the ones of the border's bin are compared with one another.
__device__ __forceinline__ uint64_t select(SampleShared& S, const Weigh& W, int n, bool by_mass, bool by_id,
                                           uint64_t target, uint64_t upto) {
  uint64_t least = kAll, most = kAll;
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kSampThreads) {
    const uint64_t key = S.list[i];
    least = min(least, key);
    if (key <= upto) most = min(most, ~key);
  }
  block_join<true>(S, &least, &most);
  const uint32_t lo = (uint32_t)(least >> 32), span = (uint32_t)(~most >> 32) - lo;
  const int shift = max(0, 32 - __clz(span) - kLocalBits);
  for (int i = threadIdx.x; i < kLocal; i += kSampThreads) S.local[i] = 0;
  if (threadIdx.x == 0) S.local_n = 0;
  __syncthreads();
  auto bin_of = [&](uint64_t key) { return (int)(((uint32_t)(key >> 32) - lo) >> shift); };
  auto worth = [&](uint64_t key) {
    return by_mass ? W.mass(from_rank(~(uint32_t)(by_id ? key : key >> 32))) : (uint64_t)1;
  };
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kSampThreads) {
    const uint64_t key = S.list[i];
    if (key <= upto)
      atomicAdd(reinterpret_cast<unsigned long long*>(&S.local[bin_of(key)]), (unsigned long long)worth(key));
  }
  __syncthreads();
  {
    static_assert(kLocal == 2 * kSampThreads && kLocal == 1 << kLocalBits, "two bins a thread");
    const uint64_t v0 = S.local[2 * threadIdx.x], v1 = S.local[2 * threadIdx.x + 1];
    const uint64_t left = block_before(S, v0 + v1);
    if (left < target && target <= left + v0 + v1) {
      const bool second = target > left + v0;
      S.found = 2 * threadIdx.x + second;
      S.warp_b[0] = left + (second ? v0 : 0);
    }
  }
  __syncthreads();
  const int bin = S.found;
  target -= S.warp_b[0];
  // its keys, together (as many as there is room for)
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kSampThreads) {
    const uint64_t key = S.list[i];
    if (key <= upto && bin_of(key) == bin) {
      const uint32_t at = atomicAdd(&S.local_n, 1u);
      if (at < kLocal) S.local[at] = key;
    }
  }
  __syncthreads();
  const int in = (int)S.local_n;
  const bool all = in > kLocal;  // else go through the whole list
  const int m = all ? n : in;
#pragma unroll 1
  for (int i = threadIdx.x; i < m; i += kSampThreads) {
    const uint64_t key = all ? S.list[i] : S.local[i];
    if (all && !(key <= upto && bin_of(key) == bin)) continue;
    uint64_t before = 0;
#pragma unroll 1
    for (int j = 0; j < m && before < target; ++j) {
      const uint64_t other = all ? S.list[j] : S.local[j];
      if (other < key && (!all || (other <= upto && bin_of(other) == bin))) before += worth(other);
    }
    if (before < target && target <= before + worth(key)) S.warp_b[1] = key;
  }
  __syncthreads();
  return S.warp_b[1];
}

// The rest of a row from its n candidates, kFew < n <= kList (whole CTAs).
__device__ __forceinline__ void finish_many(SampleShared& S, const SampleArgs& A, int b, const Weigh& W,
                                            const Filters& f, int n, uint64_t all_mass) {
  uint64_t upto = kAll;
#pragma unroll 1
  for (int by_mass = 0; by_mass < 2; ++by_mass) {
    if (by_mass ? !f.by_p : !f.by_k) continue;
    uint64_t target = (uint64_t)f.k;
    if (by_mass) {
      uint64_t in = 0, same = 0;  // the mass that is in the list, up to top-k's border
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += kSampThreads)
        if (S.list[i] <= upto) in += W.mass(logit_of(S.list[i]));
      block_join<false>(S, &in, &same);
      const double want = ceil((double)f.p * (double)(f.by_k ? in : all_mass));
      target = want > 1.0 ? (uint64_t)want : (uint64_t)1;
      if (target > in) continue;  // all of the list (min-p ends it)
    }
    if (by_mass || target < (uint64_t)n) upto = select(S, W, n, by_mass, false, target, upto);
  }
  // the kept ones together
  __syncthreads();
  if (threadIdx.x == 0) S.local_n = 0;
  __syncthreads();
  uint64_t key[kEach], mass = 0, kept = 0;
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int i = e * kSampThreads + threadIdx.x;
    key[e] = i < n ? S.list[i] : kAll;
    const bool on = i < n && key[e] <= upto && (f.floor_w == 0.0 || W.weight(logit_of(key[e])) >= f.floor_w);
    if (!on) key[e] = kAll;
    if (on) mass += W.mass(logit_of(key[e]));
    kept += on;
  }
  block_join<false>(S, &mass, &kept);  // every key is read
  if (kept <= kFew) {
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (key[e] != kAll) {
        const uint32_t at = atomicAdd(&S.local_n, 1u);
        S.list[at] = key[e];
        S.local[at] = W.mass(logit_of(key[e])) << 1 | 1;
      }
    __syncthreads();
    draw_few(S, A, b, W, f.u, (int)kept);
    return;
  }
  // many: in the order of ids
#pragma unroll
  for (int e = 0; e < kEach; ++e)
    if (key[e] != kAll) {
      const uint32_t at = atomicAdd(&S.local_n, 1u);
      S.list[at] = key[e] << 32 | key[e] >> 32;
    }
  __syncthreads();
  const uint64_t want = min((uint64_t)(f.u * (double)mass), mass - 1);
  const uint64_t drawn = select(S, W, (int)kept, true, true, want + 1, kAll);
  if (threadIdx.x == 0) answer(A, b, W, (uint32_t)(drawn >> 32), from_rank(~(uint32_t)drawn), mass, (int)kept);
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
  // the row's settings, asked for before its logits
  const float temperature = A.temperature ? A.temperature[b] : 1.f, u_part = A.uniform[b];
  const float p = A.top_p ? A.top_p[b] : 1.f, mp = A.min_p ? A.min_p[b] : 0.f;
  const int k = A.top_k ? A.top_k[b] : 0;

  for (int i = threadIdx.x; i < kBins; i += kSampThreads) S.count[i] = 0;
  if (threadIdx.x == 0) S.list_n = 0;

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
  f.k = k;
  f.p = p;
  f.by_k = k > 0 && (uint32_t)k < finite;
  f.by_p = p < 1.f;
  f.floor_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
  f.u = u_part > 0.f ? fmin((double)u_part, 1.0) : 0.0;
  const bool by_k = f.by_k, by_p = f.by_p;
  const double floor_w = f.floor_w;
  const bool filtered = by_k || by_p || floor_w > 0.0;

  // The mass of all tokens: what a row without filters draws from, and top-p
  // alone is measured by.  For the latter, tokens of 2^-kTail and more fall into
  // buckets of 1/80 of their weights' log2; a bucket sums up 2^13 times what its
  // tokens weigh against its near edge, rounded down (1 - x ln 2 <= 2^-x); 2^18
  // tokens fit 32 bits.
  constexpr float kSteps = 80.f;
  static_assert(kTail * kSteps < kBins, "a bucket for every token");
  uint64_t all_mass = 0;
  if (!filtered || (by_p && !by_k)) {
    uint64_t v = 0;
#pragma unroll 1
    for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
      const float4 x4 = *reinterpret_cast<const float4*>(z + i);
      const float x[4] = {x4.x, x4.y, x4.z, x4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float t = W.log2_weight(x[e]);
        if (t < -kTail)
          v += W.tail_mass(x[e], t);
        else if (x[e] > -INFINITY)
          v += W.heavy_mass(x[e]);
        if (filtered && !(t < -kTail)) {
          const float at = fmaxf(-t, 0.f) * kSteps, edge = floorf(at);  // a NaN is 0
          atomicAdd(&S.count[(int)edge], (uint32_t)(8192.f - (at - edge) * (5678.27f / kSteps)));
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
                if (left <= rest && rest < left + u[e])  // in one lane
                  answer(A, b, W, (uint32_t)(base + i + e), z[i + e], all_mass, (int)finite);
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

  // What is kept: tokens up to place `upto`, of weight floor_w at least.
  uint64_t upto = kAll;
  bool known = false;  // upto is
  {
    // the candidates: tokens no further than `reach` from the largest logit, or
    // (flat rows under top-p alone) those of the border's buckets
    float reach = INFINITY;
    int border_bin = -1;
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
      // each CTA sums up its share of the buckets over the cluster; the share
      // that reaches the target is then read by all
      const int share = kBins / cluster + (kBins % cluster != 0);  // >= 256
      const int first = rank * share, mine_n = max(0, min(share, kBins - first));
      const double want = ceil((double)p * (double)all_mass);
      const uint64_t target = by_k ? (uint64_t)k : want > 1.0 ? (uint64_t)want : 1;
      auto worth = [&](int bin, uint64_t c) {  // mass at the near edge, less what the float arithmetic may add
        return by_k ? c : __double2ull_rd((double)c * (double)(exp2f(32.f - bin / kSteps) * 0.999999f));
      };
      uint64_t sum = 0, tokens = 0;
#pragma unroll 1
      for (int i = threadIdx.x; i < mine_n; i += kSampThreads) {
        uint32_t got[kMaxCluster];
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)  // all on their way at once
          got[r] = r < cluster ? cluster_load32(cluster_address(&S.count[first + i], r)) : 0;
        uint32_t c = 0;
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r) c += got[r];
        S.count[first + i] = c;  // this share of this CTA's buckets is read by itself alone
        tokens += (c + 8191) >> 13;
        sum += worth(first + i, c);
      }
      block_join<false>(S, &sum, &tokens);
      meet(S, turn, sum, tokens);
      sum = words(S, turn, 0, cluster, 0);
      tokens = words(S, turn, 1, cluster, 0);
      const uint64_t upto_rank = warp_scan64(sum), tokens_upto = warp_scan64(tokens);
      const uint32_t over = __ballot_sync(0xFFFFFFFFu, lane < cluster && upto_rank >= target);
      int bin = kBins;  // not reached
      uint64_t near = 0;  // tokens up to the bucket (top-p), roughly
      if (over) {
        const int owner = __ffs(over) - 1;
        uint64_t left = __shfl_sync(0xFFFFFFFFu, upto_rank - sum, owner);
        near = __shfl_sync(0xFFFFFFFFu, tokens_upto - tokens, owner);
        const int at0 = owner * share, q = (share + kSampThreads - 1) / kSampThreads;
        uint64_t c[kEach], all = 0, in_bins = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const int i = at0 + threadIdx.x * q + e;
          const bool in = e < q && i < min(at0 + share, kBins);
          const uint32_t n_in = in ? cluster_load32(cluster_address(&S.count[i], owner)) : 0;
          c[e] = worth(i, n_in);
          all += c[e];
          in_bins += (n_in + 8191) >> 13;
        }
        if (threadIdx.x == 0) S.found = kBins;
        left += block_before(S, all);
        __syncthreads();  // warp_a is read
        const uint64_t nearer = block_before(S, in_bins) + in_bins;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          if (left < target && target <= left + c[e]) {
            S.found = at0 + threadIdx.x * q + e;
            S.warp_b[0] = nearer;
          }
          left += c[e];
        }
        __syncthreads();
        bin = S.found;
        near += S.warp_b[0];
      }
      // the bucket's far edge, and what the bucketing rounds
      if (bin < kBins && by_k) reach = (bin + 1) * ((float)kRange / kBins) * 1.00001f;
      if (bin < kBins && !by_k) {
        reach = ((bin + 1) * (1.f / kSteps) * 1.00001f) / W.log2_t;
        if (near > kList - kList / 16) border_bin = bin;
      }
    }
    // (with top-k, only its tokens may be dropped by min-p afterwards)
    if (floor_w > 0.0 && !by_k) {
      const float least = temperature * (0.01f - logf((float)floor_w));
      if (least < reach) {
        reach = least;
        border_bin = -1;
      }
    }
    // the first CTA's go straight into its list, another's together
    uint64_t nearer = 0;
    if (threadIdx.x == 0) S.local_n = 0;
    __syncthreads();
#pragma unroll 1
    for (int i = seg_lo + 4 * lane; i < seg_hi; i += 128) {
      const float4 v = *reinterpret_cast<const float4*>(z + i);
      const float x[4] = {v.x, v.y, v.z, v.w};
      if (!(W.zmax - fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) <= reach)) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        bool in = x[e] > -INFINITY && W.zmax - x[e] <= reach;
        if (border_bin >= 0 && in) {
          const float at = fmaxf(-W.log2_weight(x[e]), 0.f) * kSteps;
          in = at >= (float)(border_bin - 1) && at < (float)(border_bin + 1);
          if (at < (float)(border_bin - 1)) nearer += W.mass(x[e]);
        }
        if (!in) continue;
        const uint32_t at = atomicAdd(rank == 0 ? &S.list_n : &S.local_n, 1u);
        if (at < kList) S.list[at] = place(x[e], base + i + e);
      }
    }
    if (border_bin >= 0) {
      uint64_t same = 0;
      block_join<false>(S, &nearer, &same);
      turn ^= 1;
      if (threadIdx.x == 0) S.word[turn][0] = nearer;
    }
    if (rank != 0) {
      __syncthreads();
      const uint32_t n_local = S.local_n;
      if (n_local) {
        if (threadIdx.x == 0) S.local_at = cluster_add32(cluster_address(&S.list_n, 0), n_local);
        __syncthreads();
        const uint32_t to = cluster_address(S.list, 0), at = S.local_at;
        for (uint32_t i = threadIdx.x; i < n_local && at + i < kList; i += kSampThreads)
          cluster_store64(to + 8 * (at + i), S.list[i]);
      }
    }
    cluster_barrier();
    const uint32_t listed = cluster_load32(cluster_address(&S.list_n, 0));
    if (border_bin < 0 && listed <= kList) {
      cluster_arrive();  // this CTA has read the number
      if (rank == 0) {
        if (listed <= kFew)
          finish_few(S, A, b, W, f, (int)listed, all_mass);
        else
          finish_many(S, A, b, W, f, (int)listed, all_mass);
      }
      cluster_wait();
      return;
    }
    if (border_bin >= 0 && listed <= kList) {
      // the border among the listed ones, if it is among them
      nearer = warp_sum64(words(S, turn, 0, cluster, 0));
      turn ^= 1;
      if (rank == 0) {
        uint64_t in = 0, same = 0, last = kAll;
#pragma unroll 1
        for (int i = threadIdx.x; i < (int)listed; i += kSampThreads) in += W.mass(logit_of(S.list[i]));
        block_join<false>(S, &in, &same);
        const double want = ceil((double)p * (double)all_mass);
        const uint64_t target = want > 1.0 ? (uint64_t)want : (uint64_t)1;
        if (nearer < target && target - nearer <= in)
          last = select(S, W, (int)listed, true, false, target - nearer, kAll);
        if (threadIdx.x == 0) S.word[turn][0] = last;
      }
      cluster_barrier();
      upto = word(S, turn, 0, 0);
      known = upto != kAll;
    }
  }

  // The longer way.  Its buckets: the distance from zmax in steps of `range` /
  // 2048; everything beyond 40 T (a share of 4e-18 each) falls into the last
  // one.  The distance rounds, the product rounds and the cut keeps the order,
  // so bins are ordered.
  float range = 0.f;
  if (!known && (by_k || by_p)) {
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

  uint64_t sum = 0, before = 0, mine = 0, kept = 0;
  // 0: top-k's border; 1: the mass of what it keeps, and top-p's border;
  // 2: the kept mass; 3: as 2, of the tokens of one logit (a tie at a border)
  float tie = 0.f;
  uint64_t target = 0;
  bool tied = false, tied_mass = false;
#pragma unroll 1
  for (int phase = known ? 2 : 0; phase < 3;) {
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
            answer(A, b, W, (uint32_t)(base + at), z[at], sum, (int)kept);
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
      // tokens beyond it together weigh less than half of the 1 - p that is left out:
      // no more than vocab times what one at the distance weighs
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
          const uint64_t last = select(S, W, (int)tokens, by_mass, false, target, kAll);
          if (threadIdx.x == 0) S.word[turn][0] = last;
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
