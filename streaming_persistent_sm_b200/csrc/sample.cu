// wpk_sample: the next token of each row of logits, by temperature, top-k,
// top-p and min-p, with given uniform numbers.
//
// A cluster of CTAs takes a row.  Each CTA reads its slice of the row once into
// shared memory and all further passes run there: one read of the logits is what
// the operator has to move.  Nothing is sorted but the few tokens around a
// border: to find the last token that top-k or top-p keeps, the tokens fall into
// 2048 buckets by their distance from the largest logit, the counts (or masses)
// of the buckets, summed over the cluster, say in which bucket the border lies,
// and that bucket's tokens are sorted - after cutting its range of logits into
// 2048 again where it holds too many.  What is kept is then "up to this (logit,
// id)", one comparison a token.
//
// A token's weight exp((z - zmax) / T) is computed in 64 bits and held as a
// whole multiple of 2^-45, so that sums do not depend on their order (shared
// atomics, clusters of any size) and decisions at a border are those of the
// definition.  B200 runs 64-bit arithmetic at half the 32-bit rate.
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
constexpr int kList = 1024;         // tokens of the border's bucket that are sorted
constexpr int kMaxVocab = 1 << 18;  // 2^18 weights of at most 2^45 fit 63 bits
constexpr int kMaxCluster = 8;
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

struct Weigh {  // weights of a row's tokens
  float zmax;
  double inv_t;
  __device__ __forceinline__ double weight(float z) const {
    return z > -INFINITY ? exp_neg(((double)z - (double)zmax) * inv_t) : 0.0;
  }
  __device__ __forceinline__ uint64_t mass(float z) const { return __double2ull_rn(weight(z) * kOne); }
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

// Shared memory of a CTA: `fixed` bytes, then the slice's logits.
struct SampleShared {
  uint64_t mass[kBins];
  uint64_t list[kList];
  uint32_t count[kBins];
  uint64_t warp_a[kSampWarps], warp_b[kSampWarps];
  uint64_t word[2][4];  // what this CTA tells the others, in turn
  uint32_t list_n;
  int found;
  uint32_t pad[2];
};
static_assert(sizeof(SampleShared) % 16 == 0, "the slice behind it is aligned");

// Sums (or minima) of two values over the CTA, in every thread; warp_a keeps
// the warps' sums of the first.
template <bool kMin>
__device__ __forceinline__ void block_join(SampleShared& S, uint64_t* a, uint64_t* b) {
  const int warp = threadIdx.x >> 5;
  const uint64_t wa = kMin ? warp_min64(*a) : warp_sum64(*a), wb = kMin ? warp_min64(*b) : warp_sum64(*b);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    S.warp_a[warp] = wa;
    S.warp_b[warp] = wb;
  }
  __syncthreads();
  uint64_t ja = S.warp_a[0], jb = S.warp_b[0];
#pragma unroll 1
  for (int w = 1; w < kSampWarps; ++w) {
    ja = kMin ? min(ja, S.warp_a[w]) : ja + S.warp_a[w];
    jb = kMin ? min(jb, S.warp_b[w]) : jb + S.warp_b[w];
  }
  *a = ja;
  *b = jb;
}

// Publishes this CTA's words (thread 0's) and meets the others; word(turn, i, r)
// then reads rank r's, until the next meeting but one.
__device__ __forceinline__ void meet(SampleShared& S, int& turn, uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  turn ^= 1;
  if (threadIdx.x == 0) {
    S.word[turn][0] = a;
    S.word[turn][1] = b;
    S.word[turn][2] = c;
    S.word[turn][3] = d;
  }
  cluster_barrier();
}
__device__ __forceinline__ uint64_t word(const SampleShared& S, int turn, int i, int rank) {
  return cluster_load64(cluster_address(&S.word[turn][i], rank));
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
  const int warp = threadIdx.x >> 5;
  const uint64_t upto = warp_scan64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 31) S.warp_a[warp] = upto;
  __syncthreads();
  uint64_t left = upto - v;
#pragma unroll 1
  for (int w = 0; w < warp; ++w) left += S.warp_a[w];
  return left;
}

template <typename T>
__global__ void __launch_bounds__(kSampThreads) wpk_sample_kernel(const SampleArgs A) {
  extern __shared__ __align__(128) uint8_t smem[];
  SampleShared& S = *reinterpret_cast<SampleShared*>(smem);
  float* z = reinterpret_cast<float*>(smem + sizeof(SampleShared));
  const int cluster = A.cluster, rank = blockIdx.x % cluster, b = blockIdx.x / cluster;
  const int base = min(A.vocab, rank * A.slice), n = min(A.vocab - base, A.slice);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int turn = 0;

  // read the slice; the best token, the lowest logit that is not masked
  uint64_t best = kAll, low = kAll, finite = 0, bad = 0;
  {
    const T* src = static_cast<const T*>(A.logits) + b * A.stride + base;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kSampThreads) {
      const float zi = to_float(src[i]) + 0.f;  // -0 becomes +0
      z[i] = zi;
      if (!(zi < INFINITY)) bad = 1;
      if (zi > -INFINITY) {
        best = min(best, place(zi, base + i));
        low = min(low, (uint64_t)rank_bits(zi));
        ++finite;
      }
    }
  }
  block_join<false>(S, &finite, &bad);
  block_join<true>(S, &best, &low);
  meet(S, turn, best, low, finite, bad);
  finite = bad = 0;
#pragma unroll 1
  for (int r = 0; r < cluster; ++r) {
    best = min(best, word(S, turn, 0, r));
    low = min(low, word(S, turn, 1, r));
    finite += word(S, turn, 2, r);
    bad |= word(S, turn, 3, r);
  }
  const float temperature = A.temperature ? A.temperature[b] : 1.f;
  const bool none = bad != 0 || finite == 0;
  if (none || !(temperature > 0.f)) {  // as for every CTA of the cluster
    if (rank == 0 && threadIdx.x == 0) {
      A.tok[b] = none ? -1 : (int)(uint32_t)best;
      if (A.logprob) A.logprob[b] = none ? NAN : 0.f;
      if (A.kept) A.kept[b] = none ? 0 : 1;
    }
    cluster_barrier();  // no CTA leaves while another may read its words
    return;
  }

  Weigh W;
  W.zmax = from_rank(~(uint32_t)(best >> 32));
  W.inv_t = 1.0 / (double)temperature;
  // buckets: the distance from zmax in steps of `range` / 2048; everything
  // beyond 40 T (a share of 4e-18 each) falls into the last one.  The distance
  // rounds, the product rounds and the cut keeps the order, so bins are ordered.
  const float range = fminf(W.zmax - from_rank((uint32_t)low), 40.f * temperature);
  const float bins_per = range > 0.f ? kBins / range : 0.f;
  const int k = A.top_k ? A.top_k[b] : 0;
  const float p = A.top_p ? A.top_p[b] : 1.f;
  const float mp = A.min_p ? A.min_p[b] : 0.f;
  const double floor_w = mp > 0.f ? fmin((double)mp, 1.0) : 0.0;
  // a warp's tokens where the order of ids matters
  const int per = ((n + kSampWarps - 1) / kSampWarps + 31) & ~31;
  const int seg_lo = min(n, warp * per), seg_hi = min(n, seg_lo + per);
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
    if (phase == 0 && !tied && !(k > 0 && (uint64_t)k < finite)) {
      phase = 1;
      continue;
    }
    if (phase == 1 && !tied && !(p < 1.f)) {
      phase = 2;
      continue;
    }
    if (phase > 0 || tied) {
      // sums in the order of ids: masses of the kept tokens, or the tied tokens' number
      uint64_t v = 0, c = 0;
      const double least = phase == 2 ? floor_w : 0.0;
#pragma unroll 1
      for (int i = seg_lo + lane; i < seg_hi; i += 32) {
        const float zi = z[i];
        if (!(zi > -INFINITY) || place(zi, base + i) > upto) continue;
        if (tied) {
          v += zi == tie;
          continue;
        }
        const double w = W.weight(zi);
        if (w < least) continue;
        v += __double2ull_rn(w * kOne);
        ++c;
      }
      block_join<false>(S, &v, &c);
      mine = v;
      meet(S, turn, v, c, 0, 0);
      sum = before = kept = 0;
#pragma unroll 1
      for (int r = 0; r < cluster; ++r) {
        const uint64_t a = word(S, turn, 0, r);
        if (r < rank) before += a;
        sum += a;
        kept += word(S, turn, 1, r);
      }
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
          const float u = A.uniform[b];
          want = min((uint64_t)((u > 0.f ? fmin((double)u, 1.0) : 0.0) * (double)sum), sum - 1);
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
                  const double w = tied ? 0.0 : W.weight(zi);
                  a = tied ? (uint64_t)(zi == tie) : w < floor_w ? 0 : __double2ull_rn(w * kOne);
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
        meet(S, turn, here ? place(tie, base + S.found) : kAll, 0, 0, 0);
        uint64_t last = kAll;
#pragma unroll 1
        for (int r = 0; r < cluster; ++r) last = min(last, word(S, turn, 0, r));
        upto = last;
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
      // tokens with w below (1 - p) sum / (2 vocab) hold at most half of what
      // top-p leaves out, so the border is above them (and 0.1 for rounding)
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
            to = min((int)((W.zmax - zi) * bins_per), kBins - 1);
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
          to = min((int)((W.zmax - zi) * bins_per), kBins - 1);
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
          int size = 32;
          while (size < (int)tokens) size *= 2;
          for (int i = tokens + threadIdx.x; i < size; i += kSampThreads) S.list[i] = kAll;
          __syncthreads();
#pragma unroll 1
          for (int s = 2; s <= size; s *= 2)
#pragma unroll 1
            for (int j = s / 2; j > 0; j /= 2) {
              for (int i = threadIdx.x; i < size / 2; i += kSampThreads) {
                const int x = 2 * i - (i & (j - 1)), y = x + j;
                const uint64_t a = S.list[x], c = S.list[y];
                if ((a > c) == ((x & s) == 0)) {
                  S.list[x] = c;
                  S.list[y] = a;
                }
              }
              __syncthreads();
            }
          uint64_t v[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int i = 2 * threadIdx.x + e;
            v[e] = i >= (int)tokens ? 0 : by_mass ? W.mass(from_rank(~(uint32_t)(S.list[i] >> 32))) : 1;
          }
          uint64_t left = block_before(S, v[0] + v[1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (left < target && target <= left + v[e]) S.word[turn][0] = S.list[2 * threadIdx.x + e];
            left += v[e];
          }
        }
        cluster_barrier();
        upto = word(S, turn, 0, 0);
        ++phase;
        break;
      }
      block_join<true>(S, &least, &most);
      meet(S, turn, least, most, 0, 0);
#pragma unroll 1
      for (int r = 0; r < cluster; ++r) {
        least = min(least, word(S, turn, 0, r));
        most = min(most, word(S, turn, 1, r));
      }
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
  // CTAs of a row: one up to 8192 tokens; else as many as keep the slices in
  // shared memory, and up to 8 while the SMs (148) are not full
  if (vocab > 8192) {
    a.cluster = std::max(1, (vocab + kMaxVocab / kMaxCluster - 1) / (kMaxVocab / kMaxCluster));
    while (a.cluster < kMaxCluster && batch * a.cluster < 148) ++a.cluster;
  }
  a.slice = ((vocab + a.cluster - 1) / a.cluster + 31) / 32 * 32;
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
