// A paged KV cache held in 4 bits: append (with the position rotation on the
// way), read back, and the checks of all its entry points.  The attention over
// it is in kv4_attention.cu.
//
// A row of HD values (one token, one kv head, K or V) is handled by HD / 16
// lanes.  Lane j holds dims 8j .. 8j + 7 and HD / 2 + 8j .. + 7, so that both
// halves of a rotated pair are in one lane and its sixteen codes are two 32-bit
// words of the row.  A CTA takes consecutive tokens of one head: their rows are
// neighbours in a page.
//
// A row's place takes some loads that wait for one another (the search for its
// sequence, the position, the page id, the angles), 2 us or so; the append's rows
// are under way before their place is known.
//
// Measured, 8 kv heads of 64, bf16: 32 prompts of up to 496 tokens appended in 23 us
// (their 31 MB: 1.3 TB/s), read back in 10; 48 single tokens in 5 to 8 us, one in 3.1
// (latency).  The append is bound by instructions: codes in 32 bits with bounds, and
// where a bound says that a value may lie on a code's border, the exact decision;
// 16-bit values lie on ties of their own scale so often that most warps take it
// somewhere.
#include <limits.h>

#include "kv4.cuh"
#include "kv4_host.h"
#include "op_util.cuh"

namespace wpk {
namespace {

constexpr int kThreadsKv4 = 128;
constexpr int kOf = 16;  // values of a row that a lane holds

// Sequence of token t: the last b with indptr[b] <= t, searched by the LANES
// lanes of a row together (each round they probe LANES evenly spaced starts,
// so 48 sequences take two rounds of loads).
template <int LANES>
__device__ __forceinline__ int find_sequence(const Kv4Dev& c, int n_seq, int t, int j, uint32_t mask) {
  int lo = 0, n = n_seq;
  while (n > 1) {
    const int step = (n + LANES - 1) / LANES;
    const int at = j * step;
    const bool below = at < n && c.indptr[lo + at] <= t;
    const int hits = __popc(__ballot_sync(mask, below) & mask);
    const int skip = max(hits - 1, 0) * step;
    lo += skip;
    n = min(step, n - skip);
  }
  return lo;
}

// Where token t of the call lives: its page id (-1: no place), its row in the
// page and its position; false: the token belongs to no sequence.
template <int LANES>
__device__ __forceinline__ bool locate(const Kv4Dev& c, int t, int j, uint32_t mask, int* block, int* row,
                                       int* position) {
  *block = -1;
  *row = *position = 0;
  const int n_seq = kv4_sequences(c);
  int b, q0, n;
  if (c.indptr) {
    b = find_sequence<LANES>(c, n_seq, t, j, mask);
  } else {
    b = t / c.each;
  }
  if (t >= c.total || b >= n_seq) return false;
  kv4_new(c, b, &q0, &n);
  if (t < q0 || t - q0 >= n) return false;
  const int first = c.pos[b];
  const int64_t p = (int64_t)first + (t - q0);
  if (first < 0 || p >= (int64_t)c.max_blocks * c.page_tokens || p >= c.rope_positions) return true;
  const int slot = kv4_slot(c, (int)p);
  const int id = c.table[(int64_t)b * c.max_blocks + slot];
  if (id < 0 || id >= c.n_blocks) return true;
  *block = id;
  *row = (int)p - slot * c.page_tokens;
  *position = (int)p;
  return true;
}

// The largest bf16 number <= x (as its bits), within the finite range.
__device__ __forceinline__ uint32_t bf16_down(float x) {
  uint32_t u = __float_as_uint(x);
  if (u & 0xFFFFu) u = (u & 0x80000000u) ? u + 0x10000u : u;  // away from zero below it
  u >>= 16;
  return u == 0xFF80u ? 0xFF7Fu : u;
}
__device__ __forceinline__ uint32_t bf16_near(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
// The bf16 number next to x >= 0, ties to even, rounded once: a float that is
// not x itself gets an odd last bit, so that it never looks like a tie.
__device__ __forceinline__ uint32_t bf16_near(double x) {
  float f = __double2float_rz(x);
  if ((double)f != x) f = __uint_as_float(__float_as_uint(f) | 1u);
  return bf16_near(f);
}

// Codes of the lane's values from exact ones.
__device__ __noinline__ uint2 exact_codes(const double* x, float z, float s) {
  uint32_t w[2] = {0, 0};
#pragma unroll 1
  for (int e = 0; e < kOf; ++e) {
    const double c = s > 0.f ? rint((x[e] - (double)z) / (double)s) : 0.0;
    const uint32_t n = (uint32_t)fmin(fmax(c, 0.0), 15.0);
    // value e is the (e % 4)-th of its half of word (e / 4) % 2
    w[(e >> 2) & 1] |= n << (4 * ((e & 3) + (e >= kOf / 2 ? 4 : 0)));
  }
  return make_uint2(w[0], w[1]);
}

// The lane's values in 64 bits: turned (each product is exact, the sum rounds
// once), or as they are.
template <bool kTurn>
__device__ __forceinline__ void exact_values(const float (&a)[kOf], const float (&cs)[kOf], double* x) {
#pragma unroll
  for (int e = 0; e < kOf / 2; ++e) {
    const double lo = a[e], hi = a[kOf / 2 + e];
    x[e] = kTurn ? lo * cs[2 * e] - hi * cs[2 * e + 1] : lo;
    x[kOf / 2 + e] = kTurn ? hi * cs[2 * e] + lo * cs[2 * e + 1] : hi;
  }
}

// A row in 64 bits throughout.
template <int LANES>
__device__ __noinline__ uint3 quantise_exactly(const double* x, uint32_t mask) {
  double lo = x[0], hi = x[0];
  bool fine = true;
  for (int e = 0; e < kOf; ++e) {
    lo = fmin(lo, x[e]);
    hi = fmax(hi, x[e]);
    fine = fine && isfinite(x[e]);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = fmin(lo, __shfl_xor_sync(mask, lo, o));
    hi = fmax(hi, __shfl_xor_sync(mask, hi, o));
  }
  if (__ballot_sync(mask, !fine) & mask) return make_uint3(0u, 0u, 0x7FC00000u);  // s = 0, z = NaN: reads as NaN
  const uint32_t zb = bf16_down(__double2float_rd(lo));
  const float z = __uint_as_float(zb << 16);
  const uint32_t sb = bf16_near((hi - (double)z) / 15.0);
  const uint2 w = exact_codes(x, z, __uint_as_float(sb << 16));
  return make_uint3(w.x, w.y, sb | zb << 16);
}

// Sixteen codes of this lane and the row's (s, z) word, those of exact arithmetic.
// The work is done in 32 bits with bounds: a turned value is off by at most 2^-23
// of |a cos| + |b sin| (a product and a sum round), which 2 max |a| max |cos, sin|
// bounds.  Where z or s could be
// another bf16 number within the bounds (one row in some thousands), the row is
// done again in 64 bits; where a quotient is as near to the border between two
// codes, the lane's codes are (one turned value in 10^5).  Values that are not
// turned lie on the border itself more often - 16-bit numbers, their distance
// from z and s have few digits - and there the remainder x - z - c s decides,
// which 32 bits hold exactly where they hold x - z.
template <int LANES, bool kTurn>
__device__ __forceinline__ uint3 quantise(const float (&a)[kOf], const float (&cs)[kOf], uint32_t mask) {
  constexpr int HALF = kOf / 2;
  float x[kOf], bound = 0.f;
  if (kTurn) {
    float am = 0.f, cm = 0.f;
#pragma unroll
    for (int e = 0; e < kOf; e += 2) {
      am = max3(am, fabsf(a[e]), fabsf(a[e + 1]));
      cm = max3(cm, fabsf(cs[e]), fabsf(cs[e + 1]));
    }
    bound = 2.f * am * cm;
#pragma unroll
    for (int e = 0; e < HALF; e += 2) {
      const F2 lo = pair(a[e], a[e + 1]), hi = pair(a[HALF + e], a[HALF + e + 1]);
      const F2 co = pair(cs[2 * e], cs[2 * e + 2]), si = pair(cs[2 * e + 1], cs[2 * e + 3]);
      const F2 minus = pair(-cs[2 * e + 1], -cs[2 * e + 3]);
      const float2 r = split(fma2(lo, co, mul2(hi, minus))), q = split(fma2(hi, co, mul2(lo, si)));
      x[e] = r.x;
      x[e + 1] = r.y;
      x[HALF + e] = q.x;
      x[HALF + e + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < kOf; ++e) x[e] = a[e];
  }
  float lo = x[0], hi = x[0];
  F2 none = pair(0.f, 0.f);  // a NaN where any value is one, or infinite
#pragma unroll
  for (int e = 0; e < kOf; e += 2) {
    lo = min3(lo, x[e], x[e + 1]);
    hi = max3(hi, x[e], x[e + 1]);
    none = fma2(pair(x[e], x[e + 1]), pair(0.f, 0.f), none);
  }
  const float2 no = split(none);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
    if (kTurn) bound = fmaxf(bound, __shfl_xor_sync(0xFFFFFFFFu, bound, o));
  }
  const float off = kTurn ? bound * 0x1p-22f : 0.f;  // twice the bound, for the sums below
  const bool fine = (__ballot_sync(0xFFFFFFFFu, no.x != 0.f || no.y != 0.f) & mask) == 0;
  const uint32_t zb = bf16_down(lo + off);
  const float z = __uint_as_float(zb << 16);
  const float d = hi - z;
  const float least = (d - off) * (0.06666667f * 0.9999995f), most = (d + off) * (0.06666667f * 1.0000005f);
  const uint32_t sb = bf16_near(most);
  if (!fine || (kTurn && bf16_down(lo - off) != zb) || bf16_near(least) != sb || !(most < 1e37f)) {
    double exact[kOf];
    exact_values<kTurn>(a, cs, exact);
    return quantise_exactly<LANES>(exact, mask);
  }
  // (x - z) / s lies within 0 .. 15.03 and what `close` leaves, so the nearest
  // whole number within 0 .. 15; adding 1.5 * 2^23 leaves it in the low bits, ties
  // to even.  The upper bits of a word's eight sums cancel against a constant.
  const float s = __uint_as_float(sb << 16), inv = s > 0.f ? 1.0f / s : 0.f;
  const float close = 0.5f - fmaf(off, inv, 4e-6f);  // no closer to a whole number and a half than this
  const F2 z2 = pair(-z, -z), inv2 = pair(inv, inv), up = pair(12582912.f, 12582912.f),
           down = pair(-12582912.f, -12582912.f), neg = pair(-1.f, -1.f);
  uint32_t w[2] = {0u - 0x4B400000u * 0x11111111u, 0u - 0x4B400000u * 0x11111111u};
  float far = 0.f;
#pragma unroll
  for (int e = 0; e < kOf; e += 2) {
    const F2 t = mul2(add2(pair(x[e], x[e + 1]), z2), inv2), r = add2(t, up);
    const float2 rs = split(r), f = split(fma2(add2(r, down), neg, t));
    far = max3(far, fabsf(f.x), fabsf(f.y));
    const int at = 4 * ((e & 3) + (e >= HALF ? 4 : 0));
    w[(e >> 2) & 1] += (__float_as_uint(rs.x) << at) + (__float_as_uint(rs.y) << (at + 4));
  }
  if (!(far <= close)) {  // (a NaN of an infinite inv: close is one)
    bool held = !kTurn && inv < 1e37f;
    if (!kTurn) {
      w[0] = w[1] = 0;
      const float half = 0.5f * s;  // s is no denormal number here: inv is finite
#pragma unroll
      for (int e = 0; e < kOf; ++e) {
        const float y = x[e] - z;
        held = held && y + z == x[e] && x[e] - y == z;  // nothing was rounded off
        const float r = y * inv + 12582912.f, rest = fmaf(-(r - 12582912.f), s, y);
        int c = (int)(__float_as_uint(r) & 15u);
        if (rest > half || (rest == half && (c & 1))) ++c;
        if (-rest > half || (-rest == half && (c & 1))) --c;
        w[(e >> 2) & 1] |= (uint32_t)c << (4 * ((e & 3) + (e >= HALF ? 4 : 0)));
      }
    }
    if (!held) {
      double exact[kOf];
      exact_values<kTurn>(a, cs, exact);
      const uint2 r = exact_codes(exact, z, s);
      w[0] = r.x;
      w[1] = r.y;
    }
  }
  return make_uint3(w[0], w[1], sb | zb << 16);
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  load4(p, f);
  load4(p + 4, f + 4);
}

// A row comes in once and leaves as HD / 2 + 4 bytes; bound by the instructions of
// its codes.
template <typename T, int HD, bool kTurn>
__global__ void __launch_bounds__(kThreadsKv4, kTurn ? 7 : 8)
    kv4_append_kernel(const Kv4Dev c, const T* __restrict__ k, int64_t k_tok, int64_t k_head, const T* __restrict__ v,
                      int64_t v_tok, int64_t v_head, const float* __restrict__ rope) {
  constexpr int LANES = HD / kOf;
  const int lane = threadIdx.x & 31, j = lane % LANES, head = blockIdx.y;
  const uint32_t mask = ((1u << LANES) - 1u) << (lane - j);
  const int t = blockIdx.x * (kThreadsKv4 / LANES) + threadIdx.x / LANES;
  float kx[kOf] = {}, vx[kOf] = {}, cs[kOf] = {};
  if (t < c.total) {
    const T* kp = k + t * k_tok + head * k_head + 8 * j;
    const T* vp = v + t * v_tok + head * v_head + 8 * j;
    load8(vp, vx);
    load8(vp + HD / 2, vx + 8);
    load8(kp, kx);
    load8(kp + HD / 2, kx + 8);
  }
  int block, row, position;
  locate<LANES>(c, t, j, mask, &block, &row, &position);
  if (kTurn && block >= 0) {
    const float* a = rope + ((int64_t)position * (HD / 2) + 8 * j) * 2;
    load8(a, cs);
    load8(a + 8, cs + 8);
  }
  const uint3 vq = quantise<LANES, false>(vx, cs, mask);
  const uint3 kq = quantise<LANES, kTurn>(kx, cs, mask);
  if (block < 0) return;
  uint8_t* page = kv4_page(c, block, head);
  const int codes = c.page_tokens * (HD / 2);
  *reinterpret_cast<uint2*>(page + row * (HD / 2) + 8 * j) = make_uint2(kq.x, kq.y);
  *reinterpret_cast<uint2*>(page + codes + row * (HD / 2) + 8 * j) = make_uint2(vq.x, vq.y);
  uint32_t* sz = reinterpret_cast<uint32_t*>(page + 2 * codes) + row;
  if (j == 0) sz[0] = kq.z;
  if (j == 1) sz[c.page_tokens] = vq.z;
}

// A word of a row's codes as values, to dims 4w and HD / 2 + 4w of it.
template <int HD, typename T>
__device__ __forceinline__ void read_word(uint32_t w, uint32_t sz, T* out) {
  const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xFFFF0000u);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fmaf(s, (float)((w >> (4 * e)) & 15u), z);
  store4(out, x);
  store4(out + HD / 2, x + 4);
}

// The append's traffic, the other way, in twice the time of its bytes: a row's codes
// wait for the loads that say where they are, and leave as 8 bytes a store.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreadsKv4)
    kv4_read_kernel(const Kv4Dev c, T* __restrict__ k, int64_t k_tok, int64_t k_head, T* __restrict__ v, int64_t v_tok,
                    int64_t v_head) {
  constexpr int LANES = HD / kOf;
  const int lane = threadIdx.x & 31, j = lane % LANES, head = blockIdx.y;
  const uint32_t mask = ((1u << LANES) - 1u) << (lane - j);
  const int t = blockIdx.x * (kThreadsKv4 / LANES) + threadIdx.x / LANES;
  int block, row, position;
  if (!locate<LANES>(c, t, j, mask, &block, &row, &position)) return;
  uint2 kw = make_uint2(0, 0), vw = kw;
  uint32_t ksz = 0, vsz = 0;
  if (block >= 0) {
    const int codes = c.page_tokens * (HD / 2);
    const uint8_t* page = kv4_page(c, block, head);
    const uint32_t* sz = reinterpret_cast<const uint32_t*>(page + 2 * codes) + row;
    kw = *reinterpret_cast<const uint2*>(page + row * (HD / 2) + 8 * j);
    vw = *reinterpret_cast<const uint2*>(page + codes + row * (HD / 2) + 8 * j);
    ksz = sz[0];
    vsz = sz[c.page_tokens];
  }
  T *kp = k + t * k_tok + head * k_head + 8 * j, *vp = v + t * v_tok + head * v_head + 8 * j;
  read_word<HD>(kw.x, ksz, kp);
  read_word<HD>(kw.y, ksz, kp + 4);
  read_word<HD>(vw.x, vsz, vp);
  read_word<HD>(vw.y, vsz, vp + 4);
}

template <int HD>
dim3 row_blocks(const Kv4Dev& c) {
  constexpr int tokens = kThreadsKv4 / (HD / kOf);
  return dim3((unsigned)((c.total + tokens - 1) / tokens), (unsigned)c.n_kv);
}

template <typename T, int HD>
void launch_append(const Kv4Dev& c, const Kv4Tensor& k, const Kv4Tensor& v, const float* rope, cudaStream_t s) {
  const T *kp = static_cast<const T*>(k.p), *vp = static_cast<const T*>(v.p);
  if (rope)
    kv4_append_kernel<T, HD, true>
        <<<row_blocks<HD>(c), kThreadsKv4, 0, s>>>(c, kp, k.token, k.head, vp, v.token, v.head, rope);
  else
    kv4_append_kernel<T, HD, false>
        <<<row_blocks<HD>(c), kThreadsKv4, 0, s>>>(c, kp, k.token, k.head, vp, v.token, v.head, rope);
}

template <typename T, int HD>
void launch_read(const Kv4Dev& c, const Kv4Tensor& k, const Kv4Tensor& v, cudaStream_t s) {
  kv4_read_kernel<T, HD><<<row_blocks<HD>(c), kThreadsKv4, 0, s>>>(
      c, static_cast<T*>(const_cast<void*>(k.p)), k.token, k.head, static_cast<T*>(const_cast<void*>(v.p)), v.token,
      v.head);
}

int launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return WPK_OK;
  char msg[160];
  snprintf(msg, sizeof msg, "%s: %s", what, cudaGetErrorString(e));
  return op_fail(WPK_ERR_CUDA, msg);
}

// Checks of a tensor of the call.
const char* tensor_problem(const Kv4Tensor& x, int dtype) {
  const uintptr_t align = dtype == WPK_F32 ? 16 : 8;
  if (!x.p) return "null tensor";
  if ((uintptr_t)x.p % align) return "a tensor must be aligned to 4 elements";
  if (x.token % 4 || x.head % 4 || x.token < 0 || x.head < 0) return "strides must be multiples of 4 elements, >= 0";
  return nullptr;
}

// And of one that the call writes: rows of their own.
const char* output_problem(const Kv4Tensor& x, int dtype, int total, int heads, int head_dim) {
  const char* bad = tensor_problem(x, dtype);
  if (bad) return bad;
  if ((total > 1 && x.token < head_dim) || (heads > 1 && x.head < head_dim)) return "rows that are written must not overlap";
  return nullptr;
}

}  // namespace

// Checks what all calls share and fills the device view; returns WPK_OK or the
// code of a recorded failure.
int kv4_view(const wpk_kv4_cache* cache, const int32_t* pos, const int32_t* indptr, int total, int dtype,
             const float* rope, int rope_positions, Kv4Dev* d) {
  if (!cache || !pos) return op_fail(WPK_ERR_INVALID_ARG, "null cache or positions");
  if (!cache->pages_dev || !cache->block_table_dev) return op_fail(WPK_ERR_INVALID_ARG, "null pages or block table");
  if ((uintptr_t)cache->pages_dev % 16) return op_fail(WPK_ERR_INVALID_ARG, "pages must be 16-byte aligned");
  if (cache->batch <= 0 || cache->max_blocks <= 0 || cache->n_kv_heads <= 0 || cache->n_blocks <= 0)
    return op_fail(WPK_ERR_INVALID_ARG, "cache sizes must be positive");
  if (cache->n_blocks > INT_MAX) return op_fail(WPK_ERR_SHAPE, "more than 2^31 - 1 pages");
  int64_t bytes = 0;
  const int rc = wpk_kv4_page_bytes(cache->head_dim, cache->page_tokens, &bytes);
  if (rc) return rc;
  if ((int64_t)cache->max_blocks * cache->page_tokens > INT_MAX)
    return op_fail(WPK_ERR_SHAPE, "a sequence of more than 2^31 - 1 positions");
  if (dtype != WPK_F32 && dtype != WPK_BF16 && dtype != WPK_F16) return op_fail(WPK_ERR_INVALID_ARG, "bad dtype");
  if (total < 0) return op_fail(WPK_ERR_INVALID_ARG, "total must be >= 0");
  if (cache->n_kv_heads > 65535) return op_fail(WPK_ERR_SHAPE, "more than 65535 kv heads");
  if ((int64_t)total * cache->n_kv_heads > INT_MAX) return op_fail(WPK_ERR_SHAPE, "more than 2^31 - 1 rows");
  if (!indptr && total % cache->batch)
    return op_fail(WPK_ERR_SHAPE, "without indptr, total must be a multiple of the batch");
  if (rope && rope_positions <= 0) return op_fail(WPK_ERR_INVALID_ARG, "rope_positions must be positive");
  if ((uintptr_t)rope % 16) return op_fail(WPK_ERR_INVALID_ARG, "the rope table must be 16-byte aligned");
  d->pages = static_cast<uint8_t*>(cache->pages_dev);
  d->table = cache->block_table_dev;
  d->n_blocks = cache->n_blocks;
  d->batch = cache->batch;
  d->max_blocks = cache->max_blocks;
  d->n_kv = cache->n_kv_heads;
  d->page_tokens = cache->page_tokens;
  d->page_bytes = (int)bytes;
  d->page_magic = kv4_page_magic(cache->page_tokens);
  d->pos = pos;
  d->indptr = indptr;
  d->n_seq = nullptr;
  d->total = total;
  d->each = total / cache->batch;
  d->rope_positions = rope ? rope_positions : INT_MAX;
  return WPK_OK;
}

int kv4_append_launch(const Kv4Dev& d, int head_dim, const Kv4Tensor& k, const Kv4Tensor& v, int dtype,
                      const float* rope, cudaStream_t s) {
  if (d.total == 0) return WPK_OK;
  const bool wide = head_dim == 128;
  if (dtype == WPK_F32)
    wide ? launch_append<float, 128>(d, k, v, rope, s) : launch_append<float, 64>(d, k, v, rope, s);
  else if (dtype == WPK_BF16)
    wide ? launch_append<__nv_bfloat16, 128>(d, k, v, rope, s) : launch_append<__nv_bfloat16, 64>(d, k, v, rope, s);
  else
    wide ? launch_append<__half, 128>(d, k, v, rope, s) : launch_append<__half, 64>(d, k, v, rope, s);
  return launched("wpk_kv4_append");
}

}  // namespace wpk

using namespace wpk;

extern "C" {

int wpk_kv4_page_bytes(int head_dim, int page_tokens, int64_t* bytes) {
  if (!bytes) return op_fail(WPK_ERR_INVALID_ARG, "null output");
  if (head_dim != 64 && head_dim != 128) return op_fail(WPK_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (page_tokens <= 0 || page_tokens % 16 || page_tokens > 256)
    return op_fail(WPK_ERR_INVALID_ARG, "page_tokens must be a multiple of 16, <= 256");
  *bytes = (int64_t)page_tokens * 2 * (head_dim / 2 + 4);
  return WPK_OK;
}

int wpk_kv4_append(const wpk_kv4_cache* cache, const int32_t* pos_dev, const int32_t* indptr_dev, int total,
                   const void* k_dev, int64_t k_token_stride, int64_t k_head_stride, const void* v_dev,
                   int64_t v_token_stride, int64_t v_head_stride, int dtype, const float* rope_dev,
                   int rope_positions, void* stream) {
  Kv4Dev d;
  const int rc = kv4_view(cache, pos_dev, indptr_dev, total, dtype, rope_dev, rope_positions, &d);
  if (rc) return rc;
  const Kv4Tensor k{k_dev, k_token_stride, k_head_stride}, v{v_dev, v_token_stride, v_head_stride};
  const char* bad = tensor_problem(k, dtype);
  if (!bad) bad = tensor_problem(v, dtype);
  if (bad) return op_fail(WPK_ERR_INVALID_ARG, bad);
  return kv4_append_launch(d, cache->head_dim, k, v, dtype, rope_dev, static_cast<cudaStream_t>(stream));
}

int wpk_kv4_read(const wpk_kv4_cache* cache, const int32_t* pos_dev, const int32_t* indptr_dev, int total, void* k_dev,
                 int64_t k_token_stride, int64_t k_head_stride, void* v_dev, int64_t v_token_stride,
                 int64_t v_head_stride, int dtype, void* stream) {
  Kv4Dev d;
  const int rc = kv4_view(cache, pos_dev, indptr_dev, total, dtype, nullptr, 0, &d);
  if (rc) return rc;
  const Kv4Tensor k{k_dev, k_token_stride, k_head_stride}, v{v_dev, v_token_stride, v_head_stride};
  const char* bad = output_problem(k, dtype, total, cache->n_kv_heads, cache->head_dim);
  if (!bad) bad = output_problem(v, dtype, total, cache->n_kv_heads, cache->head_dim);
  if (bad) return op_fail(WPK_ERR_INVALID_ARG, bad);
  if (total == 0) return WPK_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = cache->head_dim == 128;
  if (dtype == WPK_F32)
    wide ? launch_read<float, 128>(d, k, v, s) : launch_read<float, 64>(d, k, v, s);
  else if (dtype == WPK_BF16)
    wide ? launch_read<__nv_bfloat16, 128>(d, k, v, s) : launch_read<__nv_bfloat16, 64>(d, k, v, s);
  else
    wide ? launch_read<__half, 128>(d, k, v, s) : launch_read<__half, 64>(d, k, v, s);
  return launched("wpk_kv4_read");
}

int wpk_kv4_attention(const wpk_kv4_cache* cache, const int32_t* pos_dev, const int32_t* indptr_dev, int total,
                      int max_new, const void* q_dev, int64_t q_token_stride, int64_t q_head_stride, int n_heads,
                      int dtype, const float* rope_dev, int rope_positions, float scale, void* out_dev,
                      int64_t out_token_stride, int64_t out_head_stride, void* stream) {
  Kv4Dev d;
  const int rc = kv4_view(cache, pos_dev, indptr_dev, total, dtype, rope_dev, rope_positions, &d);
  if (rc) return rc;
  const Kv4Tensor q{q_dev, q_token_stride, q_head_stride}, o{out_dev, out_token_stride, out_head_stride};
  const char* bad = tensor_problem(q, dtype);
  if (!bad) bad = output_problem(o, dtype, total, n_heads, cache->head_dim);
  if (bad) return op_fail(WPK_ERR_INVALID_ARG, bad);
  if (n_heads <= 0 || n_heads % cache->n_kv_heads)
    return op_fail(WPK_ERR_INVALID_ARG, "n_heads must be a positive multiple of n_kv_heads");
  if (max_new < 0) return op_fail(WPK_ERR_INVALID_ARG, "max_new must be >= 0");
  if (!(scale >= 0.f) || !(scale <= 3e38f)) return op_fail(WPK_ERR_INVALID_ARG, "scale must be finite and >= 0");
  return kv4_attention_launch(d, cache->head_dim, max_new, q, n_heads, dtype, rope_dev, scale, o,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
