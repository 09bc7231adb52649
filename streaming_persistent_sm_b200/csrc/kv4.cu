// A paged KV cache held in 4 bits: append (with the position rotation on the
// way), read back, and the checks of all its entry points.  The attention over
// it is in kv4_attention.cu.
//
// A row of HD values (one token, one kv head, K or V) is handled by HD / 8
// lanes.  Lane j holds dims 4j .. 4j + 3 and HD / 2 + 4j .. + 3, so that both
// halves of a rotated pair are in one lane and its eight codes are one 32-bit
// word of the row.
#include <limits.h>

#include "kv4.cuh"
#include "kv4_host.h"
#include "op_util.cuh"

namespace wpk {
namespace {

constexpr int kThreadsKv4 = 128;

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

// Where row t of the call lives: its page (NULL: no place), its row in the
// page and its position; false: the row belongs to no sequence.
template <int LANES>
__device__ __forceinline__ bool locate(const Kv4Dev& c, int t, int head, int j, uint32_t mask, uint8_t** page, int* row,
                                       int* position) {
  *page = nullptr;
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
  const int slot = (int)p / c.page_tokens;
  const int block = c.table[(int64_t)b * c.max_blocks + slot];
  if (block < 0 || block >= c.n_blocks) return true;
  *page = kv4_page(c, block, head);
  *row = (int)p - slot * c.page_tokens;
  *position = (int)p;
  return true;
}

// The largest bf16 number <= x (as its bits), within the finite range.
__device__ __forceinline__ uint32_t bf16_down(double x) {
  uint32_t u = __float_as_uint(__double2float_rd(x));
  if (u & 0xFFFFu) u = (u & 0x80000000u) ? u + 0x10000u : u;  // away from zero below it
  u >>= 16;
  return u == 0xFF80u ? 0xFF7Fu : u;
}

// The bf16 number next to x >= 0, ties to even, rounded once: a float that is
// not x itself gets an odd last bit, so that it never looks like a tie.
__device__ __forceinline__ uint32_t bf16_near(double x) {
  float f = __double2float_rz(x);
  if ((double)f != x) f = __uint_as_float(__float_as_uint(f) | 1u);
  return __bfloat16_as_ushort(__float2bfloat16_rn(f));
}

__device__ __forceinline__ float lane_min(float a, float b) { return fminf(a, b); }
__device__ __forceinline__ float lane_max(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ double lane_min(double a, double b) { return fmin(a, b); }
__device__ __forceinline__ double lane_max(double a, double b) { return fmax(a, b); }

// Eight codes of this lane and the row's (s, z) word from the row's values, x
// in a type R that holds them exactly (float as given, double when rotated).
// The quotient (x - z) / s is computed in 32 bits, off by less than 3e-6; where
// it comes within 1e-4 of a border between two codes it is computed again in 64.
template <int LANES, typename R>
__device__ __forceinline__ void quantise(const R (&x)[8], uint32_t mask, uint32_t* codes, uint32_t* sz) {
  R lo = x[0], hi = x[0];
  bool fine = true;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    lo = lane_min(lo, x[e]);
    hi = lane_max(hi, x[e]);
    fine = fine && isfinite(x[e]);
  }
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) {
    lo = lane_min(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, o));
    hi = lane_max(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, o));
  }
  fine = (__ballot_sync(0xFFFFFFFFu, !fine) & mask) == 0;
  if (!fine) {  // s = 0, z = NaN: the row reads as NaN
    *codes = 0;
    *sz = 0x7FC00000u;
    return;
  }
  const uint32_t zb = bf16_down((double)lo);
  const float z = __uint_as_float(zb << 16);
  const uint32_t sb = bf16_near(((double)hi - (double)z) / 15.0);
  const float s = __uint_as_float(sb << 16);
  const float inv = 1.0f / s;
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float t = (float)(x[e] - (R)z) * inv;
    float c = rintf(t);
    if (!(fabsf(fabsf(t - c) - 0.5f) > 1e-4f) || !(inv < 3e38f))  // near a border, or s too small for inv
      c = s > 0.f ? (float)rint(((double)x[e] - (double)z) / (double)s) : 0.f;
    w |= (uint32_t)fminf(fmaxf(c, 0.f), 15.f) << (4 * e);
  }
  *codes = w;
  *sz = sb | (zb << 16);
}

// Bound by bytes: a row comes in once and leaves as HD / 2 + 4 bytes.  The
// rotation in 64 bits (two products and a sum a value, each product exact) makes
// the codes those of exact arithmetic.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreadsKv4)
    kv4_append_kernel(const Kv4Dev c, const T* __restrict__ k, int64_t k_tok, int64_t k_head, const T* __restrict__ v,
                      int64_t v_tok, int64_t v_head, const float* __restrict__ rope) {
  constexpr int LANES = HD / 8;
  const int lane = threadIdx.x & 31, j = lane % LANES;
  const uint32_t mask = ((1u << LANES) - 1u) << (lane - j);
  const uint32_t r = blockIdx.x * (kThreadsKv4 / LANES) + threadIdx.x / LANES;
  const int head = r % (uint32_t)c.n_kv, t = r / (uint32_t)c.n_kv;
  uint8_t* page;
  int row, position;
  locate<LANES>(c, t, head, j, mask, &page, &row, &position);
  float kx[8] = {}, vx[8] = {};
  if (page) {
    const T* kp = k + t * k_tok + head * k_head + 4 * j;
    const T* vp = v + t * v_tok + head * v_head + 4 * j;
    load4(kp, kx);
    load4(kp + HD / 2, kx + 4);
    load4(vp, vx);
    load4(vp + HD / 2, vx + 4);
  }
  uint32_t kw, ksz, vw, vsz;
  if (rope) {
    double x[8] = {};
    if (page) {
      float cs[8];
      const float* a = rope + ((int64_t)position * (HD / 2) + 4 * j) * 2;
      load4(a, cs);
      load4(a + 4, cs + 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const double co = cs[2 * e], si = cs[2 * e + 1], lo = kx[e], hi = kx[4 + e];
        x[e] = lo * co - hi * si;
        x[4 + e] = hi * co + lo * si;
      }
    }
    quantise<LANES>(x, mask, &kw, &ksz);
  } else {
    quantise<LANES>(kx, mask, &kw, &ksz);
  }
  quantise<LANES>(vx, mask, &vw, &vsz);
  if (!page) return;
  const int codes = c.page_tokens * (HD / 2);
  *reinterpret_cast<uint32_t*>(page + row * (HD / 2) + 4 * j) = kw;
  *reinterpret_cast<uint32_t*>(page + codes + row * (HD / 2) + 4 * j) = vw;
  uint32_t* sz = reinterpret_cast<uint32_t*>(page + 2 * codes) + row;
  if (j == 0) sz[0] = ksz;
  if (j == 1) sz[c.page_tokens] = vsz;
}

template <int HD, typename T>
__device__ __forceinline__ void read_row(uint32_t w, uint32_t sz, T* out) {
  const float s = __uint_as_float(sz << 16), z = __uint_as_float(sz & 0xFFFF0000u);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fmaf(s, (float)((w >> (4 * e)) & 15u), z);
  store4(out, x);
  store4(out + HD / 2, x + 4);
}

// Bound by bytes: the append's traffic, the other way.
template <typename T, int HD>
__global__ void __launch_bounds__(kThreadsKv4)
    kv4_read_kernel(const Kv4Dev c, T* __restrict__ k, int64_t k_tok, int64_t k_head, T* __restrict__ v, int64_t v_tok,
                    int64_t v_head) {
  constexpr int LANES = HD / 8;
  const int lane = threadIdx.x & 31, j = lane % LANES;
  const uint32_t mask = ((1u << LANES) - 1u) << (lane - j);
  const uint32_t r = blockIdx.x * (kThreadsKv4 / LANES) + threadIdx.x / LANES;
  const int head = r % (uint32_t)c.n_kv, t = r / (uint32_t)c.n_kv;
  uint8_t* page;
  int row, position;
  if (!locate<LANES>(c, t, head, j, mask, &page, &row, &position)) return;
  uint32_t kw = 0, vw = 0, ksz = 0, vsz = 0;
  if (page) {
    const int codes = c.page_tokens * (HD / 2);
    kw = *reinterpret_cast<const uint32_t*>(page + row * (HD / 2) + 4 * j);
    vw = *reinterpret_cast<const uint32_t*>(page + codes + row * (HD / 2) + 4 * j);
    const uint32_t* sz = reinterpret_cast<const uint32_t*>(page + 2 * codes) + row;
    ksz = sz[0];
    vsz = sz[c.page_tokens];
  }
  read_row<HD>(kw, ksz, k + t * k_tok + head * k_head + 4 * j);
  read_row<HD>(vw, vsz, v + t * v_tok + head * v_head + 4 * j);
}

template <int HD>
uint32_t row_blocks(const Kv4Dev& c) {
  constexpr int rows = kThreadsKv4 / (HD / 8);
  return (uint32_t)(((int64_t)c.total * c.n_kv + rows - 1) / rows);
}

template <typename T, int HD>
void launch_append(const Kv4Dev& c, const Kv4Tensor& k, const Kv4Tensor& v, const float* rope, cudaStream_t s) {
  kv4_append_kernel<T, HD><<<row_blocks<HD>(c), kThreadsKv4, 0, s>>>(
      c, static_cast<const T*>(k.p), k.token, k.head, static_cast<const T*>(v.p), v.token, v.head, rope);
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
  const char* bad = tensor_problem(k, dtype);
  if (!bad) bad = tensor_problem(v, dtype);
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
  if (!bad) bad = tensor_problem(o, dtype);
  if (bad) return op_fail(WPK_ERR_INVALID_ARG, bad);
  if (n_heads <= 0 || n_heads % cache->n_kv_heads)
    return op_fail(WPK_ERR_INVALID_ARG, "n_heads must be a positive multiple of n_kv_heads");
  if (max_new < 0) return op_fail(WPK_ERR_INVALID_ARG, "max_new must be >= 0");
  if (!(scale >= 0.f) || !(scale <= 3e38f)) return op_fail(WPK_ERR_INVALID_ARG, "scale must be finite and >= 0");
  return kv4_attention_launch(d, cache->head_dim, max_new, q, n_heads, dtype, rope_dev, scale, o,
                              static_cast<cudaStream_t>(stream));
}

}  // extern "C"
