// Which page of a sequence holds a position (host and device; a test compiles it
// with the host compiler).
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define WPK_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define WPK_HOST_DEVICE inline
#endif

namespace wpk {

// Pages hold 16 m tokens, m <= 16, so position / page_tokens is
// (position / 16) / m, here by the factor 2^35 / m rounded up: below 2^31 the
// first quotient is below 2^27, the product below 2^63, and the rounding adds
// less than 2^27 / 2^35 = 2^-8 < 1 / m, so the whole part is exact.
WPK_HOST_DEVICE uint64_t kv4_page_magic(int page_tokens) {
  const uint64_t m = (uint64_t)page_tokens / 16;
  return ((1ull << 35) + m - 1) / m;
}
WPK_HOST_DEVICE int kv4_slot_of(int position, uint64_t magic) {
  return (int)(((uint64_t)((uint32_t)position >> 4) * magic) >> 35);
}

}  // namespace wpk
