// What the attention kernels over a 4-bit cache share: copies, codes as fp16
// operands, and what each type keeps.
#pragma once
#include <type_traits>

#include "op_util.cuh"
#include "ptx.cuh"

namespace wpk {

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

constexpr uint32_t kEven = 0x000F000Fu, kOdd = 0x00F000F0u;

// The codes less kLess of two even nibbles, and of two odd ones times 16.
template <int kLess = 8>
__device__ __forceinline__ uint32_t centred_even(uint32_t w) {
  const uint32_t u = (w & kEven) | 0x64006400u, less = (0x6400u + kLess) * 0x10001u;  // 1024 + kLess
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&less));
  return *reinterpret_cast<const uint32_t*>(&d);
}
template <int kLess = 8>
__device__ __forceinline__ uint32_t centred_odd(uint32_t w) {
  const uint32_t u = (w & kOdd) | 0x64006400u, less = (0x6400u + 16 * kLess) * 0x10001u;
  const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&u), *reinterpret_cast<const __half2*>(&less));
  return *reinterpret_cast<const uint32_t*>(&d);
}

template <bool kCentre>
__device__ __forceinline__ uint32_t codes_even(uint32_t w) {
  return kCentre ? centred_even(w) : w & kEven;
}
template <bool kCentre>
__device__ __forceinline__ uint32_t codes_odd(uint32_t w) {
  return kCentre ? centred_odd(w) : w & kOdd;
}

// Exponent fields of V's scales that the weights of a row follow: a weight stays
// below 2^(141 - field), so that times a scale s it is below 2^15, what an fp16
// operand holds, and times an offset y below 2^79, which 2^31 keys sum up within
// fp32.  A field below kLeastExp would let the sum of 2^31 weights overflow.
constexpr uint32_t kLeastExp = 45;
__device__ __forceinline__ uint32_t v_key_exp(float s, float y) {
  const uint32_t es = (__float_as_uint(s) >> 23) & 255u, ey = (__float_as_uint(y) >> 23) & 255u;
  return max(max(min(es, 254u), ey == 255u ? 0u : ey - min(ey, 64u)), kLeastExp);  // a NaN says nothing
}

// A key's weight times its scale is an fp16 number of at most 2^15, and as long
// as the exponent fields of the keys so far differ by no more than kSpread, their
// largest stands for all: the product that counts most is then above 2^2, and
// what the others lose below 2^-14 (2^-25 each) is nothing beside it.  Where they
// differ by more, the bound follows each row's own largest product, so that a
// value of no weight, or one that the row does not see, costs the others nothing.
// Operands that hold values (bf16, many rows) have one power of two for all keys,
// or one for each, by the same rule: 2^12 below the largest, which stands at 2^15
// at most, a value keeps all of fp16's digits.
constexpr uint32_t kSpread = 12;

// What a type's precision asks for.  bf16: Q and P rounded to fp16 (2^-11 at most), V's
// codes as they are (they add 5e-4 to the 1.7e-3 that the output's rounding is off,
// relative, of random values).  fp16: Q to 22 bits, V centred.  fp32: K centred and P
// to 22 bits too.  All: the products of a step (few rows) or tile in sums of their own,
// since the tensor pipe cuts off what its sums cannot hold: over 2^18 keys in one sum
// fp16 answers came out 4e-3 too small.
template <typename T>
struct Keep {
  static constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value, kFp32 = std::is_same<T, float>::value;
  static constexpr bool kQLow = !kBf16, kPLow = kFp32, kCentreK = kFp32, kCentreV = !kBf16;
};

}  // namespace wpk
