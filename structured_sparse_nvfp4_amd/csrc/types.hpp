// Element types of the calls that take f32, bf16 and f16 alike (the codes of include/ssnvfp4.h:
// SSN_F32, SSN_BF16, SSN_F16): conversions to f32 and back, rounded to nearest even.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssn {

constexpr int kF32 = 0, kBF16 = 1, kF16 = 2;

__device__ __forceinline__ float bf16_of(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float f16_of(uint16_t b) { return (float)__builtin_bit_cast(_Float16, b); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
__device__ __forceinline__ uint16_t to_f16(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }

// a 16-bit value of type t (kBF16 or kF16)
__device__ __forceinline__ float float16_of(uint16_t b, int t) { return t == kF16 ? f16_of(b) : bf16_of(b); }

// v >= 0 rounded to the 16-bit type t (through f32), at most its largest finite value
__device__ __forceinline__ uint16_t round16_sat(double v, int t) {
  if (t == kF16) return to_f16(fminf((float)v, 65504.f));
  return to_bf16(fminf((float)v, __uint_as_float(0x7F7F0000u)));
}

__device__ __forceinline__ void store_elem(void* p, int t, int64_t i, float v) {
  if (t == kF32) ((float*)p)[i] = v;
  else ((uint16_t*)p)[i] = t == kF16 ? to_f16(v) : to_bf16(v);
}

}  // namespace ssn
