// One block of NVFP4, shared by the kernels that quantise (k_quant.hip: weights, k_kv_cache.hip: keys and
// values): the E4M3 scale of 16 values and their E2M1 codes, every rounding decision exact.
#pragma once
#include "common.hpp"

namespace ssn {

// E4M3 nearest-even of q >= 0, saturating at 448 (0x7E); q is an exactly rounded float64.
__device__ __forceinline__ uint32_t e4m3_rne(double q) {
  if (!(q < 448.0)) return 0x7Eu;
  if (q < 0.015625) {                          // below 2^-6: subnormal spacing 2^-9
    double m = rint(q * 512.0);                // exact scaling; rint ties to even
    return (uint32_t)m;                        // 8 -> 0x08 (= 2^-6), still correct
  }
  int e = ilogb(q);                            // -6 .. 8
  double mant = ldexp(q, -e) - 1.0;            // [0, 1), exact
  double m8 = rint(mant * 8.0);
  if (m8 >= 8.0) { m8 = 0.0; e += 1; }
  return (uint32_t)(((e + 7) << 3) | (int)m8);
}

__device__ __forceinline__ double e4m3_f64(uint32_t b) {
  int e = (b >> 3) & 15, m = b & 7;
  return e == 0 ? ldexp((double)m, -9) : ldexp(1.0 + m / 8.0, e - 7);
}

// Per block of 16 values: S, then 16 codes packed into 8 bytes.
//
// E2M1 decision thresholds m * d (exact float64 products): ties at 0.25, 1.25, 2.5 and 5 go
// down, at 0.75, 1.75 and 3.5 up, so code = [a > 0.25d] + [a >= 0.75d] + [a > 1.25d] +
// [a >= 1.75d] + [a > 2.5d] + [a >= 3.5d] + [a > 5d]. For a float x: x > T <=> x > RD(T), and
// x >= T <=> x >= RU(T), so rounding each threshold once to f32 (down, resp. up) keeps every
// decision exact. The seven tests are evaluated as a three-level search: bit 2 of the code is
// [a >= 1.75d], bit 1 is [a >= 0.75d] or [a >= 3.5d], bit 0 the remaining test of that quarter.
struct Thresholds {
  float e175, e075, e35, g025, g125, g25, g5;
};

// The thresholds are passed by value so that they stay in registers: the quarter's threshold is
// picked with two selects, not by indexing a spilled copy of the struct.
__device__ __forceinline__ uint32_t e2m1_code(float a, float e175, float e075, float e35, float g025, float g125,
                                              float g25, float g5) {
  const bool b2 = a >= e175;
  const float t1 = b2 ? e35 : e075;
  const bool b1 = a >= t1;
  const float lo = b1 ? g125 : g025;
  const float hi = b1 ? g5 : g25;
  const bool b0 = a > (b2 ? hi : lo);
  return ((uint32_t)b2 << 2) | ((uint32_t)b1 << 1) | (uint32_t)b0;
}

// S and the 16 codes of one block.
__device__ __forceinline__ void quantize_block(const float (&w)[16], double st, u32x2& code, uint32_t& S) {
  float amax = 0.f;
#pragma unroll
  for (int t = 0; t < 16; ++t) amax = fmaxf(amax, fabsf(w[t]));
  S = 0;
  if (st > 0.0) S = e4m3_rne((double)amax / (6.0 * st));
  const double d = st * e4m3_f64(S);           // exact: <= 24 + 4 significant bits
  uint32_t lo = 0, hi = 0;                     // a block whose scale is zero stores code 0x0
  if (d > 0.0) {
    Thresholds th;
    th.g025 = __double2float_rd(0.25 * d); th.g125 = __double2float_rd(1.25 * d);
    th.g25 = __double2float_rd(2.5 * d);   th.g5 = __double2float_rd(5.0 * d);
    th.e075 = __double2float_ru(0.75 * d); th.e175 = __double2float_ru(1.75 * d);
    th.e35 = __double2float_ru(3.5 * d);
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      uint32_t c = e2m1_code(fabsf(w[t]), th.e175, th.e075, th.e35, th.g025, th.g125, th.g25, th.g5);
      c |= (__float_as_uint(w[t]) >> 28) & 8u;  // sign bit -> bit 3 (keeps -0 for tiny negatives)
      if (t < 8) lo |= c << (4 * t); else hi |= c << (4 * (t - 8));
    }
  }
  code[0] = lo; code[1] = hi;
}

}  // namespace ssn
