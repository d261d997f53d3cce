// Integer 4-bit weights with group scales: quantise, dequantise, and the matrix-vector product for
// one token or a few, plain and grouped by expert.
//
//   W_hat[n, k] = s[n, g] * (q[n, k] - z[n, g]),  g = k / group,   q in 0..15, z = 8 without zeros
//   Y[m, n] = sum_k X[m, k] W_hat[n, k] = sum_g s[n, g] * sum_{k in g} X[m, k] (q[n, k] - z[n, g])
//
// The sum inside a group runs over whole numbers times activations, in f32, and the scale multiplies
// it once: no weight is ever rounded.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------------------ quantise
// The whole number nearest to w / s (s > 0), halves to the even one.
__device__ __forceinline__ float nearest_multiple(float w, float s) { return (float)rint((double)w / (double)s); }

// One thread per group.
__global__ __launch_bounds__(kThreads) void k_int4_quantize(const void* __restrict__ W, int wt, int64_t N, int64_t K,
                                                            int64_t group, int64_t groups, uint8_t* __restrict__ codes,
                                                            uint16_t* __restrict__ scales, int st,
                                                            uint8_t* __restrict__ zeros) {
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < N * groups; i += (int64_t)gridDim.x * kThreads) {
    const int64_t n = i / groups, g = i - n * groups;
    const int64_t k0 = g * group, k1 = min(K, k0 + group);
    float lo = 0.f, hi = 0.f;
    for (int64_t k = k0; k < k1; ++k) {
      const float w = load_elem(W, wt, n * K + k);
      lo = fminf(lo, w);
      hi = fmaxf(hi, w);
    }
    const double range = zeros ? ((double)hi - (double)lo) / 15.0 : (double)fmaxf(hi, -lo) / 7.0;
    const uint16_t sb = round16_sat(range, st);
    const float s = float16_of(sb, st);
    float z = 8.f;
    if (zeros) z = s > 0.f ? fminf(fmaxf(nearest_multiple(-lo, s), 0.f), 15.f) : 0.f;
    for (int64_t k = k0; k < k1; k += 2) {
      uint32_t b = 0;
      for (int j = 0; j < 2; ++j) {
        const float w = load_elem(W, wt, n * K + k + j);
        const float q = s > 0.f ? fminf(fmaxf(nearest_multiple(w, s) + z, 0.f), 15.f) : z;
        b |= (uint32_t)q << (4 * j);
      }
      codes[(n * K + k) / 2] = (uint8_t)b;
    }
    scales[i] = sb;
    if (zeros) zeros[i] = (uint8_t)z;
  }
}

// One thread per pair of codes.
__global__ __launch_bounds__(kThreads) void k_int4_dequantize(const uint8_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales, int st,
                                                              const uint8_t* __restrict__ zeros, int64_t N, int64_t K,
                                                              int64_t group, int64_t groups, void* __restrict__ out,
                                                              int ot) {
  const int64_t Kh = K / 2;
  for (int64_t i = blockIdx.x * (int64_t)kThreads + threadIdx.x; i < N * Kh; i += (int64_t)gridDim.x * kThreads) {
    const int64_t n = i / Kh, k = 2 * (i - n * Kh), sg = n * groups + k / group;
    const float s = float16_of(scales[sg], st), z = zeros ? (float)zeros[sg] : 8.f;
    store_elem(out, ot, 2 * i, ((float)(codes[i] & 15) - z) * s);
    store_elem(out, ot, 2 * i + 1, ((float)(codes[i] >> 4) - z) * s);
  }
}

// ------------------------------------------------------------------------------ product
// One wave per (weight row, row of Y): lanes along K in pieces of 32 codes, which lie in one group.
__global__ __launch_bounds__(64) void k_int4_gemv(Int4GemvArgs a) {
  const int lane = threadIdx.x;
  const int64_t No = a.silu ? a.N / 2 : a.N;
  const int64_t n0 = blockIdx.x;
  for (int64_t r = blockIdx.y; r < a.M; r += gridDim.y) {
    int e = 0;
    if (a.offsets) {
      int found = -1;
      for (int i = lane; i < a.E; i += 64) {
        const int lo = min(max(a.offsets[i], 0), (int)a.M), hi = min(max(a.offsets[i + 1], 0), (int)a.M);
        if (r >= lo && r < hi) found = i;
      }
      for (int d = 32; d; d >>= 1) found = max(found, __shfl_xor(found, d, 64));
      if (found < 0) continue;   // a row of no expert: left as it was
      e = found;
    }
    int64_t src = r;
    if (a.offsets) src = min(max(a.row_token ? (int64_t)a.row_token[r] : r, (int64_t)0), a.x_rows - 1);
    float y[2] = {0.f, 0.f};
    for (int p = 0; p < (a.silu ? 2 : 1); ++p) {
      const int64_t n = (int64_t)e * a.N + n0 + p * No;
      float acc = 0.f;
      for (int64_t c = lane; c < a.K / 32; c += 64) {
        const int64_t sg = n * a.groups + 32 * c / a.group;
        const float s = float16_of(a.scales[sg], a.s_type), z = a.zeros ? (float)a.zeros[sg] : 8.f;
        const uint8_t* q = a.codes + (n * a.K + 32 * c) / 2;
        float dot = 0.f;
        for (int j = 0; j < 16; ++j) {
          const int64_t k = src * a.K + 32 * c + 2 * j;
          dot += load_elem(a.X, a.x_type, k) * ((float)(q[j] & 15) - z);
          dot += load_elem(a.X, a.x_type, k + 1) * ((float)(q[j] >> 4) - z);
        }
        acc += s * dot;
      }
      for (int d = 32; d; d >>= 1) acc += __shfl_xor(acc, d, 64);
      y[p] = acc;
    }
    if (lane == 0) store_elem(a.Y, a.y_type, r * No + n0, a.silu ? y[0] / (1.f + expf(-y[0])) * y[1] : y[0]);
  }
}

}  // namespace

hipError_t launch_int4_quantize(const void* W, int w_type, int64_t N, int64_t K, int64_t group, uint8_t* codes,
                                uint16_t* scales, int s_type, uint8_t* zeros, hipStream_t s) {
  const int64_t groups = (K + group - 1) / group;
  const int64_t blocks = std::min<int64_t>((N * groups + kThreads - 1) / kThreads, 1 << 16);
  hipLaunchKernelGGL(k_int4_quantize, dim3((unsigned)blocks), dim3(kThreads), 0, s, W, w_type, N, K, group, groups,
                     codes, scales, s_type, zeros);
  return hipGetLastError();
}

hipError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, int s_type, const uint8_t* zeros,
                                  int64_t N, int64_t K, int64_t group, void* out, int out_type, hipStream_t s) {
  const int64_t groups = (K + group - 1) / group;
  const int64_t blocks = std::min<int64_t>((N * (K / 2) + kThreads - 1) / kThreads, 1 << 16);
  hipLaunchKernelGGL(k_int4_dequantize, dim3((unsigned)blocks), dim3(kThreads), 0, s, codes, scales, s_type, zeros, N,
                     K, group, groups, out, out_type);
  return hipGetLastError();
}

hipError_t launch_int4_gemv(const Int4GemvArgs& a, hipStream_t s) {
  const int64_t No = a.silu ? a.N / 2 : a.N;
  hipLaunchKernelGGL(k_int4_gemv, dim3((unsigned)No, (unsigned)std::min<int64_t>(a.M, 65535)), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssn
