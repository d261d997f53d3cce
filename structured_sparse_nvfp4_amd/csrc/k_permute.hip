// Tokens to expert order and back, with the routing weights applied, and the gradients of both.
//
// Entry f = t k + j of a routing (token t, slot j) owns row row_of[f] of the expert-ordered rows, or none
// (a value outside [0, R)). With w(f) the entry's weight (1 without weights), A the token side [T, D] and B
// the row side [R, D], all four calls are one of two movements:
//   scatter  B[row(f)] = w(f) A[t]                    permute, and unpermute's gradient (A = dout)
//   gather   A[t] = sum_j w(f) B[row(f)]              unpermute, and permute's gradient (B = dXp)
// and the weights' gradient of either is dw(f) = <A'[t], B'[row(f)]>, with the forward's input on one side
// and the incoming gradient on the other. Sums run in f32 in slot order.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256;

// Sum over the block's threads (every thread gets it).
__device__ __forceinline__ float block_sum(float v) {
  __shared__ float part[kThreads / 64];
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kThreads / 64; ++i) s += part[i];
  return s;
}

// One block per token.
__global__ __launch_bounds__(kThreads) void k_moe_scatter(PermuteArgs a) {
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x)
    for (int j = 0; j < a.k; ++j) {
      const int64_t f = t * a.k + j, r = a.row_of[f];
      const bool has = r >= 0 && r < a.R;
      const float w = a.w ? a.w[f] : 1.f;
      float dot = 0.f;
      if (has)
        for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
          const float v = load_elem(a.A, a.a_type, t * a.D + d);
          if (a.w || a.a_type != a.b_type) store_elem(a.B_out, a.b_type, r * a.D + d, a.w ? w * v : v);
          else if (a.a_type == kF32) ((uint32_t*)a.B_out)[r * a.D + d] = ((const uint32_t*)a.A)[t * a.D + d];
          else ((uint16_t*)a.B_out)[r * a.D + d] = ((const uint16_t*)a.A)[t * a.D + d];
          if (a.dw) dot += v * load_elem(a.B, a.b_type, r * a.D + d);
        }
      if (a.dw) {
        dot = block_sum(dot);
        if (threadIdx.x == 0) a.dw[f] = dot;
      }
    }
}

__global__ __launch_bounds__(kThreads) void k_moe_gather(PermuteArgs a) {
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      float acc = 0.f;
      for (int j = 0; j < a.k; ++j) {
        const int64_t f = t * a.k + j, r = a.row_of[f];
        if (r >= 0 && r < a.R) {
          acc = __builtin_fmaf(a.w ? a.w[f] : 1.f, load_elem(a.B, a.b_type, r * a.D + d), acc);
        }
      }
      store_elem(a.A_out, a.a_type, t * a.D + d, acc);
    }
    if (a.dw)
      for (int j = 0; j < a.k; ++j) {
        const int64_t f = t * a.k + j, r = a.row_of[f];
        float dot = 0.f;
        if (r >= 0 && r < a.R)
          for (int64_t d = threadIdx.x; d < a.D; d += kThreads)
            dot += load_elem(a.A, a.a_type, t * a.D + d) * load_elem(a.B, a.b_type, r * a.D + d);
        dot = block_sum(dot);
        if (threadIdx.x == 0) a.dw[f] = dot;
      }
  }
}

}  // namespace

hipError_t launch_moe_scatter(const PermuteArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_moe_scatter, dim3((unsigned)std::min<int64_t>(a.T, 1 << 20)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_moe_gather(const PermuteArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_moe_gather, dim3((unsigned)std::min<int64_t>(a.T, 1 << 20)), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace ssn
