// Tokens to expert order and back, with the routing weights applied, and the gradients of both.
//
// Entry f = t k + j of a routing (token t, slot j) owns row row_of[f] of the expert-ordered rows, or none
// (a value outside [0, R)). With w(f) the entry's weight (1 without weights), A the token side [T, D] and B
// the row side [R, D], all four calls are one of two movements:
//   scatter  B[row(f)] = w(f) A[t]                    permute, and unpermute's gradient (A = dout)
//   gather   A[t] = sum_j w(f) B[row(f)]              unpermute, and permute's gradient (B = dXp)
// and the weights' gradient of either is dw(f) = <A'[t], B'[row(f)]>, with the forward's input on one side
// and the incoming gradient on the other: it needs only the rows that the movement reads anyway, or one
// more read beside its writes, and is taken in the same pass. Sums run in f32 in slot order.
//
// Memory-bound: the token side moves once and the row side once. So the work is cut along the tokens, where
// a token's row is read once for all its slots, and not along the rows, which would read it k times through
// eight L2s. WT waves share a token (as many as its row has 512 elements, at most four), a lane moves
// eight elements at a time, and the slots' rows are fetched kBatch together. Rows need not be aligned: the
// memory system takes 16-byte accesses at any element, and only a row's last D % 8 elements go singly.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256, kVec = 8;

template <int T>
struct Elem {
  using Word = uint16_t;
};
template <>
struct Elem<kF32> {
  using Word = float;
};

// eight elements at a pointer aligned to one
template <int T>
struct Vec {
  typename Elem<T>::Word e[kVec];
};

template <int T>
__device__ __forceinline__ Vec<T> load_vec(const void* p, int64_t i, int n) {
  Vec<T> v;
  const auto* q = (const typename Elem<T>::Word*)p + i;
  if (n >= kVec) {
    __builtin_memcpy(&v, q, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) v.e[j] = j < n ? q[j] : (typename Elem<T>::Word)0;
  }
  return v;
}

template <int T>
__device__ __forceinline__ void store_vec(void* p, int64_t i, int n, const Vec<T>& v) {
  auto* q = (typename Elem<T>::Word*)p + i;
  if (n >= kVec) {
    __builtin_memcpy(q, &v, sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j < n) q[j] = v.e[j];
  }
}

template <int T>
__device__ __forceinline__ float to_f32(const Vec<T>& v, int j) {
  if constexpr (T == kF32) return v.e[j];
  else return float16_of(v.e[j], T);
}

template <int T>
__device__ __forceinline__ void from_f32(Vec<T>& v, int j, float f) {
  if constexpr (T == kF32) v.e[j] = f;
  else v.e[j] = T == kF16 ? to_f16(f) : to_bf16(f);
}

// the sum of the wave's lanes, in lane 63
__device__ __forceinline__ float wave_sum_last(float v) {
  auto add = [&](int moved) { v += __int_as_float(moved); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x112, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x114, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x118, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));   // row_bcast 15, 31
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
  return v;
}

// Both movements. AT, BT: types of the token and the row side; WT: waves per token; DOT: dw too.
template <bool GATHER, int AT, int BT, int WT, bool DOT>
__global__ __launch_bounds__(kThreads) void k_permute(PermuteArgs a) {
  constexpr int kBatch = BT == kF32 || (DOT && AT == kF32) ? 8 : 16;   // rows under way together
  constexpr int kTokens = kThreads / (64 * WT);                        // per workgroup
  constexpr int kMaxSlots = 64;
  __shared__ float dots[DOT ? kThreads / 64 : 1][DOT ? kMaxSlots : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, part = wave % WT;
  const int k = a.k, D = (int)a.D;
  for (int64_t t0 = (int64_t)blockIdx.x * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * kTokens) {
    const int64_t t = t0 + wave / WT;
    const bool live = t < a.T;                  // uniform in a wave; all waves meet at the barriers
    if (DOT)
      for (int j = lane; j < k; j += 64) dots[wave][j] = 0.f;
    if (live)
      for (int d = kVec * (64 * part + lane); d - kVec * lane < D; d += kVec * 64 * WT) {
        const int n = D - d;                    // elements left; lanes past the end have none
        Vec<AT> av = {};
        if ((!GATHER || DOT) && n > 0) av = load_vec<AT>(a.A, t * D + d, n);
        float sum[kVec] = {};
        for (int j0 = 0; j0 < k; j0 += kBatch) {
          int row[kBatch];
          float w[kBatch];
          Vec<BT> bv[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const int64_t f = t * k + min(j0 + i, k - 1);
            row[i] = __builtin_amdgcn_readfirstlane(a.row_of[f]);
            if (j0 + i >= k || row[i] >= a.R) row[i] = -1;
            w[i] = a.w ? a.w[f] : 1.f;
          }
          if (GATHER || DOT)
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (row[i] >= 0 && n > 0) bv[i] = load_vec<BT>(a.B, (int64_t)row[i] * D + d, n);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (row[i] < 0) continue;           // no row: nothing moves, dw stays 0
            float dot = 0.f;
            if (n > 0) {
              if constexpr (GATHER) {
#pragma unroll
                for (int q = 0; q < kVec; ++q) sum[q] = __builtin_fmaf(w[i], to_f32(bv[i], q), sum[q]);
              } else {
                Vec<BT> out;
                if (AT == BT && !a.w) {         // a copy: every bit as it is
                  __builtin_memcpy(&out, &av, sizeof out);
                } else {
#pragma unroll
                  for (int q = 0; q < kVec; ++q) from_f32(out, q, w[i] * to_f32(av, q));
                }
                store_vec<BT>(a.B_out, (int64_t)row[i] * D + d, n, out);
              }
              if (DOT)
#pragma unroll
                for (int q = 0; q < kVec; ++q) dot = __builtin_fmaf(to_f32(av, q), to_f32(bv[i], q), dot);
            }
            if (DOT) {
              dot = wave_sum_last(dot);
              if (lane == 63) dots[wave][j0 + i] += dot;
            }
          }
        }
        if (GATHER && n > 0) {
          Vec<AT> out;
#pragma unroll
          for (int q = 0; q < kVec; ++q) from_f32(out, q, sum[q]);
          store_vec<AT>(a.A_out, t * D + d, n, out);
        }
      }
    if constexpr (DOT) {
      __syncthreads();
      if (live && part == 0)
        for (int j = lane; j < k; j += 64) {
          float s = 0.f;
#pragma unroll
          for (int p = 0; p < WT; ++p) s += dots[wave + p][j];
          a.dw[t * k + j] = s;
        }
      __syncthreads();
    }
  }
}

template <bool GATHER, int AT, int BT, bool DOT>
hipError_t launch_wt(const PermuteArgs& a, hipStream_t s) {
  const int wt = a.D <= 512 ? 1 : a.D <= 1024 ? 2 : 4;
  const int64_t tokens = kThreads / 64 / wt, blocks = (a.T + tokens - 1) / tokens;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 22));
  if (wt == 1) hipLaunchKernelGGL((k_permute<GATHER, AT, BT, 1, DOT>), grid, dim3(kThreads), 0, s, a);
  else if (wt == 2) hipLaunchKernelGGL((k_permute<GATHER, AT, BT, 2, DOT>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_permute<GATHER, AT, BT, 4, DOT>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <bool GATHER, int AT, int BT>
hipError_t launch_dot(const PermuteArgs& a, hipStream_t s) {
  return a.dw ? launch_wt<GATHER, AT, BT, true>(a, s) : launch_wt<GATHER, AT, BT, false>(a, s);
}

template <bool GATHER>
hipError_t launch_types(const PermuteArgs& a, hipStream_t s) {
  if (a.a_type == kF32) {
    if (a.b_type == kF32) return launch_dot<GATHER, kF32, kF32>(a, s);
    return a.b_type == kF16 ? launch_dot<GATHER, kF32, kF16>(a, s) : launch_dot<GATHER, kF32, kBF16>(a, s);
  }
  return a.a_type == kF16 ? launch_dot<GATHER, kF16, kF16>(a, s) : launch_dot<GATHER, kBF16, kBF16>(a, s);
}

}  // namespace

hipError_t launch_moe_scatter(const PermuteArgs& a, hipStream_t s) { return launch_types<false>(a, s); }
hipError_t launch_moe_gather(const PermuteArgs& a, hipStream_t s) { return launch_types<true>(a, s); }

}  // namespace ssn
