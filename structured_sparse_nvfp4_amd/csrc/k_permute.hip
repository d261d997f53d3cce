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
// eight L2s. WT waves share a token (as many as its row has 512 elements, at most four), a lane moves eight
// elements at a time (four where f32 rows are only written), and the slots' rows are fetched kBatch together.
// Lane j of a wave loads slot j's row number and weight, once per token: loaded by the slot's turn, each batch
// waited for them (8 tokens x 10, D = 2048: permute 4.0 against 3.2 us, 4096 tokens unpermute 41.5 against
// 38.1). Rows need not be aligned: the memory system takes 16-byte accesses at any element. 4096 tokens x 10,
// D = 2048, bf16: permute 38 us, 4.8 TB/s, where a large copy reaches 5.0.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256;

// V elements, packed as they lie in memory
template <int T, int V>
struct Vec {
  u32x4 w[T == kF32 ? V / 4 : 1];
};

// the first n of them (all V if n >= V) at element i of p, which is aligned to one element
template <int T, int V>
__device__ __forceinline__ Vec<T, V> load_vec(const void* p, int64_t i, int n) {
  Vec<T, V> v = {};
  if (n >= V) {
    __builtin_memcpy(&v, (const char*)p + i * (T == kF32 ? 4 : 2), sizeof v);
  } else {
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
      if (j < n) {
        if constexpr (T == kF32) v.w[j / 4][j % 4] = ((const uint32_t*)p)[i + j];
        else v.w[0][j / 2] |= (uint32_t)((const uint16_t*)p)[i + j] << (16 * (j & 1));
      }
  }
  return v;
}

// STREAM: past the caches
template <int T, int V, bool STREAM>
__device__ __forceinline__ void store_vec(void* p, int64_t i, int n, const Vec<T, V>& v) {
  if (n >= V) {
    if constexpr (STREAM) {
      typedef u32x4 __attribute__((aligned(2))) loose;
#pragma unroll
      for (int j = 0; j < (int)(sizeof v / 16); ++j)
        __builtin_nontemporal_store(v.w[j], (loose*)((char*)p + i * (T == kF32 ? 4 : 2)) + j);
    } else {
      __builtin_memcpy((char*)p + i * (T == kF32 ? 4 : 2), &v, sizeof v);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V - 1; ++j)
      if (j < n) {
        if constexpr (T == kF32) ((uint32_t*)p)[i + j] = v.w[j / 4][j % 4];
        else ((uint16_t*)p)[i + j] = (uint16_t)(v.w[0][j / 2] >> (16 * (j & 1)));
      }
  }
}

template <int T, int V>
__device__ __forceinline__ float to_f32(const Vec<T, V>& v, int j) {
  if constexpr (T == kF32) return __uint_as_float(v.w[j / 4][j % 4]);
  const uint32_t w = v.w[0][j / 2];
  if constexpr (T == kBF16) return j & 1 ? bf16_hi(w) : bf16_lo(w);
  return f16_of((uint16_t)(j & 1 ? w >> 16 : w));
}

// two values into elements j and j + 1 (j even)
template <int T, int V>
__device__ __forceinline__ void from_f32(Vec<T, V>& v, int j, float lo, float hi) {
  if constexpr (T == kF32) {
    v.w[j / 4][j % 4] = __float_as_uint(lo);
    v.w[j / 4][j % 4 + 1] = __float_as_uint(hi);
  } else if constexpr (T == kBF16) {
    v.w[0][j / 2] = pk_bf16_rne(lo, hi);
  } else {
    v.w[0][j / 2] = (uint32_t)to_f16(lo) | (uint32_t)to_f16(hi) << 16;
  }
}

// The sums of four values over the wave's lanes, one in the last lane of each 16: of v[0], v[2], v[1], v[3]
// (halves of the wave and then of each half change places, so that one addition serves two values).
__device__ __forceinline__ float wave_sums(const float* v) {
  auto swapped = [](bool half, float x, float y) {
    const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
    const auto r = half ? __builtin_amdgcn_permlane32_swap(a, b, false, false) : __builtin_amdgcn_permlane16_swap(a, b, false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  float s = swapped(false, swapped(true, v[0], v[1]), swapped(true, v[2], v[3]));
  auto add = [&](int moved) { s += __int_as_float(moved); };
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x111, 0xF, 0xF, false));   // row_shr 1, 2, 4, 8
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x112, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x114, 0xF, 0xF, false));
  add(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x118, 0xF, 0xF, false));
  return s;
}

// Both movements. AT, BT: types of the token and the row side; WT: waves per token; DOT: dw too; STREAM: rows
// are written past the caches.
template <bool GATHER, int AT, int BT, int WT, bool DOT, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_permute(PermuteArgs a) {
  // Rows under way together. 4, 8 and 16 of 16 bits (4096 tokens x 10, D = 2048, bf16): unpermute 38.1, 38.4,
  // 38.8 us, with dw 76.4, 80.8, 88.7 (permute 38 each); 4 of f32 (2048 x 8, D = 4096) 122.7 against 120.1 us.
  constexpr int kBatch = BT == kF32 ? 8 : 4;
  // Elements a lane moves at a time. Eight of f32 are two accesses that leave every other 16 bytes to each other:
  // stores alone run better as whole lines (that f32 permute 63.4 against 72.4 us), loads better in eights
  // (unpermute 62.1 against 63.1 us, its gradient with dw 120.1 against 126.1).
  constexpr int kVec = AT == kF32 && BT == kF32 && !GATHER && !DOT ? 4 : 8;
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
    // lane j has slot j's row, -1 for none, and weight
    int own_row = -1;
    float own_w = 1.f;
    if (live && lane < k) {
      own_row = a.row_of[t * k + lane];
      if (own_row >= a.R) own_row = -1;
      if (a.w) own_w = a.w[t * k + lane];
    }
    if (live)
      for (int d = kVec * (64 * part + lane); d - kVec * lane < D; d += kVec * 64 * WT) {
        // The row's last kVec elements, where so many no longer follow: the lane before has the first `twice`
        // of them too, and computes the same. Rows under kVec elements go element by element.
        const bool in = d < D;
        const int at = max(0, min(d, D - kVec)), n = min(D, kVec), twice = d - at;
        Vec<AT, kVec> av = {};
        if ((!GATHER || DOT) && in) av = load_vec<AT, kVec>(a.A, t * D + at, n);
        float sum[kVec] = {};
        for (int j0 = 0; j0 < k; j0 += kBatch) {
          int row[kBatch];
          float w[kBatch];
          Vec<BT, kVec> bv[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            row[i] = j0 + i < k ? __builtin_amdgcn_readlane(own_row, (j0 + i) & 63) : -1;
            w[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(own_w), (j0 + i) & 63));
          }
          if (GATHER || DOT)
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (row[i] >= 0 && in) bv[i] = load_vec<BT, kVec>(a.B, (int64_t)row[i] * D + at, n);
          float dot[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            dot[i] = 0.f;
            if (row[i] < 0) continue;           // no row: nothing moves, dw stays 0
            if (in) {
              if constexpr (GATHER) {
#pragma unroll
                for (int q = 0; q < kVec; ++q) sum[q] = __builtin_fmaf(w[i], to_f32(bv[i], q), sum[q]);
              } else {
                Vec<BT, kVec> out;
                if (AT == BT && !a.w) {         // a copy: every bit as it is
                  __builtin_memcpy(&out, &av, sizeof out);
                } else {
#pragma unroll
                  for (int q = 0; q < kVec; q += 2) from_f32(out, q, w[i] * to_f32(av, q), w[i] * to_f32(av, q + 1));
                }
                store_vec<BT, kVec, STREAM>(a.B_out, (int64_t)row[i] * D + at, n, out);
              }
              if (DOT)
#pragma unroll
                for (int q = 0; q < kVec; ++q)
                  if (q >= twice) dot[i] = __builtin_fmaf(to_f32(av, q), to_f32(bv[i], q), dot[i]);
            }
          }
          if (DOT)
#pragma unroll
            for (int i = 0; i < kBatch; i += 4) {
              const float s = wave_sums(dot + i);
              const int j = j0 + i + (lane >> 5 | (lane >> 4 & 1) << 1);
              if (lane % 16 == 15 && j < k) dots[wave][j] += s;
            }
        }
        if (GATHER && in) {
          Vec<AT, kVec> out;
#pragma unroll
          for (int q = 0; q < kVec; q += 2) from_f32(out, q, sum[q], sum[q + 1]);
          store_vec<AT, kVec, false>(a.A_out, t * D + at, n, out);
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

template <bool GATHER, int AT, int BT, bool DOT, bool STREAM>
hipError_t launch_wt(const PermuteArgs& a, hipStream_t s) {
  const int wt = a.D <= 512 ? 1 : a.D <= 1024 ? 2 : 4;
  const int64_t tokens = kThreads / 64 / wt, blocks = (a.T + tokens - 1) / tokens;
  const dim3 grid((unsigned)std::min<int64_t>(blocks, 1 << 22));
  const auto kernel = wt == 1 ? k_permute<GATHER, AT, BT, 1, DOT, STREAM>
                              : wt == 2 ? k_permute<GATHER, AT, BT, 2, DOT, STREAM> : k_permute<GATHER, AT, BT, 4, DOT, STREAM>;
  hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

// Rows that the 256 MB cache does not hold are written past it: 2048 x 8, D = 4096, f32 (268 MB) 53.5 against
// 63.5 us, 4096 x 10, D = 2048, f32 (336 MB) with the unpermute that reads them 143 against 174 us. Fewer are
// better found there: bf16 (168 MB) with the unpermute 73.5 against 65.0 us. With dw as many are read, and that
// f32 gradient took 128.7 against 119.7 us.
template <bool GATHER, int AT, int BT, bool DOT>
hipError_t launch_stream(const PermuteArgs& a, hipStream_t s) {
  if constexpr (!GATHER && !DOT)
    if (std::min(a.R, a.T * a.k) * a.D >= ((int64_t)256 << 20) / (BT == kF32 ? 4 : 2)) return launch_wt<GATHER, AT, BT, DOT, true>(a, s);
  return launch_wt<GATHER, AT, BT, DOT, false>(a, s);
}

template <bool GATHER, int AT, int BT>
hipError_t launch_dot(const PermuteArgs& a, hipStream_t s) {
  return a.dw ? launch_stream<GATHER, AT, BT, true>(a, s) : launch_stream<GATHER, AT, BT, false>(a, s);
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
