// Shared by the integer 4-bit products (k_int4.hip: up to 16 rows of Y, k_int4_wide.hip: more rows, or a
// longer K).
//
//   W_hat[n, k] = s[n, g] * (q[n, k] - z[n, g]),  g = k / group,   q in 0..15, z = 8 without zero points
//   Y[m, n] = sum_k X[m, k] W_hat[n, k] = sum_g s[n, g] * sum_{k in g} X[m, k] (q[n, k] - z[n, g])
//
// The sum inside a group runs over whole numbers times activations, in f32, and the scale multiplies
// it once: no weight is ever rounded.
//
// A wave walks chunks of 128 k of 16 weight rows: lane l holds row l % 16, k = 32 (l / 16) .. + 31, 16 bytes
// of codes, and v_mfma_f32_16x16x32 multiplies them with the activations as the A operand (lane l: row
// l % 16 of X) in four steps of 8 k per lane. Its result has row 4 (l / 16) + i of X in register i, weight
// row l % 16.
//
// Codes to operand: the bytes w & 0x0F0F0F0F (even k) and (w >> 4) & 0x0F0F0F0F (odd k), read as E4M3,
// stand for q 2^-9 exactly (0..7 are its subnormals, 8..15 its first binade), so one v_cvt_scalef32_pk
// with scale 2^9 turns two of them into whole numbers in bf16 or f16: seven instructions for eight
// codes. The operand's k then runs 0 2 4 6 1 3 5 7, and the activations are put in that order.
//
// The zero point enters after the sum: sum x (q - z) = sum x q - z sum x, with sum x from one more
// matrix instruction per step whose weights are all ones.
//
// A group of a multiple of 128 covers whole chunks (or their part before the end of K), and any order of k
// inside a chunk serves. For finer groups the four dwords of the lanes that share a row are transposed
// first (v_permlane32_swap, v_permlane16_swap), so that step s holds k = 32 s .. + 31, which lie in one
// group, and every FOLD steps (1, or 2 for multiples of 64) are scaled by themselves.
#pragma once
#include "common.hpp"
#include "launch.hpp"
#include "pipeline.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kChunk = 128;                  // k per step of a wave's loop
constexpr uint32_t kOutside = 0x80000000u;   // a byte offset past the end of every buffer resource

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// A resource of `bytes` bytes: loads at offsets past its end give zero and make no traffic.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

template <bool F16X>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F16X)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

template <bool F16X, bool HI>
__device__ __forceinline__ uint32_t codes_pair(uint32_t bytes) {
  if constexpr (F16X)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(bytes, 512.f, HI));
  else
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(bytes, 512.f, HI));
}

// eight codes -> eight whole numbers, k order 0 2 4 6 1 3 5 7
template <bool F16X>
__device__ __forceinline__ u32x4 codes_operand(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  return u32x4{codes_pair<F16X, false>(lo), codes_pair<F16X, true>(lo), codes_pair<F16X, false>(hi),
               codes_pair<F16X, true>(hi)};
}

// the same in natural order: two more instructions, for kernels whose activations serve few codes
template <bool F16X>
__device__ __forceinline__ u32x4 codes_operand_natural(uint32_t w) {
  const uint32_t lo = w & 0x0F0F0F0Fu, hi = (w >> 4) & 0x0F0F0F0Fu;
  const uint32_t a = __builtin_amdgcn_perm(hi, lo, 0x05010400u), b = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
  return u32x4{codes_pair<F16X, false>(a), codes_pair<F16X, true>(a), codes_pair<F16X, false>(b),
               codes_pair<F16X, true>(b)};
}

// eight activations (two per word) in the order 0 2 4 6 1 3 5 7
__device__ __forceinline__ u32x4 x_operand(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x[1], x[0], 0x05040100u), __builtin_amdgcn_perm(x[3], x[2], 0x05040100u),
               __builtin_amdgcn_perm(x[1], x[0], 0x07060302u), __builtin_amdgcn_perm(x[3], x[2], 0x07060302u)};
}

// lane l's dword j and lane group l / 16 change places: out[s] of group g = in[g] of group s
__device__ __forceinline__ u32x4 transpose4(u32x4 v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// the value of lane group s (16 lanes) in every group: out[s]
__device__ __forceinline__ u32x4 spread4(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  return u32x4{b[0], b[1], c[0], c[1]};
}

// the sum of the two halves of the wave (of the two 16-lane groups of each half), in every lane
__device__ __forceinline__ float sum_halves(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_quarters(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// a where the mask's bits are set, else b (v_bfi_b32, where a conditional may become a branch)
__device__ __forceinline__ float choose(uint32_t mask, float a, float b) {
  return __uint_as_float((mask & __float_as_uint(a)) | (~mask & __float_as_uint(b)));
}

// silu(g) = g / (1 + exp(-g)) on the base-2 exponential and the reciprocal of the hardware; exp(-g) = inf
// gives -0, exp(-g) = 0 gives g.
__device__ __forceinline__ float silu(float g) {
  return g * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-g * 1.44269504088896341f));
}

// Inclusive sum over the wave's lanes (row_shr 1, 2, 4, 8 inside the rows of 16 lanes, then row_bcast 15 and
// 31 across them).
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
  return v;
}

// What a workgroup of a grouped product does. The experts' rows, at most `rows` at a time, are slots in
// the experts' order; the grid's workgroups are dealt out evenly to the slots that there are, which only
// the device knows: workgroup b takes part `part` of the `parts` that share its slot. Every wave finds this for itself
// from the offsets, without a barrier; the results are uniform.
struct Slot {
  int e, r0, cnt, part, parts;
};
__device__ __forceinline__ bool find_slot(const int32_t* __restrict__ off, int E, int R, int rows, int max_parts,
                                          Slot& out) {
  constexpr int kBatch = 8;                   // offsets per lane at a time: one round up to 512 experts
  const int lane = threadIdx.x & 63;
  int total = 0, lo[kBatch], hi[kBatch], inc[kBatch];
  auto scan = [&](int e0) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int e = min(e0 + 64 * i + lane, E);
      lo[i] = off[e];
      hi[i] = off[min(e + 1, E)];
    }
    int sum = 0;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      lo[i] = min(max(lo[i], 0), R);
      hi[i] = min(max(hi[i], lo[i]), R);
      inc[i] = sum + wave_scan((hi[i] - lo[i] + rows - 1) / rows);
      sum = __builtin_amdgcn_readlane(inc[i], 63);
    }
    return sum;
  };
  const int rounds = (E + 64 * kBatch - 1) / (64 * kBatch);
  for (int i = 0; i < rounds; ++i) total += scan(64 * kBatch * i);
  if (total == 0) return false;
  out.parts = max(1, min((int)gridDim.x / total, max_parts));
  int slot = blockIdx.x / out.parts;
  out.part = blockIdx.x - slot * out.parts;
  if (slot >= total) return false;
  for (int i = 0; i < rounds; ++i) {
    if (rounds > 1) total = scan(64 * kBatch * i);
    if (slot < total) {
      for (int j = 0; j < kBatch; ++j) {
        const unsigned long long beyond = __ballot(inc[j] > slot);
        if (!beyond) continue;
        const int l = __builtin_ctzll(beyond);
        const int a = __builtin_amdgcn_readlane(lo[j], l), b = __builtin_amdgcn_readlane(hi[j], l);
        const int left = __builtin_amdgcn_readlane(inc[j], l) - slot;   // this slot and the expert's slots behind it
        out.e = 64 * (kBatch * i + j) + l;
        out.r0 = a + rows * ((b - a + rows - 1) / rows - left);
        out.cnt = min(rows, b - out.r0);
        return true;
      }
    }
    slot -= total;
  }
  return false;
}

// steps of 32 k that share a scale: 4 (a whole chunk), 2 or 1
inline int int4_fold(int64_t group) { return group % 128 == 0 ? 4 : group % 64 == 0 ? 2 : 1; }

}  // namespace
}  // namespace ssn
