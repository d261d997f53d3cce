// The 4-bit cache of keys and values: quantised as it is written, and read back.
//
// A block of 16 values along a head's width is quantised by the rule of nvfp4_quantize with a given tensor scale
// (the head's): S = E4M3(amax / (6 s_h)), code = E2M1(x / (s_h S)), every decision exact (nvfp4_block.hpp); read
// back it is E2M1(code) E4M3(S) s_h, the f32 product rounded once to f32 and from there to a 16-bit type.
//
// Both kernels move each value once and are bound by memory. A workgroup takes tokens of one head, keys or
// values, and its lanes lie along a token's blocks first: the rows it reads are runs of 2 D or 4 D bytes, and the
// values' scales, whose tokens are innermost, come together where the slots of consecutive tokens are consecutive.
#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "nvfp4_block.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256;

// where a slot's token lies in a head of the cache; false if it has none
__device__ __forceinline__ bool place(const KvCache& c, int64_t slot, int h, int64_t& row, int64_t& vscale) {
  if (slot < 0) return false;
  const int64_t p = slot / c.page;
  if (p >= c.pages) return false;
  const int64_t o = slot - p * c.page, head = p * c.heads + h;
  row = head * c.page + o;                          // of codes and the keys' scales
  vscale = head * (c.D / 16) * c.page + o;          // of the values' scales, a step of `page` to the next block
  return true;
}

__global__ void k_kv_clear(int64_t* bad) { *bad = 0; }

template <int T>
__global__ __launch_bounds__(kThreads) void k_kv_append(KvAppendArgs a) {
  const int nb = a.c.D / 16, per = kThreads / nb;   // blocks of a token, tokens of a workgroup
  const int tl = threadIdx.x / nb, b = threadIdx.x - tl * nb;
  const int64_t t = (int64_t)blockIdx.x * per + tl;
  const int h = blockIdx.y, values = blockIdx.z;
  if (tl >= per || t >= a.T) return;
  const int64_t slot = a.slots[t];
  int64_t row, vs;
  if (!place(a.c, slot, h, row, vs)) {
    if (a.bad && slot >= 0 && h == 0 && b == 0 && !values) atomicAdd((unsigned long long*)a.bad, 1ull);
    return;
  }
  const int64_t i = (values ? t * a.v_token + h * a.v_head : t * a.k_token + h * a.k_head) + 16 * b;
  const void* src = values ? a.V : a.K;
  float w[16];
  if constexpr (T == kF32) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const f32x4 v = ((const f32x4*)((const float*)src + i))[u];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[4 * u + e] = v[e];
    }
  } else {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x4 v = ((const u32x4*)((const uint16_t*)src + i))[u];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint16_t x = (uint16_t)(v[e / 2] >> (16 * (e & 1)));
        w[8 * u + e] = T == kF16 ? f16_of(x) : bf16_of(x);
      }
    }
  }
  u32x2 code;
  uint32_t S;
  quantize_block(w, (double)(values ? a.c.v_ts : a.c.k_ts)[h], code, S);
  if (values) {
    *(u32x2*)(a.c.v_codes + row * (a.c.D / 2) + 8 * b) = code;
    a.c.v_scales[vs + (int64_t)b * a.c.page] = (uint8_t)S;
  } else {
    *(u32x2*)(a.c.k_codes + row * (a.c.D / 2) + 8 * b) = code;
    a.c.k_scales[row * nb + b] = (uint8_t)S;
  }
}

// eight values a lane: four bytes of codes, 16 or 32 bytes out
template <int T>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvReadArgs a) {
  const int n8 = a.c.D / 8, per = kThreads / n8;
  const int tl = threadIdx.x / n8, b = threadIdx.x - tl * n8;
  const int64_t t = (int64_t)blockIdx.x * per + tl;
  const int h = blockIdx.y, values = blockIdx.z;
  if (tl >= per || t >= a.T) return;
  int64_t row, vs;
  float v[8] = {};
  if (place(a.c, a.slots[t], h, row, vs)) {
    const uint32_t w = *(const uint32_t*)((values ? a.c.v_codes : a.c.k_codes) + row * (a.c.D / 2) + 4 * b);
    const float S = e4m3_f32(values ? a.c.v_scales[vs + (int64_t)(b / 2) * a.c.page] : a.c.k_scales[row * (a.c.D / 16) + b / 2]);
    const float ts = (values ? a.c.v_ts : a.c.k_ts)[h];
    const f32x2 p[4] = {fp4x2_f32<0>(w), fp4x2_f32<1>(w), fp4x2_f32<2>(w), fp4x2_f32<3>(w)};
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (p[e / 2][e & 1] * S) * ts;     // E2M1 * E4M3 is exact, then one rounding
  }
  const int64_t o = (t * a.c.heads + h) * a.c.D + 8 * b;
  void* dst = values ? a.V : a.K;
  if constexpr (T == kF32) {
    ((f32x4*)((float*)dst + o))[0] = f32x4{v[0], v[1], v[2], v[3]};
    ((f32x4*)((float*)dst + o))[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 r;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      r[u] = T == kBF16 ? pk_bf16_rne(v[2 * u], v[2 * u + 1])
                        : (uint32_t)to_f16(v[2 * u]) | (uint32_t)to_f16(v[2 * u + 1]) << 16;
    *(u32x4*)((uint16_t*)dst + o) = r;
  }
}

template <typename A, typename F>
hipError_t by_type(const A& a, F&& launch) {
  if (a.type == kF32) launch(std::integral_constant<int, kF32>());
  else if (a.type == kBF16) launch(std::integral_constant<int, kBF16>());
  else launch(std::integral_constant<int, kF16>());
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s) {
  if (a.bad) hipLaunchKernelGGL(k_kv_clear, dim3(1), dim3(1), 0, s, a.bad);
  if (a.T == 0) return hipGetLastError();
  const int per = kThreads / (a.c.D / 16);
  const dim3 grid((unsigned)((a.T + per - 1) / per), (unsigned)a.c.heads, 2);
  return by_type(a, [&](auto t) { hipLaunchKernelGGL((k_kv_append<decltype(t)::value>), grid, dim3(kThreads), 0, s, a); });
}

hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int per = kThreads / (a.c.D / 8);
  const dim3 grid((unsigned)((a.T + per - 1) / per), (unsigned)a.c.heads, 2);
  return by_type(a, [&](auto t) { hipLaunchKernelGGL((k_kv_read<decltype(t)::value>), grid, dim3(kThreads), 0, s, a); });
}

}  // namespace ssn
