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

constexpr int kThreads = 256, kUnroll = 4;

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

// 16 values as loaded
template <int T>
struct Sixteen {
  u32x4 v[T == kF32 ? 4 : 2];
};

template <int T>
__device__ __forceinline__ Sixteen<T> load16(const void* p, int64_t i) {
  Sixteen<T> x;
#pragma unroll
  for (int u = 0; u < (int)(sizeof x / 16); ++u) x.v[u] = ((const u32x4*)((const char*)p + i * (T == kF32 ? 4 : 2)))[u];
  return x;
}

// A lane takes one block of a token's keys and the same of its values: all loads of both, the slot's among them, are
// in flight together.
template <int T>
__global__ __launch_bounds__(kThreads) void k_kv_append(KvAppendArgs a) {
  const int nb = a.c.D / 16, per = kThreads / nb;   // blocks of a token, tokens of a workgroup
  const int tl = threadIdx.x / nb, b = threadIdx.x - tl * nb;
  const int64_t t = (int64_t)blockIdx.x * per + tl;
  const int h = blockIdx.y;
  if (tl >= per || t >= a.T) return;
  const Sixteen<T> in[2] = {load16<T>(a.K, t * a.k_token + h * a.k_head + 16 * b),
                            load16<T>(a.V, t * a.v_token + h * a.v_head + 16 * b)};
  const int64_t slot = a.slots[t];
  const float ts[2] = {a.c.k_ts[h], a.c.v_ts[h]};
  int64_t row, vs;
  if (!place(a.c, slot, h, row, vs)) {
    if (a.bad && slot >= 0 && h == 0 && b == 0) atomicAdd((unsigned long long*)a.bad, 1ull);
    return;
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    float w[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      if constexpr (T == kF32) w[e] = __uint_as_float(in[kv].v[e / 4][e % 4]);
      else if constexpr (T == kBF16) w[e] = e & 1 ? bf16_hi(in[kv].v[e / 8][e % 8 / 2]) : bf16_lo(in[kv].v[e / 8][e % 8 / 2]);
      else w[e] = f16_of((uint16_t)(in[kv].v[e / 8][e % 8 / 2] >> (16 * (e & 1))));
    }
    u32x2 code;
    uint32_t S;
    quantize_block(w, (double)ts[kv], code, S);
    *(u32x2*)((kv ? a.c.v_codes : a.c.k_codes) + row * (a.c.D / 2) + 8 * b) = code;
    if (kv) a.c.v_scales[vs + (int64_t)b * a.c.page] = (uint8_t)S;
    else a.c.k_scales[row * nb + b] = (uint8_t)S;
  }
}

// Eight values of a token's keys and of its values a lane, for U tokens at once: four bytes of codes in, 16 or 32 bytes
// out, each.
template <int T, int U, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvReadArgs a) {
  const int n8 = a.c.D / 8, per = kThreads / n8;
  const int tl = threadIdx.x / n8, b = threadIdx.x - tl * n8;
  const int64_t t0 = (int64_t)blockIdx.x * (per * U) + tl;
  const int h = blockIdx.y;
  if (tl >= per || t0 >= a.T) return;
  const float ts[2] = {a.c.k_ts[h], a.c.v_ts[h]};
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) slot[u] = t0 + u * per < a.T ? a.slots[t0 + u * per] : -1;
  uint32_t code[U][2], S[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    int64_t row, vs;
    code[u][0] = code[u][1] = S[u][0] = S[u][1] = 0;
    if (place(a.c, slot[u], h, row, vs)) {
      code[u][0] = *(const uint32_t*)(a.c.k_codes + row * (a.c.D / 2) + 4 * b);
      code[u][1] = *(const uint32_t*)(a.c.v_codes + row * (a.c.D / 2) + 4 * b);
      S[u][0] = a.c.k_scales[row * (a.c.D / 16) + b / 2];
      S[u][1] = a.c.v_scales[vs + (int64_t)(b / 2) * a.c.page];
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t0 + u * per >= a.T) return;
    const int64_t o = ((t0 + u * per) * a.c.heads + h) * a.c.D + 8 * b;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t w = code[u][kv];
      const float s = e4m3_f32(S[u][kv]);
      const f32x2 p[4] = {fp4x2_f32<0>(w), fp4x2_f32<1>(w), fp4x2_f32<2>(w), fp4x2_f32<3>(w)};
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = (p[e / 2][e & 1] * s) * ts[kv];   // E2M1 * E4M3 is exact, then one rounding
      u32x4 r[T == kF32 ? 2 : 1];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (T == kF32) r[e / 4][e % 4] = __float_as_uint(v[e]);
        else if (e % 2 == 0)
          r[0][e / 2] = T == kBF16 ? pk_bf16_rne(v[e], v[e + 1]) : (uint32_t)to_f16(v[e]) | (uint32_t)to_f16(v[e + 1]) << 16;
      }
      u32x4* dst = (u32x4*)((char*)(kv ? a.V : a.K) + o * (T == kF32 ? 4 : 2));
#pragma unroll
      for (int x = 0; x < (int)(sizeof r / 16); ++x) {
        if constexpr (STREAM) __builtin_nontemporal_store(r[x], dst + x);
        else dst[x] = r[x];
      }
    }
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
  const dim3 grid((unsigned)((a.T + per - 1) / per), (unsigned)a.c.heads);
  return by_type(a, [&](auto t) { hipLaunchKernelGGL((k_kv_append<decltype(t)::value>), grid, dim3(kThreads), 0, s, a); });
}

// Keys and values that together pass kStream bytes are written past the caches.
constexpr int64_t kStream = (int64_t)128 << 20;
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int per = kThreads / (a.c.D / 8);
  const bool stream = 2 * a.T * a.c.heads * a.c.D * (a.type == kF32 ? 4 : 2) >= kStream;
  // few tokens: one a lane, so that more workgroups share them
  const int U = a.T * a.c.heads / per >= 8 * 256 ? kUnroll : 1;
  const dim3 grid((unsigned)((a.T + per * U - 1) / (per * U)), (unsigned)a.c.heads);
  return by_type(a, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (stream) hipLaunchKernelGGL((k_kv_read<T, kUnroll, true>), dim3((unsigned)((a.T + per * kUnroll - 1) / (per * kUnroll)), (unsigned)a.c.heads), dim3(kThreads), 0, s, a);
    else if (U > 1) hipLaunchKernelGGL((k_kv_read<T, kUnroll, false>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_kv_read<T, 1, false>), grid, dim3(kThreads), 0, s, a);
  });
}

}  // namespace ssn
