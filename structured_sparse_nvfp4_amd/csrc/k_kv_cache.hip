// The 4-bit cache of keys and values: quantised as it is written, and read back.
//
// A block of 16 values along a head's width is quantised by the rule of nvfp4_quantize with a given tensor scale
// (the head's): S = E4M3(amax / (6 s_h)), code = E2M1(x / (s_h S)), every decision exact (nvfp4_block.hpp); read
// back it is E2M1(code) E4M3(S) s_h, the f32 product rounded once to f32 and from there to a 16-bit type.
//
// Both kernels move each value once: 8192 tokens x 8 heads x 128 of bf16 written in 10.7 us (43 MB, 4.0 TB/s, the start and
// two dependent reads 3 of it; 395 vector instructions for 64 blocks a wave issue 0.76 of the time), read in 9.3 (4.6
// TB/s); 65536 read in 51 (344 MB, 6.8 TB/s); 8 written in 3.4 and read in 2.7. A workgroup takes tokens of one head, keys or
// values, and its lanes lie along a token's blocks first: the rows it reads are runs of 2 D or 4 D bytes, and the
// values' scales, whose tokens are innermost, come together where the slots of consecutive tokens are consecutive.
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "nvfp4_block.hpp"
#include "types.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256, kUnroll = 4;

// slot / page by a multiplication: exact for slots up to 2^44 and pages up to 2^20, since m page - 2^64 < page
struct Slots {
  uint64_t m;
  int64_t end;                                     // slots of the cache
};
Slots slots_of(const KvCache& c) { return {~(uint64_t)0 / (uint64_t)c.page + 1, c.pages * c.page}; }

// where a slot's token lies in a head of the cache; false if it has none
__device__ __forceinline__ bool place(const KvCache& c, const Slots& s, int64_t slot, int h, int64_t& row, int64_t& vscale) {
  if (slot < 0 || slot >= s.end) return false;
  const int64_t p = (int64_t)__umul64hi((uint64_t)slot, s.m);
  const int64_t o = slot - p * c.page, head = p * c.heads + h;
  row = head * c.page + o;                          // of codes and the keys' scales
  vscale = head * (c.D / 16) * c.page + o;          // of the values' scales, a step of `page` to the next block
  return true;
}

__global__ void k_kv_clear(int64_t* bad) { *bad = 0; }

// S and the codes of one block on the conversion instructions, where that can be told to be exact. The quotients
// amax / (6 s_h) and x / (s_h S) are formed in f32 as a lower and an upper bound: a reciprocal or a rounded constant, a
// rounded scale and two products are off by less than 2^-21 together, and the bounds are 2^-20 apart from the middle.
// Rounding is monotone, so where both bounds round to one value the quotient does too (both are converted by one
// instruction, a pair of scales or two pairs of codes). False where they differ (a quotient next to the middle of two
// values: one block in some ten thousand, unless s_h is a power of two and x has few bits), where a value is not
// finite, and for scales so small or large that f32 would not hold the bounds. The exact rule then takes over: 15.9 us
// with it alone, 10.7 with this, for 8192 tokens x 8 heads x 128 of bf16.
__device__ __forceinline__ bool quantize_bounds(const float (&w)[16], float st, u32x2& code, uint32_t& S) {
  constexpr float kUp = 1.f + 0x1p-20f, kDown = 1.f - 0x1p-20f;
  float amax = 0.f, finite = 0.f;
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    amax = fmaxf(amax, fabsf(w[t]));
    finite = fmaf(w[t], 0.f, finite);              // 0, or NaN
  }
  const float q = amax * (1.f / (6.f * st));
  const uint32_t two = __builtin_amdgcn_cvt_pk_fp8_f32(fminf(q * kDown, 448.f), fminf(q * kUp, 448.f), 0, false);
  S = two & 0xFFu;
  const float d = st * e4m3_f32(S), inv = __builtin_amdgcn_rcpf(d), down = inv * kDown, up = inv * kUp, most = 7.f * d;
  uint32_t lo[2] = {0, 0}, hi[2] = {0, 0};
  auto convert = [&](auto sel) {                   // the four words in turn: each conversion writes a byte of its own
    constexpr int s = decltype(sel)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float a = __builtin_amdgcn_fmed3f(w[8 * h + 2 * s], -most, most), b = __builtin_amdgcn_fmed3f(w[8 * h + 2 * s + 1], -most, most);
      lo[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo[h], a * down, b * down, 1.f, s);
      hi[h] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(hi[h], a * up, b * up, 1.f, s);
    }
  };
  convert(std::integral_constant<int, 0>());
  convert(std::integral_constant<int, 1>());
  convert(std::integral_constant<int, 2>());
  convert(std::integral_constant<int, 3>());
  const bool zero = S == 0;                        // a block whose scale is zero stores code 0x0
  code[0] = zero ? 0u : lo[0];
  code[1] = zero ? 0u : lo[1];
  const bool same = zero || (lo[0] == hi[0] && lo[1] == hi[1]);
  return st > 1e-30f && st < 1e30f && finite == 0.f && S == two >> 8 && same;
}

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
__global__ __launch_bounds__(kThreads) void k_kv_append(KvAppendArgs a, Slots sl) {
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
  if (!place(a.c, sl, slot, h, row, vs)) {
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
    if (!quantize_bounds(w, ts[kv], code, S)) quantize_block(w, (double)ts[kv], code, S);
    *(u32x2*)((kv ? a.c.v_codes : a.c.k_codes) + row * (a.c.D / 2) + 8 * b) = code;
    if (kv) a.c.v_scales[vs + (int64_t)b * a.c.page] = (uint8_t)S;
    else a.c.k_scales[row * nb + b] = (uint8_t)S;
  }
}

// Eight values of a token's keys and of its values a lane, for U tokens at once: four bytes of codes in, 16 or 32 bytes
// out, each, so that a wave's loads and stores are whole runs and U loads of each kind wait together.
template <int T, int U, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_kv_read(KvReadArgs a, Slots sl) {
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
    if (place(a.c, sl, slot[u], h, row, vs)) {
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
  return by_type(a, [&](auto t) { hipLaunchKernelGGL((k_kv_append<decltype(t)::value>), grid, dim3(kThreads), 0, s, a, slots_of(a.c)); });
}

// Keys and values that together pass kStream bytes are written past the caches: 65536 tokens x 8 x 128 of bf16 (268 MB)
// 53 us, 72 without; 32768 28.0 and 29.3. Below, what is read back stays there for the product that follows, though
// the call itself would gain up to 32 MB (4096 tokens 5.8 us, 6.5 cached).
constexpr int64_t kStream = (int64_t)128 << 20;
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s) {
  const int per = kThreads / (a.c.D / 8);
  const bool stream = 2 * a.T * a.c.heads * a.c.D * (a.type == kF32 ? 4 : 2) >= kStream;
  // few tokens: one a lane, so that more workgroups share them (512 x 8 x 128 4.0 us, 5.2 with four; 2048 4.9 both, 8192
  // 10.5 with one, 9.6 with four)
  const int U = a.T * a.c.heads / per >= 8 * 256 ? kUnroll : 1;
  const dim3 grid((unsigned)((a.T + per * U - 1) / (per * U)), (unsigned)a.c.heads);
  return by_type(a, [&](auto t) {
    constexpr int T = decltype(t)::value;
    if (stream) hipLaunchKernelGGL((k_kv_read<T, kUnroll, true>), dim3((unsigned)((a.T + per * kUnroll - 1) / (per * kUnroll)), (unsigned)a.c.heads), dim3(kThreads), 0, s, a, slots_of(a.c));
    else if (U > 1) hipLaunchKernelGGL((k_kv_read<T, kUnroll, false>), grid, dim3(kThreads), 0, s, a, slots_of(a.c));
    else hipLaunchKernelGGL((k_kv_read<T, 1, false>), grid, dim3(kThreads), 0, s, a, slots_of(a.c));
  });
}

}  // namespace ssn
