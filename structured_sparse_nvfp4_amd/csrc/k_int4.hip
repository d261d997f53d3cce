// Integer 4-bit weights with group scales: quantise, dequantise, and the matrix-vector product for
// one token or a few, plain and grouped by expert (the arithmetic is in int4.hpp).
#include <algorithm>
#include <type_traits>

#include "device_once.hpp"
#include "int4.hpp"

namespace ssn {
namespace {

constexpr int kThreads = 256;

// eight consecutive weights of type T as f32, from a pointer aligned to them
template <int T>
__device__ __forceinline__ void load8(const void* p, int64_t i, float* w) {
  if constexpr (T == kF32) {
    const f32x4 a = ((const f32x4*)p)[i / 4], b = ((const f32x4*)p)[i / 4 + 1];
#pragma unroll
    for (int j = 0; j < 4; ++j) { w[j] = a[j]; w[4 + j] = b[j]; }
  } else {
    const u32x4 v = ((const u32x4*)p)[i / 8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = T == kBF16 ? bf16_lo(v[j]) : f16_of((uint16_t)v[j]);
      w[2 * j + 1] = T == kBF16 ? bf16_hi(v[j]) : f16_of((uint16_t)(v[j] >> 16));
    }
  }
}

// ------------------------------------------------------------------------------ quantise
// A scale as the quantiser uses it: inv = 1 / s to a few units, half = s / 2, step = twice the distance from
// half to the next smaller number.
struct Step {
  float s, inv, half, step;
};
__device__ __forceinline__ Step make_step(float s) {
  const float half = 0.5f * s;
  return {s, __builtin_amdgcn_rcpf(s), half, 2.f * (half - __uint_as_float(__float_as_uint(half) - 1))};
}

// The whole number nearest to w / s, halves to the even one. q = rint(w inv) is it or a neighbour's. The
// rest w - s q is exact in one FMA (s has at most 11 significant bits and q five, and the rest is a
// multiple of w's last bit below s), so comparing it with s / 2 decides exactly; an odd q yields at s / 2 itself, that is
// beyond the next smaller number. (Where |w / s| is far beyond the codes the result is clamped anyway.)
__device__ __forceinline__ float nearest_multiple(float w, const Step& t) {
  const float q = __builtin_rintf(w * t.inv);
  const float rest = __builtin_fmaf(-t.s, q, w);
  const float odd = __builtin_amdgcn_fractf(0.5f * q);          // 0, or 0.5 for an odd q
  const float limit = __builtin_fmaf(-odd, t.step, t.half);
  return __builtin_fabsf(rest) > limit ? q + __builtin_copysignf(1.f, rest) : q;
}

// the largest of the values of the L lanes that a lane is among (L a power of two)
template <int L>
__device__ __forceinline__ float team_max(float v) {
  auto of = [&](int moved) { v = fmaxf(v, __int_as_float(moved)); };
  if (L > 1) of(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));     // quad 1 0 3 2
  if (L > 2) of(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));                // quad 2 3 0 1
  if (L > 4) of(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));    // mirrored in 8
  if (L > 8) of(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));    // mirrored in 16
  if (L > 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if (L > 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}

// One team of L lanes per group. Its 8 U L weights stay in registers between the search for the range and the
// codes, which is the whole group for the teams of a wave or less; a workgroup (L = 256) reads what goes beyond a
// second time, from the L2. f32 is bound by memory (W read, codes written), 16-bit weights by the vector units, which
// issue all the time: 20 instructions a weight for f32, 29 for bf16, whose lanes take the exact decision (below) as
// well more often than not. Two vectors of eight a lane rather than one halve what a lane spends on its group
// (the range's way across lanes, the scale, the places), 13824 x 5120, group 128: f32 58 against 63 us (5.5 TB/s), bf16
// 47 against 58; group 32, bf16: 49 against 57.
// Groups beyond 2048 have a workgroup, which holds 8192 weights: one group of 5120 to a row 60 us, with a wave and
// a second reading 79; 16 rows of 8192 4.2 against 8.7.
// Six waves per SIMD at least: left alone the compiler unpacks all of a bf16 wave's 2048 weights at once (104
// registers, four waves), groups of 1024 65 us against 54.
template <int T, int L, int U>
__global__ __launch_bounds__(kThreads, 6) void k_int4_quantize(const void* __restrict__ W, int64_t teams, int K,
                                                               int group, int groups, uint32_t* __restrict__ codes,
                                                               uint16_t* __restrict__ scales, int st,
                                                               uint8_t* __restrict__ zeros) {
  constexpr int kTeams = kThreads / L;         // per workgroup
  const int l = threadIdx.x % L;
  for (int64_t t0 = (int64_t)blockIdx.x * kTeams; t0 < teams; t0 += (int64_t)gridDim.x * kTeams) {
    const int64_t team = t0 + threadIdx.x / L;
    const bool live = team < teams;
    // row and group of this team: the workgroup's first by a uniform division, the rest by counting on
    const int64_t row0 = t0 / groups;
    const int g0 = (int)(t0 - row0 * groups) + (int)(threadIdx.x / L);
    const int64_t n = row0 + g0 / groups;
    const int k0 = g0 % groups * group, len = min(group, K - k0);
    const int64_t base = n * K + k0;
    // the group's first 8 U L weights stay in registers
    float w[U][8] = {}, lo = 0.f, hi = 0.f;
    auto extend = [&](const float* v) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) { lo = fminf(lo, v[j]); hi = fmaxf(hi, v[j]); }
    };
    if (live) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (8 * (l + L * u) < len) load8<T>(W, base + 8 * (l + L * u), w[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) extend(w[u]);
      if constexpr (L > 64)
        for (int k = 8 * (l + L * U); k < len; k += 8 * L) {
          float v[8];
          load8<T>(W, base + k, v);
          extend(v);
        }
    }
    if constexpr (L <= 64) {
      hi = team_max<L>(hi);
      lo = -team_max<L>(-lo);
    } else {                                   // the workgroup's waves meet in LDS
      __shared__ float most[2][kThreads / 64];
      const float h = team_max<64>(hi), m = team_max<64>(-lo);
      __syncthreads();                         // the group before has been read
      if (threadIdx.x % 64 == 0) most[0][threadIdx.x / 64] = h, most[1][threadIdx.x / 64] = m;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kThreads / 64; ++i) {
        hi = fmaxf(hi, most[0][i]);
        lo = fminf(lo, -most[1][i]);
      }
    }
    const double range = zeros ? ((double)hi - (double)lo) / 15.0 : (double)fmaxf(hi, -lo) / 7.0;
    const uint16_t sb = round16_sat(range, st);
    const float s0 = float16_of(sb, st);
    // subnormal scales: both sides times 2^64, exactly, or the reciprocal overflows
    const float f = s0 < 0x1p-100f ? 0x1p64f : 1.f;
    const Step step = make_step(s0 * f);
    const bool any = s0 > 0.f;
    float z = 8.f;
    if (zeros) z = any ? fminf(fmaxf(nearest_multiple(-lo * f, step), 0.f), 15.f) : 0.f;
    if (!live) continue;
    auto encode = [&](const float* v, int k) __attribute__((always_inline)) {
      // The codes as bytes, from w inv + z. With s normal that is off by less than 2^-17 from w / s + z wherever
      // it is not clamped, so only what lies within 2^-16 of a half needs the exact decision. The whole wave takes
      // it where one lane must: for normally distributed weights in groups of 128 1.5 percent of the time if they
      // are f32, 59 if they and the scales are bf16 (f16 11), as quotients of so few bits fall on halves more often.
      uint32_t even = 0, odd = 0;
      float far = 0.f;                         // the farthest from its whole number
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const float a = __builtin_amdgcn_fmed3f(__builtin_fmaf(v[j], step.inv, z), 0.f, 15.f);
        const float b = __builtin_amdgcn_fmed3f(__builtin_fmaf(v[j + 1], step.inv, z), 0.f, 15.f);
        const float qa = __builtin_rintf(a), qb = __builtin_rintf(b);
        far = fmaxf(fmaxf(far, __builtin_fabsf(a - qa)), __builtin_fabsf(b - qb));
        even = __builtin_amdgcn_cvt_pk_u8_f32(qa, j / 2, even);
        odd = __builtin_amdgcn_cvt_pk_u8_f32(qb, j / 2, odd);
      }
      if (__ballot(far > 0.5f - 0x1p-16f || f != 1.f)) {
        even = odd = 0;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const float a = __builtin_amdgcn_fmed3f(nearest_multiple(v[j] * f, step) + z, 0.f, 15.f);
          const float b = __builtin_amdgcn_fmed3f(nearest_multiple(v[j + 1] * f, step) + z, 0.f, 15.f);
          even = __builtin_amdgcn_cvt_pk_u8_f32(a, j / 2, even);
          odd = __builtin_amdgcn_cvt_pk_u8_f32(b, j / 2, odd);
        }
      }
      codes[(base + k) / 8] = any ? even | odd << 4 : 0x11111111u * (uint32_t)z;
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (8 * (l + L * u) < len) encode(w[u], 8 * (l + L * u));
    if constexpr (L > 64)
      for (int k = 8 * (l + L * U); k < len; k += 8 * L) {
        float v[8];
        load8<T>(W, base + k, v);
        encode(v, k);
      }
    if (l == 0) {
      scales[team] = sb;
      if (zeros) zeros[team] = (uint8_t)z;
    }
  }
}

// ------------------------------------------------------------------------------ dequantise
// One lane per 16 bytes of output (four or eight k) of a row, over several rows: where its group lies in a
// row is found once. STREAM: the output passes the caches by.
template <int T, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_int4_dequantize(const uint8_t* __restrict__ codes,
                                                              const uint16_t* __restrict__ scales, int st,
                                                              const uint8_t* __restrict__ zeros, int64_t N, int K,
                                                              int group, int groups, void* __restrict__ out) {
  constexpr int kPer = T == kF32 ? 4 : 8;
  using Codes = std::conditional_t<T == kF32, uint16_t, uint32_t>;
  const int v = blockIdx.x * kThreads + threadIdx.x, nv = K / kPer;
  if (v >= nv) return;
  const int g = kPer * v / group;
#pragma unroll 4
  for (int64_t n = blockIdx.y; n < N; n += gridDim.y) {
    const int64_t i = n * nv + v;
    const uint32_t c = ((const Codes*)codes)[i];
    const float s = float16_of(scales[n * groups + g], st), z = zeros ? (float)zeros[n * groups + g] : 8.f;
    float w[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) w[j] = ((float)(c >> (4 * j) & 15) - z) * s;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (T == kF32) o[j] = __float_as_uint(w[j]);
      else if constexpr (T == kBF16) o[j] = pk_bf16_rne(w[2 * j], w[2 * j + 1]);
      else o[j] = (uint32_t)to_f16(w[2 * j]) | (uint32_t)to_f16(w[2 * j + 1]) << 16;
    }
    if (STREAM) __builtin_nontemporal_store(o, (u32x4*)out + i);
    else ((u32x4*)out)[i] = o;
  }
}

// ------------------------------------------------------------------------------ product, up to 16 rows
// ---- up to 16 rows of Y: activations stay in registers
// One workgroup of W waves serves one set of up to 16 / P rows of Y and walks over units of 16 weight
// rows. Wave w owns chunks [nch w / W, nch (w + 1) / W) of K, at most C of them, and keeps their activations
// as operands in registers for its whole life, so that the loop reads only weights. Codes, scales and
// zero points come through buffer resources set to the unit's rows: what lies outside (rows past the
// last, k past the end, a chunk that the wave has not, the unit after the last) reads as zero without a
// branch and without traffic, and adds nothing. D units are in flight; a chunk's registers are refilled
// as soon as its codes are decoded.
//
// A span is FOLD steps of 32 k that share a scale (4: groups of a multiple of 128, whose chunks need no
// transposition). With few rows of Y the operand's 16 rows hold P spans of 16 / P rows each: row block p
// of pack j is span P j + p. Every span's codes multiply the whole operand, and of the result only the
// row block of that span is kept, which lies in its own lanes, where one fold serves P spans.
// The activations then take 1 / P of the registers.
//
// Memory-bound: N = 131072, K = 5120, group 128 takes 67 us at M = 1 (5.2 TB/s, where a large copy reaches 5.06),
// 74 at M = 8, 84 at M = 16; N = 13824 11.0 and 13.0 us at M = 1 and 8, of which some 3 us are the launch, the
// activations and the first weights. Groups of 32 cost four scales and a transposition per chunk: N = 131072,
// M = 8 116 us.
template <int C, int FOLD>
struct UnitLoads {
  static constexpr int kScales = (4 * C / FOLD + 3) / 4;
  u32x4 w[C];
  uint32_t s[kScales], z[kScales];           // four spans, one per lane group
};

template <bool F16X, int P, int C, int FOLD, int D, bool GROUPED, bool SILU>
__global__ __launch_bounds__(1024) void k_int4_rows(Int4GemvArgs a, int tiles) {
  constexpr int H = SILU ? 2 : 1;             // units per tile of 16 outputs: gate and up
  constexpr int SPANS = 4 * C / FOLD, PACKS = SPANS / P, ROWS = 16 / P;
  static_assert(SPANS % P == 0, "whole packs");
  static_assert(!SILU || D == 1, "gate and up take turns in one set of registers");
  using Loads = UnitLoads<C, FOLD>;
  // whether the sums of x stay in registers too, or are formed again for every unit (one more matrix
  // instruction per step: the matrix cores have the time, the registers are full)
  constexpr bool KEEP = PACKS <= (SILU ? 2 : 3);
  extern __shared__ f32x4 red[];              // [2][W][H][4 ROWS]: the waves' shares
  const int W = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int No = (int)(SILU ? a.N / 2 : a.N);
  const int K = (int)a.K, nch = (K + kChunk - 1) / kChunk, g32 = (int)(a.group / 32), groups = (int)a.groups;
  const int c_lo = nch * wave / W, nc = nch * (wave + 1) / W - c_lo;
  const int k_end = min(K, kChunk * (c_lo + nc));
  int e = 0, r0 = 0, cnt = (int)a.M, tile = blockIdx.x, stride = gridDim.x;
  // this lane's row of X; rows past the last are copies of it, whose sums are dropped
  int src;
  if constexpr (GROUPED) {
    Slot sl;
    if (!find_slot(a.offsets, a.E, (int)a.M, ROWS, tiles, sl)) return;
    e = sl.e; r0 = sl.r0; cnt = sl.cnt; tile = sl.part; stride = sl.parts;
    src = r0 + min(r16 % ROWS, cnt - 1);
    if (a.row_token) src = a.row_token[src];
  } else {
    src = min(r16 % ROWS, cnt - 1);
  }
  // the first k of a span of the wave
  auto span_k = [&](int u) { return kChunk * c_lo + 32 * FOLD * u; };
  const uint32_t kq_0 = kq & 1 ? ~0u : 0u, kq_1 = kq & 2 ? ~0u : 0u;
  // where this lane's codes, scales and zero points lie in its row of a unit: the same for every unit
  uint32_t koff[C], goff[Loads::kScales];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int k = kChunk * (c_lo + c) + 32 * kq;
    koff[c] = k < k_end ? (uint32_t)(r16 * (K / 2) + k / 2) : kOutside;
  }
#pragma unroll
  for (int i = 0; i < Loads::kScales; ++i) {
    // lane group g loads span 4 i + g; with P = 2, groups 1 and 2 change places, for the swap that follows
    const int u = 4 * i + (P == 2 ? (kq >> 1) | (kq & 1) << 1 : kq), k = span_k(u);
    goff[i] = u < SPANS && k < k_end ? (uint32_t)(r16 * groups + k / 32 / g32) : kOutside / 2;
  }
  const uint32_t z_add = a.zeros ? 0u : 8u;
  auto load_unit = [&](Loads& o, int tile, int half, int c) __attribute__((always_inline)) {
    const int rows = tile < tiles ? min(16, No - 16 * tile) : 0;
    const int64_t row = (int64_t)e * a.N + (int64_t)half * No + 16 * tile;
    const auto wr = buf_rsrc(a.codes + row * (K / 2), rows * (K / 2));
    o.w[c] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, koff[c], 0, 0));
    if (c % FOLD == 0) {                      // the chunk whose first span starts scale register c / FOLD
      const auto sr = buf_rsrc(a.scales + row * groups, rows * groups * 2);
      const auto zr = buf_rsrc(a.zeros + row * groups, a.zeros ? rows * groups : 0);
      o.s[c / FOLD] = __builtin_amdgcn_raw_buffer_load_b16(sr, 2 * goff[c / FOLD], 0, 0);
      o.z[c / FOLD] = __builtin_amdgcn_raw_buffer_load_b8(zr, goff[c / FOLD], 0, 0);
    }
  };
  // The activations, zeros where the wave has no k. Without experts their loads go out first: they come
  // from the L2, and are put in order while the first weights are on their way. With experts they wait for
  // the row's token, and the weights do not.
  const uint32_t one = F16X ? 0x3C003C00u : 0x3F803F80u;
  u32x4 ones = {one, one, one, one};
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
  u32x4 x[PACKS][FOLD];
  Loads buf[D];
  auto x_k = [&](int j, int t) {
    return span_k(P * j + r16 / ROWS) + (FOLD == 4 ? 32 * kq + 8 * t : 32 * t + 8 * kq);
  };
  auto load_x = [&]() __attribute__((always_inline)) {
    if (GROUPED) src = min(max(src, 0), (int)a.x_rows - 1);
    const uint16_t* const xp = (const uint16_t*)a.X + (int64_t)src * K;
#pragma unroll
    for (int j = 0; j < PACKS; ++j)
#pragma unroll
      for (int t = 0; t < FOLD; ++t) x[j][t] = *(const u32x4*)(xp + (x_k(j, t) < k_end ? x_k(j, t) : 0));
  };
  if (!GROUPED) load_x();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < D; ++d)
#pragma unroll
    for (int c = 0; c < C; ++c) load_unit(buf[d], tile + d * stride, 0, c);
  __builtin_amdgcn_sched_barrier(0);
  if (GROUPED) load_x();
  f32x4 xs[KEEP ? PACKS : 1];
#pragma unroll
  for (int j = 0; j < PACKS; ++j) {
    if (KEEP) xs[j] = zero4;
#pragma unroll
    for (int t = 0; t < FOLD; ++t) {
      x[j][t] = x_k(j, t) < k_end ? x_operand(x[j][t]) : u32x4{0u, 0u, 0u, 0u};
      if (KEEP) xs[j] = mfma16<F16X>(x[j][t], ones, xs[j]);
    }
  }

  // multiplies the unit in b and refills b with the unit of (next, half) as its registers come free
  auto work = [&](Loads& b, int next, int half) __attribute__((always_inline)) -> f32x4 {
    f32x4 tot = zero4;
    if (!KEEP) asm volatile("" : "+v"(ones));   // or the compiler forms the sums once, and spills them
    u32x4 szs = {};
    f32x4 part[P];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const u32x4 w = FOLD == 4 ? b.w[c] : transpose4(b.w[c]);
#pragma unroll
      for (int v = 0; v < 4 / FOLD; ++v) {
        const int u = c * (4 / FOLD) + v, j = u / P;   // span and pack
        if (u % 4 == 0) {
          const uint32_t sz = b.s[u / 4] | (b.z[u / 4] + z_add) << 16;
          if (P == 4) {
            szs[0] = sz;
          } else if (P == 2) {
            const auto r = __builtin_amdgcn_permlane16_swap(sz, sz, false, false);
            szs[0] = r[0];
            szs[1] = r[1];
          } else {
            szs = spread4(sz);
          }
        }
        part[u % P] = zero4;
#pragma unroll
        for (int t = 0; t < FOLD; ++t)
          part[u % P] = mfma16<F16X>(x[j][t], codes_operand<F16X>(w[FOLD * v + t]), part[u % P]);
        if (u % P != P - 1) continue;
        f32x4 sum = zero4;
        if (KEEP) sum = xs[j];
        else
#pragma unroll
          for (int t = 0; t < FOLD; ++t) sum = mfma16<F16X>(x[j][t], ones, sum);
        const uint32_t sz = szs[P == 1 ? u % 4 : P == 2 ? u / 2 % 2 : 0];
        const float s = float16_of((uint16_t)(sz & 0xFFFFu), a.s_type), z = (float)(sz >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // the row block's own span: lanes choose by the bits of their group
          float acc = part[0][i];
          if (P == 2) acc = choose(kq_1, part[P - 1][i], acc);
          if (P == 4) acc = choose(kq_1, choose(kq_0, part[P - 1][i], part[2 % P][i]), choose(kq_0, part[1 % P][i], acc));
          tot[i] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[i], acc), tot[i]);
        }
        asm volatile("" : "+v"(tot));         // here, or every pack's sums are held to the end
      }
      __builtin_amdgcn_sched_barrier(0);      // the refill goes out here, not further down
      load_unit(b, next, half, c);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the row blocks' shares meet in the first
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (P >= 2) tot[i] = sum_halves(tot[i]);
      if (P == 4) tot[i] = sum_quarters(tot[i]);
    }
    return tot;
  };
  // The waves' shares of K meet in LDS (two buffers, one barrier per tile), one thread per output, the waves
  // taking turns at it. A single wave stores what it holds.
  auto store = [&](int m, int n16, float y, float u) {
    const int n = 16 * tile + n16;
    if (SILU) y = silu(y) * u;
    if (m < cnt && n < No) store_elem(a.Y, a.y_type, (int64_t)(r0 + m) * No + n, y);
  };
  int turn = 0;
  auto finish = [&](const f32x4* tot) __attribute__((always_inline)) {
    if (W == 1) {
      if (4 * kq < ROWS)
#pragma unroll
        for (int i = 0; i < 4; ++i) store(4 * kq + i, r16, tot[0][i], tot[H - 1][i]);
      return;
    }
    f32x4* part = red + (turn & 1) * W * H * 4 * ROWS;
    if (4 * kq < cnt)
#pragma unroll
      for (int h = 0; h < H; ++h) part[(wave * H + h) * 4 * ROWS + lane] = tot[h];
    __builtin_amdgcn_s_waitcnt(0xC07F);       // the LDS writes; the loads under way stay so
    stage_barrier();
    int o = (int)threadIdx.x - 64 * (turn * (ROWS / 4) % W);
    if (o < 0) o += blockDim.x;
    for (; o < 16 * cnt; o += blockDim.x) {
      const int n16 = o & 15, m = o >> 4;
      const float* p = (const float*)(part + 16 * (m >> 2) + n16) + (m & 3);
      float y = 0.f, u = 0.f;
#pragma unroll 4
      for (int w = 0; w < W; ++w) {
        y += p[w * H * 16 * ROWS];
        if (SILU) u += p[(w * H + 1) * 16 * ROWS];
      }
      store(m, n16, y, u);
    }
    ++turn;
  };
  for (;;) {
    f32x4 tot[2];
    if constexpr (SILU) {
      tot[0] = work(buf[0], tile, 1);
      tot[1] = work(buf[0], tile + stride, 0);
      finish(tot);
      if ((tile += stride) >= tiles) return;
    } else {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        tot[0] = work(buf[d], tile + D * stride, 0);
        finish(tot);
        if ((tile += stride) >= tiles) return;
      }
    }
  }
}

}  // namespace

namespace {

template <int T, int L, int U>
hipError_t launch_quantize_l(const void* W, int64_t N, int64_t K, int64_t group, uint8_t* codes, uint16_t* scales,
                             int s_type, uint8_t* zeros, hipStream_t s) {
  const int64_t groups = (K - 1) / group + 1, teams = N * groups;
  const int64_t blocks = std::min<int64_t>((teams + kThreads / L - 1) / (kThreads / L), 1 << 22);
  hipLaunchKernelGGL((k_int4_quantize<T, L, U>), dim3((unsigned)blocks), dim3(kThreads), 0, s, W, teams, (int)K,
                     (int)std::min(group, K), (int)groups, (uint32_t*)codes, scales, s_type, zeros);
  return hipGetLastError();
}

// lanes per group so that a lane has two vectors of eight of it, or four of a long one: all of a group of up to 2048
template <int T>
hipError_t launch_quantize_t(const void* W, int64_t N, int64_t K, int64_t group, uint8_t* codes, uint16_t* scales,
                             int s_type, uint8_t* zeros, hipStream_t s) {
  const int64_t len = std::min(group, K);
  if (len <= 32) return launch_quantize_l<T, 2, 2>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (len <= 64) return launch_quantize_l<T, 4, 2>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (len <= 128) return launch_quantize_l<T, 8, 2>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (len <= 256) return launch_quantize_l<T, 16, 2>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (len <= 512) return launch_quantize_l<T, 32, 2>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (len <= 2048) return launch_quantize_l<T, 64, 4>(W, N, K, group, codes, scales, s_type, zeros, s);
  return launch_quantize_l<T, 256, 4>(W, N, K, group, codes, scales, s_type, zeros, s);   // the one that reads again
}

}  // namespace

hipError_t launch_int4_quantize(const void* W, int w_type, int64_t N, int64_t K, int64_t group, uint8_t* codes,
                                uint16_t* scales, int s_type, uint8_t* zeros, hipStream_t s) {
  if (w_type == kF32) return launch_quantize_t<kF32>(W, N, K, group, codes, scales, s_type, zeros, s);
  if (w_type == kF16) return launch_quantize_t<kF16>(W, N, K, group, codes, scales, s_type, zeros, s);
  return launch_quantize_t<kBF16>(W, N, K, group, codes, scales, s_type, zeros, s);
}

namespace {

template <int T>
hipError_t launch_dequantize_t(const uint8_t* codes, const uint16_t* scales, int s_type, const uint8_t* zeros, int64_t N,
                               int64_t K, int64_t group, void* out, hipStream_t s) {
  const int groups = (int)((K - 1) / group + 1);
  const int64_t bx = (K / (T == kF32 ? 4 : 8) + kThreads - 1) / kThreads;
  // four rows a lane, and more where the grid would pass its second axis or some 2^20 workgroups
  const int64_t by = std::min<int64_t>({(N + 3) / 4, 65535, std::max<int64_t>(1, (1 << 20) / bx)});
  // Output that the 256 MB cache would hardly hold until it is read is written past it: 13824 x 5120 to f32 75.6
  // against 48.2 us, to bf16 (142 MB) 43.0 against 29.0, with a product that reads it 111 against 103. Smaller
  // output is better found in the caches: 4096 x 4096 to bf16 (34 MB) with its product 28.4 against 31.9 us, to
  // f32 28.2 against 29.5.
  const bool stream = N * K >= ((int64_t)128 << 20) / (T == kF32 ? 4 : 2);
  const auto kernel = stream ? k_int4_dequantize<T, true> : k_int4_dequantize<T, false>;
  hipLaunchKernelGGL(kernel, dim3((unsigned)bx, (unsigned)by), dim3(kThreads), 0, s, codes, scales, s_type, zeros, N,
                     (int)K, (int)std::min(group, K), groups, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, int s_type, const uint8_t* zeros,
                                  int64_t N, int64_t K, int64_t group, void* out, int out_type, hipStream_t s) {
  if (out_type == kF32) return launch_dequantize_t<kF32>(codes, scales, s_type, zeros, N, K, group, out, s);
  if (out_type == kF16) return launch_dequantize_t<kF16>(codes, scales, s_type, zeros, N, K, group, out, s);
  return launch_dequantize_t<kBF16>(codes, scales, s_type, zeros, N, K, group, out, s);
}

namespace {

template <bool F16X, int P, int C, int FOLD, bool GROUPED, bool SILU>
hipError_t launch_rows_t(const Int4GemvArgs& a, hipStream_t s) {
  constexpr int ROWS = 16 / P;
  // Units in flight per wave. With the activations of 16 rows in registers a compute unit holds 16 waves, which need
  // two units each to keep the memory busy; with fewer rows a second unit in flight was slower (N = 13824,
  // K = 5120, M = 1: 11.0 against 12.5 us), and with four chunks of 16 rows there is no room for one.
  constexpr int D = P == 1 && C < 4 ? 2 : 1;
  const int nch = (int)((a.K + kChunk - 1) / kChunk), W = (nch + C - 1) / C;
  const int tiles = (int)(((SILU ? a.N / 2 : a.N) + 15) / 16);
  // As many workgroups as give a compute unit some 16 waves: more (20 or 24 waves) start more often from cold
  // activations than they hide (N = 13824, K = 5120, M = 8: 13.1 against 17.0 us).
  const int64_t wgs = (int64_t)cu_count() * std::max(1, 16 / W);
  // grouped: a workgroup at least for every slot that there may be (each expert's last may be partial), and
  // otherwise fewer than the chip holds, as each first finds its slot, token and activations. Three quarters of
  // `wgs` against half, all and twice as many: 32 tokens to 10 of 512 experts, down (K = 512) 33.9, 35.1, 33.4 and 36
  // us, gate and up (K = 2048) 57, 53, 56 and 55; 8 tokens, gate and up 21, 21, 22 and 25, down 11.8, 12.1, 13.8 and
  // 16.8; 32 tokens to 10 of 20 experts, gate and up 15.5, 14.4, 16.9 and 19.6. None is best for all: half loses 2 to 4
  // percent on down projections and gains 7 on the other two, all loses 4 to 17 percent with few or crowded rows.
  const int64_t grid = GROUPED ? std::max<int64_t>(3 * wgs / 4, std::min<int64_t>(a.E, a.M) + a.M / ROWS)
                               : std::min<int64_t>(wgs, tiles);
  hipLaunchKernelGGL((k_int4_rows<F16X, P, C, FOLD, D, GROUPED, SILU>), dim3((unsigned)grid), dim3(W * 64),
                     W == 1 ? 0 : 2 * W * (SILU ? 2 : 1) * 4 * ROWS * 16, s, a, tiles);
  return hipGetLastError();
}

// Chunks per wave (C) so that at most 16 waves cover K; rows per workgroup (16 / P) by how many there are.
// With experts the rows of each are few but unknown here, and sets of eight serve best over routings: against
// sets of four and sixteen, 32 tokens to 10 of 512 experts took 58, 57 and 60 us (gate and up, K = 2048),
// to 10 of 20 experts 15.4, 20.8 and 17.4 us, one token 7.1, 6.8 and 8.5 us.
template <bool F16X, int FOLD, bool GROUPED, bool SILU>
hipError_t launch_rows_c(const Int4GemvArgs& a, hipStream_t s) {
  const int nch = (int)((a.K + kChunk - 1) / kChunk);
  if (a.M <= 4) {
    if (nch <= 64) return launch_rows_t<F16X, 4, 4, FOLD, GROUPED, SILU>(a, s);
    return launch_rows_t<F16X, 4, 8, FOLD, GROUPED, SILU>(a, s);
  }
  if constexpr (GROUPED) {
    return launch_rows_t<F16X, 2, 4, FOLD, true, SILU>(a, s);
  } else {
    if (a.M <= 8) return launch_rows_t<F16X, 2, 4, FOLD, false, false>(a, s);
    if (nch <= 32) return launch_rows_t<F16X, 1, 2, FOLD, false, false>(a, s);
    if (nch <= 48) return launch_rows_t<F16X, 1, 3, FOLD, false, false>(a, s);
    return launch_rows_t<F16X, 1, 4, FOLD, false, false>(a, s);
  }
}

template <bool F16X, int FOLD>
hipError_t launch_rows_s(const Int4GemvArgs& a, hipStream_t s) {
  if (!a.offsets) return launch_rows_c<F16X, FOLD, false, false>(a, s);
  return a.silu ? launch_rows_c<F16X, FOLD, true, true>(a, s) : launch_rows_c<F16X, FOLD, true, false>(a, s);
}

template <bool F16X>
hipError_t launch_rows(const Int4GemvArgs& a, hipStream_t s) {
  switch (int4_fold(a.group)) {
    case 4: return launch_rows_s<F16X, 4>(a, s);
    case 2: return launch_rows_s<F16X, 2>(a, s);
    default: return launch_rows_s<F16X, 1>(a, s);
  }
}

}  // namespace

hipError_t launch_int4_gemv(const Int4GemvArgs& args, hipStream_t s) {
  Int4GemvArgs a = args;
  if (a.group >= a.K) a.group = (a.K + kChunk - 1) / kChunk * kChunk;   // one group: any length past K's end
  // what the registers of 16 waves hold: 64 chunks of K, or 128 where four rows share an operand
  const bool fits = a.K <= (a.M <= 4 ? 128 : 64) * kChunk;
  // 9 to 16 rows take long to bring into registers, which pays from some four tiles of weight rows per compute
  // unit on. This kernel against the other, us: K = 5120, M = 16, N = 13824 18.2 and 16.6, 16384 18.4 and 17.1, 20480
  // 20.4 and 23.3, 32768 27.1 and 31.6; M = 9, N = 13824 15.5 and 16.1, 32768 24.5 and 31.2. K = 2048, M = 16,
  // N = 20480 11.3 and 11.2, 24576 12.6 and 11.5, 32768 14.4 and 16.2. K = 8192, M = 16, N = 16384 25.8 and 24.2,
  // 20480 29.7 and 32.8.
  const bool pays = a.offsets || a.M <= 8 || (a.M <= 16 && a.N >= 4 * 16 * (int64_t)cu_count());
  if (!fits || !pays) return launch_int4_wide(a, s);
  return a.x_type == kF16 ? launch_rows<true>(a, s) : launch_rows<false>(a, s);
}

}  // namespace ssn
