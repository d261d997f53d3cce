// Integer 4-bit weights with group scales: quantise, dequantise, and the matrix-vector product for
// one token or a few, plain and grouped by expert.
//
//   W_hat[n, k] = s[n, g] * (q[n, k] - z[n, g]),  g = k / group,   q in 0..15, z = 8 without zeros
//   Y[m, n] = sum_k X[m, k] W_hat[n, k] = sum_g s[n, g] * sum_{k in g} X[m, k] (q[n, k] - z[n, g])
//
// The sum inside a group runs over whole numbers times activations, in f32, and the scale multiplies
// it once: no weight is ever rounded.
#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "device_once.hpp"
#include "launch.hpp"
#include "pipeline.hpp"
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
// One workgroup computes 16 NT weight rows (NT tiles of 16) for up to 16 MT rows of Y; its waves split K.
// A wave walks chunks of 128 k. Per chunk and tile a lane loads 16 bytes of codes: lane l holds row
// l % 16, k = 32 (l / 16) .. + 31, and v_mfma_f32_16x16x32 multiplies them with the activations as the
// A operand (lane l: row l % 16 of X) in four steps of 8 k per lane.
//
// Codes to operand: the bytes w & 0x0F0F0F0F (even k) and (w >> 4) & 0x0F0F0F0F (odd k), read as E4M3,
// stand for q 2^-9 exactly (0..7 are its subnormals, 8..15 its first binade), so one v_cvt_scalef32_pk
// with scale 2^9 turns two of them into whole numbers in bf16 or f16: seven instructions for eight
// codes. The operand's k then runs 0 2 4 6 1 3 5 7, and the activations are put in that order.
//
// The zero point enters after the sum: sum x (q - z) = sum x q - z sum x, with sum x from one more
// matrix instruction per step whose weights are all ones, shared by the tiles.
//
// A group of a multiple of 128 (and K with it) covers whole chunks, and any order of k inside a chunk
// serves. For finer groups the four dwords of the lanes that share a row are transposed first
// (v_permlane32_swap, v_permlane16_swap), so that step s holds k = 32 s .. + 31, which lie in one group,
// and each step is scaled by itself.
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// a source of 16 zero bytes is not needed: rows of X past the last are copies of it, whose sums are dropped
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

// eight activations (two per word) in that order
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

constexpr int kChunk = 128;   // k per step of a wave's loop

template <int MT, int NT>
struct Chunk {
  u32x4 w[NT];
  uint32_t sz[NT];            // scale bits | zero point << 16
  u32x4 x[MT][4];
};

template <bool F16X, int MT, int NT, int WAVES, bool FINE, bool GROUPED, int RING>
__global__ __launch_bounds__(WAVES * 64) void k_int4_gemv(Int4GemvArgs a, int ngroups, int64_t items) {
  constexpr int kThr = WAVES * 64, kRows = 16 * MT;
  __shared__ float red[WAVES][NT * MT * 4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  const int No = a.silu ? (int)(a.N / 2) : (int)a.N;
  const int nch = (int)((a.K + kChunk - 1) / kChunk);
  const int c_lo = nch * wave / WAVES, c_hi = nch * (wave + 1) / WAVES;
  const int g32 = (int)(a.group / 32);
  int e = 0, r0 = 0, cnt = 0;
  int64_t item = blockIdx.x, step = gridDim.x;
  if constexpr (GROUPED) {
    Slot sl;
    if (!find_slot(a.offsets, a.E, (int)a.M, kRows, ngroups, sl)) return;
    e = sl.e; r0 = sl.r0; cnt = sl.cnt; item = sl.part; step = sl.parts;
  }
  for (; item < items; item += step) {
    const int ng = (int)(item % ngroups);
    if constexpr (!GROUPED) {
      r0 = (int)(item / ngroups) * kRows;
      cnt = (int)min(a.M - r0, (int64_t)kRows);
    }
    // this lane's weight row of each tile and activation row of each row tile
    const uint8_t* wp[NT];
    int64_t sg[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      int n;
      if (a.silu) n = t * No + min(16 * ng + r16, No - 1);
      else n = min(16 * (NT * ng + t) + r16, No - 1);
      const int64_t row = (int64_t)e * a.N + n;
      wp[t] = a.codes + row * (a.K / 2);
      sg[t] = row * a.groups;
    }
    const uint16_t* xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      int64_t src = r0 + min(16 * mt + r16, cnt - 1);
      if (GROUPED) src = min(max(a.row_token ? (int64_t)a.row_token[src] : src, (int64_t)0), a.x_rows - 1);
      xp[mt] = (const uint16_t*)a.X + src * a.K;
    }
    auto load = [&](int c) -> Chunk<MT, NT> {
      Chunk<MT, NT> o;
      c = min(c, c_hi - 1);
      const int k0 = kChunk * c + 32 * kq;            // this lane's 32 codes
      const int kc = FINE ? min(k0, (int)a.K - 32) : k0;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        o.w[t] = *(const u32x4*)(wp[t] + kc / 2);
        const int64_t i = sg[t] + (FINE ? (kc / 32) / g32 : (4 * c) / g32);
        o.sz[t] = (uint32_t)a.scales[i] | (a.zeros ? (uint32_t)a.zeros[i] << 16 : 8u << 16);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = FINE ? min(kChunk * c + 32 * s, (int)a.K - 32) + 8 * kq : k0 + 8 * s;
          o.x[mt][s] = *(const u32x4*)(xp[mt] + k);
        }
      return o;
    };
    const uint32_t one = F16X ? 0x3C003C00u : 0x3F803F80u;
    const u32x4 ones = {one, one, one, one};
    f32x4 tot[NT][MT], acc[NT][MT], xs[MT];
    const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int t = 0; t < NT; ++t) tot[t][mt] = zero4;
    auto fold = [&](const uint32_t* sz) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const float s = float16_of((uint16_t)(sz[t] & 0xFFFFu), a.s_type), z = (float)(sz[t] >> 16);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            tot[t][mt][i] = __builtin_fmaf(s, __builtin_fmaf(-z, xs[mt][i], acc[t][mt][i]), tot[t][mt][i]);
      }
    };
    auto multiply = [&](const Chunk<MT, NT>& cur, int c) {
      u32x4 w[NT], szs[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w[t] = FINE ? transpose4(cur.w[t]) : cur.w[t];
        if (FINE) szs[t] = spread4(cur.sz[t]);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (FINE && kChunk * c + 32 * s >= a.K) break;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const u32x4 x = x_operand(cur.x[mt][s]);
          xs[mt] = mfma16<F16X>(x, ones, FINE || s == 0 ? zero4 : xs[mt]);
#pragma unroll
          for (int t = 0; t < NT; ++t)
            acc[t][mt] = mfma16<F16X>(x, codes_operand<F16X>(w[t][s]), FINE || s == 0 ? zero4 : acc[t][mt]);
        }
        if (FINE) {
          uint32_t sz[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) sz[t] = szs[t][s];
          fold(sz);
        }
      }
      if (!FINE) fold(cur.sz);
    };
    if (c_lo < c_hi) {
      Chunk<MT, NT> ring[RING];
#pragma unroll
      for (int u = 0; u < RING; ++u) ring[u] = load(c_lo + u);
      for (int c = c_lo; c < c_hi; c += RING) {
#pragma unroll
        for (int u = 0; u < RING; ++u) {
          if (c + u >= c_hi) break;
          const Chunk<MT, NT> cur = ring[u];
          ring[u] = load(c + u + RING);
          __builtin_amdgcn_sched_barrier(0);
          multiply(cur, c + u);
        }
      }
    }
    // the waves' shares of K meet in LDS, one thread per output
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][(t * MT + mt) * 4 + i][lane] = tot[t][mt][i];
    __syncthreads();
    const int outs = (a.silu ? 1 : NT) * MT * 4 * 64;
    for (int o = threadIdx.x; o < outs; o += kThr) {
      const int l = o & 63, j = o >> 6;
      float y = 0.f;
      for (int w = 0; w < WAVES; ++w) y += red[w][j][l];
      const int t = j / (MT * 4), mt = j / 4 % MT, m = 16 * mt + 4 * (l >> 4) + (j & 3);
      const int n = (a.silu ? 16 * ng : 16 * (NT * ng + t)) + (l & 15);
      if (a.silu) {
        float u = 0.f;
        for (int w = 0; w < WAVES; ++w) u += red[w][MT * 4 + j][l];
        y = silu(y) * u;
      }
      if (m < cnt && n < No) store_elem(a.Y, a.y_type, (int64_t)(r0 + m) * No + n, y);
    }
    __syncthreads();
  }
}

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
constexpr uint32_t kOutside = 0x80000000u;   // a byte offset past the end of every resource

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
    for (int c = 0; c < C; ++c) load_unit(buf[d], tile + (d / H) * stride, d % H, c);
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
      tot[0] = work(buf[0], D == 1 ? tile : tile + stride, D == 1 ? 1 : 0);
      tot[1] = work(buf[D - 1], tile + stride, D == 1 ? 0 : 1);
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

namespace {

template <bool F16X, int MT, int NT, int WAVES, bool FINE, bool GROUPED>
hipError_t launch_gemv_t(const Int4GemvArgs& a, hipStream_t s) {
  constexpr int kRows = 16 * MT;
  const int64_t No = a.silu ? a.N / 2 : a.N, per = a.silu ? 16 : 16 * NT;
  const int ngroups = (int)((No + per - 1) / per);
  const int64_t items = GROUPED ? ngroups : (a.M + kRows - 1) / kRows * ngroups;
  const int64_t grid = GROUPED ? std::max<int64_t>(4 * cu_count(), std::min<int64_t>(a.E, a.M) + a.M / kRows) : items;
  constexpr int kRing = MT == 1 ? 3 : MT == 2 ? 2 : 1;
  hipLaunchKernelGGL((k_int4_gemv<F16X, MT, NT, WAVES, FINE, GROUPED, kRing>),
                     dim3((unsigned)std::min<int64_t>(grid, GROUPED ? grid : 1 << 22)), dim3(WAVES * 64), 0, s, a, ngroups, items);
  return hipGetLastError();
}

#ifndef WG_CU
#define WG_CU (16 / W > 0 ? 16 / W : 1)
#endif
#ifndef GP
#define GP 2
#endif
#ifndef D4
#define D4 1
#endif
#ifndef D2
#define D2 1
#endif
template <bool F16X, int P, int C, int FOLD, int D, bool GROUPED, bool SILU>
hipError_t launch_rows_t(const Int4GemvArgs& a, hipStream_t s) {
  constexpr int ROWS = 16 / P;
  const int nch = (int)((a.K + kChunk - 1) / kChunk), W = (nch + C - 1) / C;
  const int64_t No = SILU ? a.N / 2 : a.N;
  const int tiles = (int)((No + 15) / 16);
  const int64_t wgs = (int64_t)cu_count() * WG_CU;
  // grouped: at least a workgroup for every slot that there may be (each expert's last may be partial)
  const int64_t grid = GROUPED ? std::max<int64_t>(2 * wgs, std::min<int64_t>(a.E, a.M) + a.M / ROWS)
                               : std::min<int64_t>(wgs, tiles);
  hipLaunchKernelGGL((k_int4_rows<F16X, P, C, FOLD, D, GROUPED, SILU>), dim3((unsigned)grid), dim3(W * 64),
                     W == 1 ? 0 : 2 * W * (SILU ? 2 : 1) * 4 * ROWS * 16, s, a, tiles);
  return hipGetLastError();
}

template <bool F16X, int FOLD, bool GROUPED, bool SILU>
hipError_t launch_rows_c(const Int4GemvArgs& a, hipStream_t s) {
  const int nch = (int)((a.K + kChunk - 1) / kChunk);
  if (a.M <= 4 || (GROUPED && GP == 4)) {
    if (nch <= 64) return launch_rows_t<F16X, 4, 4, FOLD, D4, GROUPED, SILU>(a, s);
    return launch_rows_t<F16X, 4, 8, FOLD, 1, GROUPED, SILU>(a, s);
  }
  if (a.M <= 8 || (GROUPED && GP == 2)) return launch_rows_t<F16X, 2, 4, FOLD, D2, GROUPED, SILU>(a, s);
  if constexpr (!GROUPED || GP == 1) {
  if (nch <= 32) return launch_rows_t<F16X, 1, 2, FOLD, 2, GROUPED, SILU>(a, s);
  if (nch <= 48) return launch_rows_t<F16X, 1, 3, FOLD, 2, GROUPED, SILU>(a, s);
  return launch_rows_t<F16X, 1, 4, FOLD, 1, GROUPED, SILU>(a, s);
  }
  return hipSuccess;
}

template <bool F16X, int FOLD>
hipError_t launch_rows_s(const Int4GemvArgs& a, hipStream_t s) {
  if (!a.offsets) return launch_rows_c<F16X, FOLD, false, false>(a, s);
  return a.silu ? launch_rows_c<F16X, FOLD, true, true>(a, s) : launch_rows_c<F16X, FOLD, true, false>(a, s);
}

template <bool F16X>
hipError_t launch_rows(const Int4GemvArgs& a, hipStream_t s) {
  if (a.group % 128 == 0) return launch_rows_s<F16X, 4>(a, s);
  return a.group % 64 == 0 ? launch_rows_s<F16X, 2>(a, s) : launch_rows_s<F16X, 1>(a, s);
}

template <bool F16X, bool FINE>
hipError_t launch_gemv_x(const Int4GemvArgs& a, hipStream_t s) {
  const bool fits = a.K <= 64 * kChunk || (a.M <= 4 && a.K <= 128 * kChunk);
  if (fits && (a.offsets || a.M <= 16)) return launch_rows<F16X>(a, s);
  if (a.offsets) return launch_gemv_t<F16X, 1, 2, 8, FINE, true>(a, s);
  if (a.M <= 16) return launch_gemv_t<F16X, 1, 2, 8, FINE, false>(a, s);
  if (a.M <= 32) return launch_gemv_t<F16X, 2, 2, 8, FINE, false>(a, s);
  return launch_gemv_t<F16X, 4, 2, 4, FINE, false>(a, s);
}

}  // namespace

hipError_t launch_int4_gemv(const Int4GemvArgs& args, hipStream_t s) {
  Int4GemvArgs a = args;
  if (a.group >= a.K) a.group = (a.K + kChunk - 1) / kChunk * kChunk;   // one group: any length past K's end
  const bool fine = a.group % kChunk || a.K % kChunk;
  if (a.x_type == kF16) return fine ? launch_gemv_x<true, true>(a, s) : launch_gemv_x<true, false>(a, s);
  return fine ? launch_gemv_x<false, true>(a, s) : launch_gemv_x<false, false>(a, s);
}

}  // namespace ssn
