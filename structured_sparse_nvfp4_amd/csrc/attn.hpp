// Shared by the attention kernels over the 4-bit cache (k_attn.hip: few query rows to a key head, k_attn_tile.hip:
// many): what a workgroup is to do, and codes to operands.
//
//   y[r, j] = scale log2(e) q_r . K_hat_j,   out_r = sum_j 2^(y[r, j] - m_r) V_hat_j / sum_j 2^(y[r, j] - m_r)
//
// The query heads that share a key head are rows like the queries themselves: row r of (sequence, key head) is query
// r / G, head r % G of its G. Both kernels form S^T = K . Q^T and O^T = V^T . P^T on the matrix cores, so a lane
// holds one row's logits of several keys, which are its own operand of the second product: P never leaves its
// registers. K_hat and V_hat without their f32 scale are E2M1 * E4M3: at most six significant bits, in 2^-10 .. 2688,
// so exact in f16, and f16 is what both products take: p then has 11 bits where bf16 would have 8. A query row is
// brought into f16's range by a power of two, which its logits' factor takes back: its largest magnitude lies in [2^15,
// 2^16) then, and f16's last bit is 2^-24. So f16 queries are exact, bf16 ones (8 bits) down to 2^-32 of the row's
// largest; below, they are off by 2^-40 of the largest at most.
#pragma once
#include "common.hpp"
#include "launch.hpp"
#include "types.hpp"

namespace ssn {

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

// p is held as 2^(y - m + 7), large logits aside (Reference): f16's normal range then reaches down to 2^-21 of a row's
// largest and its subnormals to 2^-31. The reference m of a row is raised only where some y - m passes 8, so p stays below 2^15.
constexpr float kShift = 7.f, kTop = 15.f;
constexpr float kUnset = -3e38f;                 // m of a row that has met no key
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// n / d for n < 2^31 by a multiplication: m = ceil(2^(31 + s) / d) with 2^(s - 1) < d <= 2^s is below 2^32, and its excess
// e = m d - 2^(31 + s) < d keeps n e below 2^(31 + s), so the quotient is exact
struct Divisor {
  uint32_t m, d;
  int shift;
};
inline Divisor divisor(uint32_t d) {
  int s = 0;
  while (((uint64_t)1 << s) < d) ++s;
  return {(uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d), d, 31 + s};
}
__device__ __forceinline__ int div_by(const Divisor& p, int n) { return (int)(((uint64_t)(uint32_t)n * p.m) >> p.shift); }

struct AttnLaunch {
  AttnArgs a;
  Divisor pd, gd, td, sd;      // by the 16-token units of a page, G, row_tiles and splits
  int G, row_tiles, splits;
  bool owned;                  // tiles: workgroups for those that Tq allows, not row_tiles a sequence
  int64_t each;                // queries of a sequence without q_offsets
  float* part_o;               // [item][split][R][D]
  float* part_ml;              // [item][split][R][2]
};

// one workgroup's part: its rows and its keys
struct Work {
  int b, h, row0, rows;        // rows: of the sequence and key head in all
  int64_t q0;                  // the sequence's first query
  int first_pos;               // position of its query 0 (negative: more queries than keys)
  int len;
  int lo, hi;                  // keys that some row of the workgroup keeps
  int lo_all, hi_all;          // keys that all its rows keep
};

// a sequence: its first query, its queries in all, how many of them are computed, its tokens
struct Seq {
  int64_t q0, all, n;
  int len;
};

__device__ __forceinline__ Seq find_seq(const AttnLaunch& L, int b) {
  const AttnArgs& a = L.a;
  Seq s;
  s.len = (int)min((int64_t)max(a.lens[b], 0), a.max_kv);
  if (a.q_offsets) {
    s.q0 = a.q_offsets[b];
    s.all = s.q0 < 0 ? 0 : min((int64_t)a.q_offsets[b + 1], a.Tq) - s.q0;
  } else {
    s.all = L.each;
    s.q0 = b * s.all;
  }
  s.n = max(min(s.all, a.max_q), (int64_t)0);
  return s;
}

// rows rt R .. rt R + R - 1 of sequence b
__device__ __forceinline__ bool find_work(const AttnLaunch& L, const Seq& s, int b, int h, int rt, int R, Work& w) {
  const AttnArgs& a = L.a;
  const int64_t rows = s.n * L.G, row0 = (int64_t)rt * R;
  if (row0 >= rows) return false;
  w.b = b; w.h = h; w.row0 = (int)row0; w.rows = (int)rows; w.q0 = s.q0;
  w.len = s.len;
  w.first_pos = w.len - (int)s.all;
  const int i0 = div_by(L.gd, (int)row0), i1 = div_by(L.gd, (int)min(row0 + R, rows) - 1);
  w.lo = w.lo_all = 0;
  w.hi = w.hi_all = w.len;
  if (a.causal) {
    w.hi = max(0, w.first_pos + i1 + 1);
    w.hi_all = w.first_pos + i0 + 1;
    if (a.window > 0) {
      w.lo = max(0, w.first_pos + i0 + 1 - a.window);
      w.lo_all = max(0, w.first_pos + i1 + 1 - a.window);
    }
  }
  return true;
}

// keys [lo, hi) that row r keeps; none for rows behind the last
__device__ __forceinline__ void row_keys(const AttnLaunch& L, const Work& w, int r, int& lo, int& hi) {
  lo = 0; hi = w.len;
  if (L.a.causal) {
    hi = w.first_pos + div_by(L.gd, r) + 1;
    if (L.a.window > 0) lo = hi - L.a.window;
  }
  if (r >= w.rows) hi = 0;
}

// The table's entry for 16-token unit u of sequence b, and the unit's first token in its page. A unit behind the last
// token may be asked for: the table's last entry stands in, and its tokens are masked by the caller.
__device__ __forceinline__ int page_of(const AttnLaunch& L, int b, int u, int& place) {
  const int i = div_by(L.pd, u);
  place = (u - i * (int)L.pd.d) * 16;
  return L.a.table[(int64_t)b * L.a.max_blocks + min((int64_t)i, L.a.max_blocks - 1)];
}
__device__ __forceinline__ bool is_page(const AttnLaunch& L, int p) { return p >= 0 && p < L.a.c.pages; }

__device__ __forceinline__ f16x2 as_f16x2(uint32_t w) { return __builtin_bit_cast(f16x2, w); }

// two E2M1 nibbles of byte SEL times a pair of scales
template <int SEL>
__device__ __forceinline__ uint32_t fp4x2_f16(uint32_t w, f16x2 s) {
  const f16x2 v = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL);
  return __builtin_bit_cast(uint32_t, v * s);
}

// E4M3 bytes HALF * 2 and HALF * 2 + 1 of w
template <bool HALF>
__device__ __forceinline__ f16x2 e4m3x2_f16(uint32_t w) { return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HALF); }

__device__ __forceinline__ f16x8 as_f16x8(u32x4 v) { return __builtin_bit_cast(f16x8, v); }

// eight codes of one token times one scale
__device__ __forceinline__ f16x8 fp4x8_f16(uint32_t w, _Float16 s) {
  const f16x2 ss = {s, s};
  return as_f16x8(u32x4{fp4x2_f16<0>(w, ss), fp4x2_f16<1>(w, ss), fp4x2_f16<2>(w, ss), fp4x2_f16<3>(w, ss)});
}

// Codes of two tokens, nibble by nibble of the same d: byte x of even holds d = 2x (the first token in its low
// nibble), of odd d = 2x + 1. Four instructions for sixteen codes, before they are converted.
__device__ __forceinline__ void pair_tokens(uint32_t t0, uint32_t t1, uint32_t& even, uint32_t& odd) {
  constexpr uint32_t m = 0x0F0F0F0Fu;
  even = (t0 & m) | ((t1 << 4) & ~m);
  odd = ((t0 >> 4) & m) | (t1 & ~m);
}

// two f32 rounded to f16
__device__ __forceinline__ uint32_t pk_f16(float lo, float hi) {
  const f32x2 v = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
}

// What takes a row's sums to its results: m = mantissa(s_h) / sum of the terms, and s_h's power of two last, since s_h / sum
// may lie among f32's subnormals where a result does not. 0 for a row without keys.
struct Finish {
  float m;
  int e;
  __device__ __forceinline__ float operator()(float x) const { return ldexpf(x * m, e); }
};
__device__ __forceinline__ Finish finish(float ts, float sum) {
  Finish f;
  const float m = frexpf(ts, &f.e);
  f.m = sum != 0.f ? m / sum : 0.f;
  return f;
}

// N consecutive values (a multiple of four) of type t at element i
template <int N>
__device__ __forceinline__ void store_run(void* p, int t, int64_t i, const float* x) {
  if (t == kF32) {
#pragma unroll
    for (int u = 0; u < N / 4; ++u) ((f32x4*)((float*)p + i))[u] = f32x4{x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]};
  } else {
    u32x2 w[N / 4];
#pragma unroll
    for (int u = 0; u < N / 2; ++u)
      w[u / 2][u & 1] = t == kBF16 ? pk_bf16_rne(x[2 * u], x[2 * u + 1]) : pk_f16(x[2 * u], x[2 * u + 1]);
#pragma unroll
    for (int u = 0; u < N / 4; ++u) ((u32x2*)((uint16_t*)p + i))[u] = w[u];
  }
}

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Exponent shift that brings a row's largest magnitude into [2^15, 2^16), or as near as 2^127 does (which loses nothing:
// f16 ends at 2^-24, and no bf16 lies below 2^-133); 0 for a row of zeros or not finite.
__device__ __forceinline__ int row_shift(float amax) {
  if (!(amax > 0.f) || !(amax < __builtin_inff())) return 0;
  int e;
  (void)frexpf(amax, &e);                          // amax = f 2^e, f in [1/2, 1)
  return min(16 - e, 127);
}

// scale s_h log2(e) as m 2^e: the product itself may leave f32's range where the queries bring the logits back into it
struct Factor {
  float m;
  int e;
};
__device__ __forceinline__ Factor factor_of(float scale, float ts) {
  int a, b;
  const float m = frexpf(scale, &a) * frexpf(ts, &b) * kLog2e;
  return {m, a + b};
}

// What a row of queries is multiplied by before it is rounded to f16, a power of two with the factor's sign, and what takes
// its products with K_hat to logits in powers of two: 1e-30 at least (not 0, which -inf would turn into NaN; the
// largest sum of products is 2^36). NaN for a row that is not finite: any product with an infinite query is infinite or
// undefined, so its softmax is undefined, and logits of -infinity alone would be taken for keys that it does not
// keep. NaN too where |factor| times the row's largest magnitude is 2^107 or more: below, no sum of 256 products with
// 2688 at most passes 2^127, and a logit is -infinity only where it is masked.
struct RowScale {
  float by, c;
};
__device__ __forceinline__ RowScale row_scale(float amax, const Factor& f) {
  const int sh = row_shift(amax);
  const float c = fminf(fmaxf(ldexpf(fabsf(f.m), f.e - sh), 1e-30f), 0x1p100f);
  return {c * ldexpf(amax, sh) < 0x1p107f ? ldexpf(f.m < 0.f ? -1.f : 1.f, sh) : __builtin_nanf(""), c};
}

// A row's reference as the loops hold it, less 7. They take p = 2^(s c - m) from one FMA, whose m has f32's spacing: from 2^25
// on that alone could lift p beyond f16 or drop the largest term to 0. So where |m| is 2^24 or more, m and c are both
// divided by a power of two, `up`, that leaves |m| below 2^24: terms near the largest then differ by fewer powers of two
// than they should, those whose logits are within some thirty steps (2^-24) of it. `up` follows each new reference (a
// row's first keys may have logits of -2^30 and its later ones of 1).
struct Reference {
  float m = kUnset, c, up = 1.f;
  // raised to the logit of the product s, if that is higher; returns what the sums so far are multiplied by
  __device__ __forceinline__ float raise(float s) {
    const float now = m * up, row = c * up, to = fmaxf(now, s * row - kShift);
    int e = 0;
    if (to > kUnset) (void)frexpf(to, &e);
    const int k = max(e - 24, 0);
    m = ldexpf(to, -k);
    c = ldexpf(row, -k);
    up = ldexpf(1.f, k);
    return exp2_hw(now - to);
  }
};

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// the largest magnitude of packed 16-bit values so far, as bits (those of bf16 and of f16 ascend with the magnitude)
__device__ __forceinline__ uint32_t max_bits(uint32_t m, const u32x4& x) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m), __builtin_bit_cast(u16x2, x[e] & 0x7FFF7FFFu)));
  return m;
}
__device__ __forceinline__ float max_of(uint32_t m, int type) {
  const uint32_t b = max(m & 0xFFFFu, m >> 16);
  return type == kF16 ? f16_of((uint16_t)b) : bf16_of((uint16_t)b);
}

// N packed pairs of type T times a power of two or its negative, as f16
template <int T, int N>
__device__ __forceinline__ void scale_rows(u32x4 (&x)[N], float by) {
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t w = x[j][e];
      const float lo = T == kF16 ? f16_of((uint16_t)w) : bf16_lo(w), hi = T == kF16 ? f16_of((uint16_t)(w >> 16)) : bf16_hi(w);
      x[j][e] = pk_f16(lo * by, hi * by);
    }
}

constexpr int kTileRows = 128;                   // of a workgroup of k_attn_tile
hipError_t launch_attn_tile(const AttnLaunch& L, int64_t groups, hipStream_t s);

}  // namespace ssn
