// Attention over the 4-bit cache for few query rows to a key head: a decoded token, a few tokens to verify.
//
// Bound by reading the cache. A wave walks tiles of 32 tokens; its loads go straight to registers, a tile ahead of
// the arithmetic. With v_mfma_f32_16x16x32_f16 and l the lane:
//   S^T: A = keys. Lane l holds token l % 16 of a half of the tile and d = (DP / 4) (l / 16) + 0 .. DP / 4 - 1, one run
//        of its codes; B = Q, in registers for the wave's whole life, in the same order of d. The result has tokens
//        4 (l / 16) + i of the half for row l % 16.
//   O^T: B = P, eight tokens 16 a + 4 (l / 16) + i (a = 0, 1; i = 0..3) that the lane holds already; A = values: the lane
//        takes those tokens' d = (DP / 16) (l % 16) + 0 .. DP / 16 - 1, one word (two, or half of one) a token, and
//        interleaves two tokens' nibbles before it converts them, so no transposition through LDS is needed.
// The row's maximum is a reference that is raised only where a logit passes it by 2^8: one comparison a tile, and the
// lanes of a row exchange nothing until it happens. Sums of p stay in the lane until the end, in f32.
// The waves of a workgroup take tiles in turn and add their results up in LDS; long sequences are split over
// workgroups, whose f32 results k_attn_join adds up.
#include <algorithm>

#include "attn.hpp"
#include "device_once.hpp"

namespace ssn {
namespace {

// one tile's codes and scales as loaded
template <int DP>
struct Tile {
  static constexpr int KU = DP >= 128 ? DP / 128 : 1;       // 16-byte pieces of keys a lane and half (DP 64: half of one)
  static constexpr int VW = DP == 256 ? 2 : 1;              // words of values a lane and token (DP 64: half of one)
  u32x4 k[2][KU];
  uint32_t ks[2];                                           // the keys' scales: DP / 64 bytes
  uint32_t v[8][VW];                                        // token 4 a + i
  uint32_t vs[2];                                           // the values' scales of four tokens
};

// lane offsets into a 16-token unit of a page
struct LaneAt {
  uint32_t k[2], ks[2], v, vs;
};

template <int DP>
__device__ __forceinline__ LaneAt lane_at(int D, int page, int lane) {
  const int t = lane & 15, c = lane >> 4;
  LaneAt o;
  // lanes whose part lies beyond D read another: the queries are zero there, and no output is written
  const int kd = DP / 4 * c;
  for (int u = 0; u < 2; ++u) {
    const int d = kd + 32 * u < D ? kd + 32 * u : 0;
    o.k[u] = t * (D / 2) + d / 2;
    o.ks[u] = t * (D / 16) + d / 16;
  }
  const int vd = DP / 16 * t < D ? DP / 16 * t : 0;
  o.v = 4 * c * (D / 2) + vd / 2;
  o.vs = (vd / 16) * page + 4 * c;
  return o;
}

template <int DP, int DC>
__device__ __forceinline__ void load_half(Tile<DP>& t, int a, const AttnLaunch& L, int h, int page, int place,
                                          const LaneAt& o) {
  const KvCache& c = L.a.c;
  const int D = DC ? DC : c.D;
  const int64_t head = (int64_t)page * c.heads + h, row = head * c.page + place;
  const uint8_t* kc = c.k_codes + row * (D / 2);
  const uint8_t* ks = c.k_scales + row * (D / 16);
  const uint8_t* vc = c.v_codes + row * (D / 2);
  const uint8_t* vs = c.v_scales + head * (D / 16) * c.page + place;
  if constexpr (DP == 64) {
    const u32x2 k = *(const u32x2*)(kc + o.k[0]);
    t.k[a][0][0] = k[0]; t.k[a][0][1] = k[1];
  } else {
#pragma unroll
    for (int u = 0; u < Tile<DP>::KU; ++u) t.k[a][u] = *(const u32x4*)(kc + o.k[u]);
  }
  if constexpr (DP == 64) t.ks[a] = ks[o.ks[0]];
  else if constexpr (DP == 128) t.ks[a] = *(const uint16_t*)(ks + o.ks[0]);
  else if constexpr (DC == 256) t.ks[a] = *(const uint32_t*)(ks + o.ks[0]);
  else t.ks[a] = *(const uint16_t*)(ks + o.ks[0]) | (uint32_t)*(const uint16_t*)(ks + o.ks[1]) << 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint8_t* p = vc + o.v + i * (D / 2);
    if constexpr (DP == 64) t.v[4 * a + i][0] = *(const uint16_t*)p;
    else if constexpr (DP == 128) t.v[4 * a + i][0] = *(const uint32_t*)p;
    else {
      const u32x2 v = *(const u32x2*)p;
      t.v[4 * a + i][0] = v[0]; t.v[4 * a + i][1] = v[1];
    }
  }
  t.vs[a] = *(const uint32_t*)(vs + o.vs);
}

// scale of dword j (eight codes) of a lane's keys
template <int DP>
__device__ __forceinline__ _Float16 key_scale(const f16x2 (&s)[2], int j) { return s[j / 4][(j / 2) & 1]; }

template <int DP, int NT, int DC, int W>
__global__ __launch_bounds__(64 * W, NT * DP >= 512 ? 1 : 2) void k_attn_stream(AttnLaunch L) {
  constexpr int R = 16 * NT, KS = DP / 32, MV = DP / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kb = lane >> 4;
  const int split = blockIdx.x % L.splits, item = blockIdx.x / L.splits;
  const int rt = item % L.row_tiles, bh = item / L.row_tiles;
  const int h = bh % L.a.c.heads, b = bh / L.a.c.heads;
  const int D = DC ? DC : L.a.c.D;
  Work w;
  if (!find_work(L, b, h, rt, R, w)) return;

  // queries: lane's row col of every 16, d = (DP / 4) kb + 8 j ..
  f16x8 q[NT][KS];
  float c[NT];
  int lo_r[NT], hi_r[NT];
  const float sc = L.a.scale * L.a.c.k_ts[h] * kLog2e;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = w.row0 + 16 * n + col;
    row_keys(L, w, r, lo_r[n], hi_r[n]);
    u32x4 raw[KS];
    const int i = r / L.G;
    const uint16_t* src = (const uint16_t*)L.a.Q + (w.q0 + i) * L.a.q_token + (int64_t)(h * L.G + (r - i * L.G)) * L.a.q_head;
    float amax = 0.f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const int d = DP / 4 * kb + 8 * j;
      raw[j] = r < w.rows && d < D ? *(const u32x4*)(src + d) : u32x4{0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(float16_of((uint16_t)(raw[j][e / 2] >> (16 * (e & 1))), L.a.q_type)));
    }
    amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    const int sh = row_shift(amax);
    const float sign = sc < 0.f ? -1.f : 1.f;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      u32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = pk_f16(sign * ldexpf(float16_of((uint16_t)raw[j][e], L.a.q_type), sh),
                      sign * ldexpf(float16_of((uint16_t)(raw[j][e] >> 16), L.a.q_type), sh));
      q[n][j] = as_f16x8(x);
    }
    c[n] = fmaxf(ldexpf(fabsf(sc), -sh), 1e-30f);   // not 0, which -inf would turn into NaN
  }

  f32x4 o[NT][MV] = {};
  float mc[NT], l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) { mc[n] = kUnset; l[n] = 0.f; }

  // this workgroup's tiles of 32 keys
  const int t0 = w.lo >> 5, t1 = (w.hi + 31) >> 5;
  const int per = (max(t1 - t0, 0) + L.splits - 1) / L.splits;
  const int ta = t0 + split * per, tb = min(t1, ta + per);
  const LaneAt at = lane_at<DP>(D, L.a.c.page, lane);

  Tile<DP> cur, nxt;
  int pg[2] = {}, pn[2] = {}, place[2];
  int t = ta + wave;
  if (t < tb) {
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      pg[a] = page_of(L, b, 2 * t + a, place[a]);
      load_half<DP, DC>(cur, a, L, h, max(pg[a], 0), place[a], at);
    }
  }
  for (; t < tb; t += W) {
    const int tn = t + W;
    if (tn < tb) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        pn[a] = page_of(L, b, 2 * tn + a, place[a]);
        load_half<DP, DC>(nxt, a, L, h, max(pn[a], 0), place[a], at);
      }
    }
    // logits
    f32x4 s[NT][2];
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      f16x2 ks[2];
      ks[0] = e4m3x2_f16<false>(cur.ks[a]);
      ks[1] = e4m3x2_f16<true>(cur.ks[a]);
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const f16x8 k = fp4x8_f16(cur.k[a][j / 4][j % 4], key_scale<DP>(ks, j));
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][j], s[n][a], 0, 0, 0);
      }
    }
    uint32_t vs[2] = {cur.vs[0], cur.vs[1]};
    const bool whole = 32 * t >= w.lo_all && 32 * t + 32 <= w.hi_all && pg[0] >= 0 && pg[1] >= 0;
    if (!whole) {
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 32 * t + 16 * a + 4 * kb + i;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            if (!(pg[a] >= 0 && tok >= lo_r[n] && tok < hi_r[n])) s[n][a][i] = -__builtin_inff();
          // what lies in a slot that no row keeps may be anything: its value's scale becomes 0
          if (!(pg[a] >= 0 && tok >= w.lo && tok < w.hi)) vs[a] &= ~(0xFFu << (8 * i));
        }
    }
    // reference and p
    bool raise = false;
    float top[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n] = s[n][0][0];
#pragma unroll
      for (int i = 1; i < 8; ++i) top[n] = fmaxf(top[n], s[n][i / 4][i % 4]);
      raise |= top[n] * c[n] - mc[n] > kTop;
    }
    if (__any(raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float m = top[n];
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float to = fmaxf(mc[n], m * c[n] - kShift);
        const float f = exp2_hw(mc[n] - to);
        mc[n] = to;
        l[n] *= f;
#pragma unroll
        for (int v = 0; v < MV; ++v) o[n][v] *= f;
      }
    }
    f16x8 p[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = exp2_hw(fmaf(s[n][i / 4][i % 4], c[n], -mc[n]));
        l[n] += e[i];
      }
      p[n] = as_f16x8(u32x4{pk_f16(e[0], e[1]), pk_f16(e[2], e[3]), pk_f16(e[4], e[5]), pk_f16(e[6], e[7])});
    }
    // values
    const f16x2 sv[4] = {e4m3x2_f16<false>(vs[0]), e4m3x2_f16<true>(vs[0]), e4m3x2_f16<false>(vs[1]), e4m3x2_f16<true>(vs[1])};
    uint32_t even[4][Tile<DP>::VW], odd[4][Tile<DP>::VW];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int u = 0; u < Tile<DP>::VW; ++u) pair_tokens(cur.v[2 * x][u], cur.v[2 * x + 1][u], even[x][u], odd[x][u]);
    auto value = [&](auto mi) {
      constexpr int m = decltype(mi)::value, u = m / 8, sel = (m % 8) / 2;
      if constexpr (m < MV) {
        u32x4 x;
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = fp4x2_f16<sel>(m & 1 ? odd[y][u] : even[y][u], sv[y]);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_f16x8(x), p[n], o[n][m], 0, 0, 0);
      }
    };
#define SSN_VALUE(i) value(std::integral_constant<int, i>());
    SSN_VALUE(0) SSN_VALUE(1) SSN_VALUE(2) SSN_VALUE(3) SSN_VALUE(4) SSN_VALUE(5) SSN_VALUE(6) SSN_VALUE(7)
    SSN_VALUE(8) SSN_VALUE(9) SSN_VALUE(10) SSN_VALUE(11) SSN_VALUE(12) SSN_VALUE(13) SSN_VALUE(14) SSN_VALUE(15)
#undef SSN_VALUE
    cur = nxt;
    pg[0] = pn[0]; pg[1] = pn[1];
  }

  // the waves' results brought to one reference and added up, the upper half into the lower until one is left
  __shared__ float sm[W][R], sl[W][R];
  __shared__ f32x4 so[W / 2][NT * MV][64];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
    if (kb == 0) { sm[wave][16 * n + col] = mc[n]; sl[wave][16 * n + col] = l[n]; }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float m = kUnset, sum = 0.f;
#pragma unroll
    for (int x = 0; x < W; ++x) m = fmaxf(m, sm[x][16 * n + col]);
#pragma unroll
    for (int x = 0; x < W; ++x) sum += sl[x][16 * n + col] * exp2_hw(sm[x][16 * n + col] - m);
    const float f = exp2_hw(mc[n] - m);
#pragma unroll
    for (int v = 0; v < MV; ++v) o[n][v] *= f;
    mc[n] = m; l[n] = sum;
  }
#pragma unroll
  for (int half = W / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int x = 0; x < NT * MV; ++x) so[wave - half][x][lane] = o[x / MV][x % MV];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int x = 0; x < NT * MV; ++x) o[x / MV][x % MV] += so[wave][x][lane];
    }
    __syncthreads();
  }
  if (wave) return;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = w.row0 + 16 * n + col;
    if (r >= w.rows) continue;
    if (L.splits > 1) {
      const int64_t at0 = ((int64_t)item * L.splits + split) * R + 16 * n + col;
      if (kb == 0) { L.part_ml[2 * at0] = mc[n]; L.part_ml[2 * at0 + 1] = l[n]; }
      if (!(l[n] != 0.f)) continue;                 // the join skips a part without keys
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < MV; ++v) {
          const int d = MV * (4 * kb + i) + v;
          if (d < D) L.part_o[at0 * D + d] = o[n][v][i];
        }
    } else {
      const int i0 = r / L.G;
      const int64_t head = (w.q0 + i0) * L.a.Hq + h * L.G + (r - i0 * L.G);
      const float f = l[n] != 0.f ? L.a.c.v_ts[h] / l[n] : 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < MV; ++v) {
          const int d = MV * (4 * kb + i) + v;
          if (d < D) store_elem(L.a.out, L.a.out_type, head * D + d, o[n][v][i] * f);
        }
      if (L.a.lse && kb == 0) L.a.lse[head] = l[n] != 0.f ? (mc[n] + log2f(l[n])) * kLn2 : -__builtin_inff();
    }
  }
}

// out = sum over the parts of O 2^(m - M) / sum of l 2^(m - M), one workgroup a row
constexpr int kJoin = 256;
__global__ __launch_bounds__(kJoin) void k_attn_join(AttnLaunch L, int R) {
  const int item = blockIdx.x / R, rl = blockIdx.x % R;
  const int rt = item % L.row_tiles, bh = item / L.row_tiles;
  const int h = bh % L.a.c.heads, b = bh / L.a.c.heads, D = L.a.c.D;
  Work w;
  if (!find_work(L, b, h, rt, R, w)) return;
  const int r = w.row0 + rl;
  if (r >= w.rows) return;
  const int64_t at0 = (int64_t)item * L.splits * R + rl;
  float m = kUnset;
  for (int s = 0; s < L.splits; ++s) m = fmaxf(m, L.part_ml[2 * (at0 + (int64_t)s * R)]);
  float sum = 0.f, acc = 0.f;
  const int d = threadIdx.x;
  for (int s = 0; s < L.splits; ++s) {
    const int64_t at = at0 + (int64_t)s * R;
    const float l = L.part_ml[2 * at + 1], f = exp2_hw(L.part_ml[2 * at] - m);
    if (!(l != 0.f)) continue;
    sum += l * f;
    if (d < D) acc += L.part_o[at * D + d] * f;
  }
  const int i0 = r / L.G;
  const int64_t head = (w.q0 + i0) * L.a.Hq + h * L.G + (r - i0 * L.G);
  if (d < D) store_elem(L.a.out, L.a.out_type, head * D + d, sum != 0.f ? acc * (L.a.c.v_ts[h] / sum) : 0.f);
  if (L.a.lse && d == 0) L.a.lse[head] = sum != 0.f ? (m + log2f(sum)) * kLn2 : -__builtin_inff();
}

constexpr int kWaves = 4;

struct Shape {
  int R, row_tiles, splits;
  int64_t items;
};

// Rows of a workgroup: the fewest of 16, 32 and (up to a width of 128) 64 that hold a sequence's rows. Splits: some 16 waves a compute unit,
// each with four tiles at least.
Shape shape_of(const AttnArgs& a) {
  Shape s;
  const int64_t rows = a.max_q * (a.Hq / a.c.heads);
  s.R = rows <= 16 ? 16 : rows <= 32 || a.c.D > 128 ? 32 : 64;
  s.row_tiles = (int)((rows + s.R - 1) / s.R);
  s.items = a.B * a.c.heads * s.row_tiles;
  const int64_t tiles = (a.max_kv + 31) / 32;
  const int64_t want = (4 * (int64_t)cu_count() + s.items - 1) / s.items;
  s.splits = (int)std::max<int64_t>(1, std::min(want, tiles / (4 * kWaves)));
  return s;
}

template <int DP, int DC>
void launch(const AttnLaunch& L, const Shape& s, hipStream_t st) {
  const dim3 grid((unsigned)(s.items * s.splits)), block(64 * kWaves);
  if (s.R == 16) hipLaunchKernelGGL((k_attn_stream<DP, 1, DC, kWaves>), grid, block, 0, st, L);
  else if (s.R == 32) hipLaunchKernelGGL((k_attn_stream<DP, 2, DC, kWaves>), grid, block, 0, st, L);
  else if constexpr (DP <= 128) hipLaunchKernelGGL((k_attn_stream<DP, 4, DC, kWaves>), grid, block, 0, st, L);
}

}  // namespace

int64_t attn_workspace(const AttnArgs& a) {
  const Shape s = shape_of(a);
  return s.splits > 1 ? s.items * s.splits * s.R * (a.c.D + 2) * 4 : 0;
}

int64_t attn_workgroups(const AttnArgs& a) {
  const Shape s = shape_of(a);
  return s.items * s.splits;
}

hipError_t launch_attn_stream(const AttnArgs& a, hipStream_t st) {
  const Shape s = shape_of(a);
  AttnLaunch L;
  L.a = a;
  L.pd = page_div((uint32_t)(a.c.page / 16));
  L.G = a.Hq / a.c.heads;
  L.row_tiles = s.row_tiles;
  L.splits = s.splits;
  L.part_o = (float*)a.ws;
  L.part_ml = L.part_o + (s.splits > 1 ? s.items * s.splits * s.R * a.c.D : 0);
  const int D = a.c.D;
  if (D == 64) launch<64, 64>(L, s, st);
  else if (D < 64) launch<64, 0>(L, s, st);
  else if (D == 128) launch<128, 128>(L, s, st);
  else if (D < 128) launch<128, 0>(L, s, st);
  else if (D == 256) launch<256, 256>(L, s, st);
  else launch<256, 0>(L, s, st);
  if (s.splits > 1) hipLaunchKernelGGL(k_attn_join, dim3((unsigned)(s.items * s.R)), dim3(kJoin), 0, st, L, s.R);
  return hipGetLastError();
}

}  // namespace ssn
