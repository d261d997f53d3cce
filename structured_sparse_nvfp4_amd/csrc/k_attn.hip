// Attention over the 4-bit cache for few query rows to a key head: a decoded token, a few tokens to verify.
//
// A wave walks tiles of 32 tokens; its loads go straight to registers and are replaced in place as they are used, so
// what is loaded has a tile's time to arrive. With v_mfma_f32_16x16x32_f16 and l the lane:
//   S^T: A = keys. Lane l holds token l % 16 of a half of the tile and d = (DP / 4) (l / 16) + 0 .. DP / 4 - 1, one run
//        of its codes; B = Q, in registers for the wave's whole life, in the same order of d. The result has tokens
//        4 (l / 16) + i of the half for row l % 16.
//   O^T: B = P, eight tokens 16 a + 4 (l / 16) + i (a = 0, 1; i = 0..3) that the lane holds already; A = values: the lane
//        takes those tokens' d = (DP / 16) (l % 16) + 0 .. DP / 16 - 1, one word (two, or half of one) a token, and
//        interleaves two tokens' nibbles before it converts them, so no transposition through LDS is needed.
// The row's maximum is a reference that is raised only where a logit passes it by 2^8: one comparison a tile, and the
// lanes of a row exchange nothing until it happens. Sums of p stay in the lane until the end, in f32.
// The waves of a workgroup take tiles in turn and meet in LDS; long sequences are split over workgroups, whose f32
// results k_attn_join adds up.
//
// Measured (kernels, D = 128): 32 sequences of 2048 to 8191 keys x 8 heads, 5 queries each, 183 MB of cache in 41 us (4.5
// TB/s) and 4.8 more to join them; one of 131072 x 8 heads, 151 MB in 31.4 (4.8 TB/s) and 6.3; one of 1000 x 2 heads
// 9.9. A tile has 16 matrix instructions and some 250 vector ones, 128 of them to make operands of codes; at the first of
// these the vector units issue 0.52 of the time, a wave waits 0.27 of its own for memory and 0.45 for its turn: not
// memory, which streams 6.3 TB/s and more where it is only read, but the waves' turns bound it. The rest is the start
// (sequence, page, keys: three dependent reads, some 7 us) and sequences of unequal length. Tried without gain: parts of
// one size however long the sequences are (46 -> 48 us, and 56 where parts cross them), 64 tokens a step, one page a
// tile, heads of one XCD next to each other.
#include <algorithm>
#include <type_traits>

#include "attn.hpp"
#include "device_once.hpp"
#include "pipeline.hpp"

namespace ssn {
namespace {

// The codes and scales of 16 tokens as loaded. (Types as wide as the loads: widened at the load they would be waited
// for there.)
template <int DP>
struct Unit {
  using KeyScales = std::conditional_t<DP == 64, uint8_t, std::conditional_t<DP == 128, uint16_t, u32x2>>;
  using ValueWord = std::conditional_t<DP == 64, uint16_t, uint32_t>;
  static constexpr int KU = DP >= 128 ? DP / 128 : 1;       // 16-byte pieces of keys a lane (DP 64: half of one)
  static constexpr int VW = DP == 256 ? 2 : 1;              // words of values a lane and token (DP 64: half of one)
  u32x4 k[KU];
  KeyScales ks;                                             // DP / 64 bytes
  ValueWord v[4][VW];                                       // token 4 (l / 16) + i
  uint32_t vs;                                              // scales of the four
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

// Where a unit lies: its first token's row of the codes (and of the keys' scales), and of the values' scales.
struct Place {
  int64_t row, vs;
};

// A wave-uniform base in a buffer resource and a lane offset that never changes: a load costs no vector instruction
// but itself.
template <int DP, int DC>
__device__ __forceinline__ void load_keys(Unit<DP>& t, const KvCache& c, const Place& p, const LaneAt& o) {
  const int D = DC ? DC : c.D;
  const auto kc = buf_rsrc(c.k_codes + p.row * (D / 2)), ks = buf_rsrc(c.k_scales + p.row * (D / 16));
  if constexpr (DP == 64) {
    const auto k = __builtin_amdgcn_raw_buffer_load_b64(kc, o.k[0], 0, 0);
    t.k[0][0] = k[0]; t.k[0][1] = k[1];
    t.ks = __builtin_amdgcn_raw_buffer_load_b8(ks, o.ks[0], 0, 0);
  } else {
#pragma unroll
    for (int u = 0; u < Unit<DP>::KU; ++u) t.k[u] = __builtin_amdgcn_raw_buffer_load_b128(kc, o.k[u], 0, 0);
    if constexpr (DP == 128) t.ks = __builtin_amdgcn_raw_buffer_load_b16(ks, o.ks[0], 0, 0);
    else if constexpr (DC == 256) t.ks[0] = __builtin_amdgcn_raw_buffer_load_b32(ks, o.ks[0], 0, 0);
    else {
      t.ks[0] = __builtin_amdgcn_raw_buffer_load_b16(ks, o.ks[0], 0, 0);
      t.ks[1] = __builtin_amdgcn_raw_buffer_load_b16(ks, o.ks[1], 0, 0);
    }
  }
}

template <int DP, int DC>
__device__ __forceinline__ void load_values(Unit<DP>& t, const KvCache& c, const Place& p, const LaneAt& o) {
  const int D = DC ? DC : c.D;
  const auto vc = buf_rsrc(c.v_codes + p.row * (D / 2)), vs = buf_rsrc(c.v_scales + p.vs);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t at = o.v + i * (D / 2);
    if constexpr (DP == 64) t.v[i][0] = __builtin_amdgcn_raw_buffer_load_b16(vc, at, 0, 0);
    else if constexpr (DP == 128) t.v[i][0] = __builtin_amdgcn_raw_buffer_load_b32(vc, at, 0, 0);
    else {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(vc, at, 0, 0);
      t.v[i][0] = v[0]; t.v[i][1] = v[1];
    }
  }
  t.vs = __builtin_amdgcn_raw_buffer_load_b32(vs, o.vs, 0, 0);
}

// f(0) .. f(N - 1) with constants
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>());
    each<N, I + 1>(f);
  }
}

constexpr int TU = 2, TT = 16 * TU;               // units of 16 tokens of a tile, and its tokens

template <int DP, int NT, int DC, int W>
__global__ __launch_bounds__(64 * W, W > 4 ? W / 4 : NT * DP >= 512 ? 1 : NT * DP <= 128 ? 4 : 2) void k_attn_stream(AttnLaunch L) {
  constexpr int R = 16 * NT, KS = DP / 32, MV = DP / 16;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kb = lane >> 4;
  const int D = DC ? DC : L.a.c.D;
  constexpr int SLOTS = NT == 3 ? W / 2 : W;
  __shared__ f32x2 sml[SLOTS][R];
  __shared__ __attribute__((aligned(16))) float so[SLOTS][R][DP + 4];
  // Heads first, then row sets: with eight heads (or a multiple) the row sets of one part of the keys share an L2.
  const int h = blockIdx.x, b = blockIdx.z, split = div_by(L.td, blockIdx.y);
  const int rt = blockIdx.y - split * L.row_tiles;
  Work w;
  if (!find_work(L, find_seq(L, b), b, h, rt, R, w)) return;
  const int t0 = w.lo / TT, t1 = (w.hi + TT - 1) / TT;
  const int per = div_by(L.sd, max(t1 - t0, 0) + L.splits - 1);
  const int ta = t0 + split * per, tb = min(t1, ta + per);

  // queries: lane's row col of every 16, d = (DP / 4) kb + 8 j ..
  f16x8 q[NT][KS];
  Reference ref[NT];
  int lo_r[NT], hi_r[NT];
  const Factor factor = factor_of(L.a.scale, L.a.c.k_ts[h]);
  u32x4 raw[NT][KS];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = w.row0 + 16 * n + col, rr = min(r, w.rows - 1), i = div_by(L.gd, rr);
    row_keys(L, w, r, lo_r[n], hi_r[n]);
    const uint16_t* src = (const uint16_t*)L.a.Q + (w.q0 + i) * L.a.q_token + (int64_t)(h * L.G + (rr - i * L.G)) * L.a.q_head;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      const int d = DP / 4 * kb + 8 * j;
      raw[n][j] = *(const u32x4*)(src + (DC || d < D ? d : 0));
    }
  }

  const LaneAt at = lane_at<DP>(D, L.a.c.page, lane);
  struct Pages {
    int p[TU], place[TU];
  };
  // The pages of tile t, or of the last one: every load is made, so that the waits can count them.
  auto pages_of = [&](int t) {
    Pages p;
#pragma unroll
    for (int a = 0; a < TU; ++a) p.p[a] = page_of(L, b, TU * min(t, tb - 1) + a, p.place[a]);
    return p;
  };
  auto place_of = [&](const Pages& p, Place (&to)[TU], bool (&there)[TU]) {
#pragma unroll
    for (int a = 0; a < TU; ++a) {
      there[a] = is_page(L, p.p[a]);
      const int64_t head = (int64_t)(there[a] ? p.p[a] : 0) * L.a.c.heads + h;
      to[a].row = head * L.a.c.page + p.place[a];
      to[a].vs = head * (D / 16) * L.a.c.page + p.place[a];
    }
  };
  Unit<DP> un[TU];
  Pages pg;
  Place pl[TU];
  bool there[TU], there_next[TU];
  int t = ta + wave;
  if (t < tb) {
    pg = pages_of(t);
    place_of(pg, pl, there);
    pg = pages_of(t + W);
    each<TU>([&](auto u) { load_keys<DP, DC>(un[u], L.a.c, pl[u], at); });
    each<TU>([&](auto u) { load_values<DP, DC>(un[u], L.a.c, pl[u], at); });
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const bool row = w.row0 + 16 * n + col < w.rows;
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < KS; ++j) {
      if (!row || (!DC && DP / 4 * kb + 8 * j >= D)) raw[n][j] = u32x4{0, 0, 0, 0};
      m = max_bits(m, raw[n][j]);
    }
    float amax = max_of(m, L.a.q_type);
    amax = fmaxf(amax, __shfl_xor(amax, 16, 64));
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    const RowScale scale = row_scale(amax, factor);
    if (L.a.q_type == kBF16) scale_rows<kBF16>(raw[n], scale.by);
    else scale_rows<kF16>(raw[n], scale.by);
#pragma unroll
    for (int j = 0; j < KS; ++j) q[n][j] = as_f16x8(raw[n][j]);
    ref[n].c = scale.c;
  }

  f32x4 o[NT][MV] = {};
  float l[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) l[n] = 0.f;

  // A tile's keys are replaced by the next tile's as soon as its logits are formed, its values when they are used: what
  // is loaded has a tile's time to arrive.
  for (; t < tb; t += W) {
    f32x4 s[NT][TU];
#pragma unroll
    for (int a = 0; a < TU; ++a) {
      f16x2 ks[2];
      if constexpr (DP == 256) {
        ks[0] = e4m3x2_f16<false>(un[a].ks[0]);
        ks[1] = DC ? e4m3x2_f16<true>(un[a].ks[0]) : e4m3x2_f16<false>(un[a].ks[1]);
      } else {
        ks[0] = e4m3x2_f16<false>(un[a].ks);
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) s[n][a] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < KS; ++j) {
        const f16x8 k = fp4x8_f16(un[a].k[j / 4][j % 4], ks[j / 4][(j / 2) & 1]);
#pragma unroll
        for (int n = 0; n < NT; ++n) s[n][a] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k, q[n][j], s[n][a], 0, 0, 0);
      }
    }
    place_of(pg, pl, there_next);
    pg = pages_of(t + 2 * W);
    each<TU>([&](auto u) { load_keys<DP, DC>(un[u], L.a.c, pl[u], at); });
    bool whole = TT * t >= w.lo_all && TT * t + TT <= w.hi_all;
#pragma unroll
    for (int a = 0; a < TU; ++a) whole = whole && there[a];
    if (!whole) {
#pragma unroll
      for (int a = 0; a < TU; ++a)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = TT * t + 16 * a + 4 * kb + i, in = there[a] ? -1 : 0;
#pragma unroll
          for (int n = 0; n < NT; ++n) s[n][a][i] = ((tok >= lo_r[n]) & (tok < hi_r[n]) & in) ? s[n][a][i] : -__builtin_inff();
          // what lies in a slot that no row keeps may be anything: its value's scale becomes 0
          un[a].vs &= ((tok >= w.lo) & (tok < w.hi) & in) ? ~0u : ~(0xFFu << (8 * i));
        }
    }
    // reference and p
    bool raise = false;
    float top[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      top[n] = s[n][0][0];
#pragma unroll
      for (int i = 1; i < 4 * TU; ++i) top[n] = fmaxf(top[n], s[n][i / 4][i % 4]);
      raise |= top[n] * ref[n].c - ref[n].m > kTop;
    }
    if (__any(raise)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float m = top[n];
        m = fmaxf(m, __shfl_xor(m, 16, 64));
        m = fmaxf(m, __shfl_xor(m, 32, 64));
        const float f = ref[n].raise(m);
        l[n] *= f;
#pragma unroll
        for (int v = 0; v < MV; ++v) o[n][v] *= f;
      }
    }
    f16x8 p[NT][TU / 2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int a = 0; a < TU / 2; ++a) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          e[i] = exp2_hw(fmaf(s[n][2 * a + i / 4][i % 4], ref[n].c, -ref[n].m));
          l[n] += e[i];
        }
        p[n][a] = as_f16x8(u32x4{pk_f16(e[0], e[1]), pk_f16(e[2], e[3]), pk_f16(e[4], e[5]), pk_f16(e[6], e[7])});
      }
    // values, 32 tokens at a time
    each<TU / 2>([&](auto a) {
      const f16x2 sv[4] = {e4m3x2_f16<false>(un[2 * a].vs), e4m3x2_f16<true>(un[2 * a].vs),
                           e4m3x2_f16<false>(un[2 * a + 1].vs), e4m3x2_f16<true>(un[2 * a + 1].vs)};
      uint32_t even[4][Unit<DP>::VW], odd[4][Unit<DP>::VW];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int u = 0; u < Unit<DP>::VW; ++u)
          pair_tokens(un[2 * a + x / 2].v[2 * (x & 1)][u], un[2 * a + x / 2].v[2 * (x & 1) + 1][u], even[x][u], odd[x][u]);
      each<MV>([&](auto m) {
        constexpr int u = m / 8, sel = (m % 8) / 2;
        u32x4 x;
#pragma unroll
        for (int y = 0; y < 4; ++y) x[y] = fp4x2_f16<sel>(m & 1 ? odd[y][u] : even[y][u], sv[y]);
#pragma unroll
        for (int n = 0; n < NT; ++n) o[n][m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(as_f16x8(x), p[n][a], o[n][m], 0, 0, 0);
      });
    });
    each<TU>([&](auto u) { load_values<DP, DC>(un[u], L.a.c, pl[u], at); });
#pragma unroll
    for (int a = 0; a < TU; ++a) there[a] = there_next[a];
  }

  // The waves' results meet in LDS, rows of D padded so that 16 lanes' pieces lie in different banks; then each thread
  // adds up four d of a row over the waves, brought to their common reference. Where all of them would leave LDS for
  // one workgroup a CU only (NT 3), the upper half of the waves goes into the lower first.
  float mc[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    l[n] += __shfl_xor(l[n], 16, 64);
    l[n] += __shfl_xor(l[n], 32, 64);
    mc[n] = ref[n].m * ref[n].up;
  }
  auto put = [&](int to) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (kb == 0) sml[to][16 * n + col] = f32x2{mc[n], l[n]};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < MV; v += 4)
          *(f32x4*)&so[to][16 * n + col][MV * (4 * kb + i) + v] = f32x4{o[n][v][i], o[n][v + 1][i], o[n][v + 2][i], o[n][v + 3][i]};
    }
  };
  if constexpr (SLOTS < W) {
    if (wave >= SLOTS) put(wave - SLOTS);
    __syncthreads();
    if (wave < SLOTS) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const f32x2 ml = sml[wave][16 * n + col];
        const float m = fmaxf(mc[n], ml[0]), f = exp2_hw(mc[n] - m), g = exp2_hw(ml[0] - m);
        mc[n] = m;
        l[n] = l[n] * f + ml[1] * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int v = 0; v < MV; v += 4) {
            const f32x4 x = *(const f32x4*)&so[wave][16 * n + col][MV * (4 * kb + i) + v];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][v + e][i] = o[n][v + e][i] * f + x[e] * g;
          }
      }
      put(wave);
    }
  } else {
    put(wave);
  }
  __syncthreads();
  const int D4 = D / 4;
  for (int e = threadIdx.x; e < R * D4; e += 64 * W) {
    const int row = e / D4, d = 4 * (e - row * D4), r = w.row0 + row;
    if (r >= w.rows) break;
    float m = kUnset, sum = 0.f;
    f32x2 ml[SLOTS];
#pragma unroll
    for (int x = 0; x < SLOTS; ++x) { ml[x] = sml[x][row]; m = fmaxf(m, ml[x][0]); }
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int x = 0; x < SLOTS; ++x) {
      const float f = exp2_hw(ml[x][0] - m);
      sum += ml[x][1] * f;
      acc += *(const f32x4*)&so[x][row][d] * f;
    }
    const bool any = sum != 0.f;
    if (L.splits > 1) {
      const int64_t part = ((((int64_t)b * L.a.c.heads + h) * L.row_tiles + rt) * L.splits + split) * R + row;
      if (d == 0) *(f32x2*)(L.part_ml + 2 * part) = f32x2{m, sum};
      if (any) *(f32x4*)(L.part_o + part * D + d) = acc;      // the join skips a part without keys
    } else {
      const int i = div_by(L.gd, r);
      const int64_t head = (w.q0 + i) * L.a.Hq + h * L.G + (r - i * L.G);
      const Finish f = finish(L.a.c.v_ts[h], sum);
      const float x[4] = {f(acc[0]), f(acc[1]), f(acc[2]), f(acc[3])};
      store_run<4>(L.a.out, L.a.out_type, head * D + d, x);
      if (L.a.lse && d == 0) L.a.lse[head] = any ? (m + log2f(sum)) * kLn2 : -__builtin_inff();
    }
  }
}

// out = sum over the parts of O 2^(m - M) / sum of l 2^(m - M), bound by its launch and two dependent reads. TR lanes share
// a row (a wave; four or sixteen from 17 and 65 parts on: with one wave 128 parts of 64 rows take 8 us longer): a lane
// takes four d of every G-th part, and its loads wait for nothing but the row's number. 4.7 us for 4 parts of 1280 rows of
// 128, 6.6 for 4 of 5760, 6.4 for 128 of 64.
constexpr int kMaxSplits = 256;
template <int TR>
__global__ __launch_bounds__(TR == 64 ? 256 : TR) void k_attn_join(AttnLaunch L, int R, int max_rows) {
  constexpr int RW = TR == 64 ? 4 : 1, NS = kMaxSplits / 64, U = 4;
  const int t = threadIdx.x % TR, rw = threadIdx.x / TR, lane = threadIdx.x & 63;
  const int64_t id = (int64_t)blockIdx.x * RW + rw;
  const int bh = (int)(id / max_rows), r = (int)(id - (int64_t)bh * max_rows);
  const int h = bh % L.a.c.heads, b = bh / L.a.c.heads, D = L.a.c.D;
  const Seq seq = find_seq(L, min(b, (int)L.a.B - 1));
  const bool live = b < L.a.B && r < seq.n * L.G;
  __shared__ f32x4 acc[RW][TR];
  const int rt = live ? r / R : 0, splits = live ? L.splits : 0;
  const int64_t at0 = live ? ((int64_t)bh * L.row_tiles + rt) * splits * R + (r - rt * R) : 0;
  // m and l of part s in lane s % 64
  float m[NS], l[NS], top = kUnset, sum = 0.f;
  const int ns = (splits + 63) / 64;
#pragma unroll
  for (int x = 0; x < NS; ++x) {
    m[x] = kUnset; l[x] = 0.f;
    if (x < ns && 64 * x + lane < splits) {
      const f32x2 ml = *(const f32x2*)(L.part_ml + 2 * (at0 + (int64_t)(64 * x + lane) * R));
      m[x] = ml[0]; l[x] = ml[1];
    }
  }
  const int D4 = D / 4, groups = TR / D4, g = t / D4, d = 4 * (t - g * D4);
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  const float* src = L.part_o + at0 * D + d;
  f32x4 first[U];
#pragma unroll
  for (int u = 0; u < U; ++u) first[u] = g < groups && g + u * groups < splits ? *(const f32x4*)(src + (int64_t)(g + u * groups) * R * D) : o;
#pragma unroll
  for (int x = 0; x < NS; ++x) top = fmaxf(top, m[x]);
#pragma unroll
  for (int x = 1; x < 64; x *= 2) top = fmaxf(top, __shfl_xor(top, x, 64));
#pragma unroll
  for (int x = 0; x < NS; ++x) {
    m[x] = l[x] != 0.f ? exp2_hw(m[x] - top) : 0.f;     // a part without keys wrote no O: its factor 0 drops what is read
    if (m[x] != 0.f) sum += l[x] * m[x];
  }
#pragma unroll
  for (int x = 1; x < 64; x *= 2) sum += __shfl_xor(sum, x, 64);
  auto factor = [&](int s) {
    float f = __shfl(m[0], s & 63, 64);
#pragma unroll
    for (int x = 1; x < NS; ++x)
      if (x < ns) { const float y = __shfl(m[x], s & 63, 64); if (s / 64 == x) f = y; }
    return f;
  };
  for (int s0 = 0; s0 < splits; s0 += U * groups) {
    f32x4 next[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = s0 + g + (u + U) * groups;
      next[u] = g < groups && s < splits ? *(const f32x4*)(src + (int64_t)s * R * D) : f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float f = factor(min(s0 + g + u * groups, splits - 1));
      if (f != 0.f && s0 + g + u * groups < splits) o += first[u] * f;
      first[u] = next[u];
    }
  }
  acc[rw][t] = o;
  __syncthreads();
  if (!live || t >= D4) return;
  for (int x = 1; x < groups; ++x) o += acc[rw][t + x * D4];
  const int i0 = div_by(L.gd, r);
  const int64_t head = (seq.q0 + i0) * L.a.Hq + h * L.G + (r - i0 * L.G);
  const Finish f = finish(L.a.c.v_ts[h], sum);
  const float x[4] = {f(o[0]), f(o[1]), f(o[2]), f(o[3])};
  store_run<4>(L.a.out, L.a.out_type, head * D + d, x);
  if (L.a.lse && t == 0) L.a.lse[head] = sum != 0.f ? (top + log2f(sum)) * kLn2 : -__builtin_inff();
}

constexpr int kWaves = 4, kMoreWaves = 8;

struct Shape {
  int R, row_tiles, splits, waves;
  int64_t items;
};

// STREAM. A workgroup's rows: one set of up to 48 where that holds a sequence's rows (at 45 of them 33 us; as sets of 16
// 100 against 80 at 48 rows of 32 sequences to 8191 keys), two of 32 for 49 to 64 (96 us; four of 16 115, two of 48
// 113), two of 48 for 65 to 96 (115 at 80; three of 32 139, five of 16 146): a set more decodes the keys and values again, a
// larger one leaves fewer waves. Beyond a width of 128 sets of 16 or 32 (32 rows: 44.9, two of 16 45.4). Rows that share
// keys come next to each other on one XCD, whose L2 serves the second.
// Splits: as many workgroups as the card holds at once, `resident` a CU by registers and LDS. Half of it 46.0 -> 48.8
// us (32 sequences to 8191 keys), 33.0 -> 36.6 (16 x 9 tokens), twice 49.8 and 41.0. Down to a tile a wave as long as
// that gives each CU a workgroup (one sequence of 4096 keys 9.7 us, 11.3 with kMinTiles alone, 2048 9.4 and 11.2),
// kMinTiles a wave beyond (8 sequences of 4096 keys: 14.7; with two 15.5, with eight 16.8).
// Few short sequences: one workgroup of eight waves each and no join, which saves the call a launch (1000 keys: 10.0 us
// in the kernel, 9.2 as two, of the call's 14; 2048 keys 14.7 against 9.4, so not beyond kShort tiles; sixteen waves 10.5).
// MFMA: 128 rows; splits likewise, of a workgroup's tiles.
constexpr int kMinTiles = 4, kShort = 32;
Shape shape_of(const AttnArgs& a, bool tile) {
  Shape s;
  const int64_t rows = a.max_q * (a.Hq / a.c.heads);
  const int wide = a.c.D > 128 ? 2 : 1;
  const int nt = wide == 2 ? (rows > 16 ? 2 : 1) : rows > 64 ? 3 : rows > 48 ? 2 : (int)((rows + 15) / 16);
  s.R = tile ? kTileRows : 16 * nt;
  s.row_tiles = (int)((rows + s.R - 1) / s.R);
  s.items = a.B * a.c.heads * s.row_tiles;
  // keys that a workgroup's rows can keep
  const int64_t keys = a.window > 0 ? std::min<int64_t>(a.max_kv, (int64_t)a.window + s.R + 31) : a.max_kv;
  const int64_t tiles = (keys + 31) / 32;
  const int resident = tile ? (wide == 1 ? 3 : 2) : nt * wide >= 4 ? 1 : nt * wide >= 2 ? 2 : 4;
  const int64_t want = (resident * (int64_t)cu_count() + s.items / 2) / s.items;
  const int64_t most = std::max<int64_t>(tiles / (kMinTiles * kWaves), std::min<int64_t>(tiles / kWaves, cu_count() / s.items));
  s.waves = kWaves;
  s.splits = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(want, kMaxSplits), most));
  if (!tile && nt == 1 && s.items < cu_count() && tiles <= kShort) {
    s.waves = kMoreWaves;
    s.splits = 1;
  }
  return s;
}

int64_t workspace_of(const AttnArgs& a, const Shape& s) {
  return s.splits > 1 ? s.items * s.splits * s.R * (a.c.D + 2) * 4 : 0;
}

template <int DP, int DC>
void launch(const AttnLaunch& L, const Shape& s, hipStream_t st) {
  const dim3 grid((unsigned)L.a.c.heads, (unsigned)(s.row_tiles * s.splits), (unsigned)L.a.B), block(64 * s.waves);
  if (s.waves == kMoreWaves) hipLaunchKernelGGL((k_attn_stream<DP, 1, DC, kMoreWaves>), grid, block, 0, st, L);
  else if (s.R == 16) hipLaunchKernelGGL((k_attn_stream<DP, 1, DC, kWaves>), grid, block, 0, st, L);
  else if (s.R == 32) hipLaunchKernelGGL((k_attn_stream<DP, 2, DC, kWaves>), grid, block, 0, st, L);
  else if constexpr (DP <= 128) hipLaunchKernelGGL((k_attn_stream<DP, 3, DC, kWaves>), grid, block, 0, st, L);
}

}  // namespace

// The tiles where a sequence has more rows than two sets of the stream, or one of the wide, hold. 32 sequences to 8191
// keys: 96 rows 115 us streamed, 136 as tiles, 104 rows 168 and 149; D = 64: 96 rows 84 and 93, 104 rows 110 and
// 100; D = 256, 8 sequences of 16384: 32 rows 45 and 68, 36 rows 70 and 71, 64 rows 72 and 76. One sequence of 4096 keys
// with 128 rows has too few workgroups for either (20 and 24).
bool attn_takes_tile(const AttnArgs& a) { return a.max_q * (a.Hq / a.c.heads) > (a.c.D > 128 ? 32 : 96); }

int64_t attn_workspace(const AttnArgs& a) {
  return std::max(workspace_of(a, shape_of(a, false)), workspace_of(a, shape_of(a, true)));
}

// Workgroups: row_tiles a sequence, or, where those are too many, the tiles that Tq queries can have (find_item).
bool tiles_owned(const AttnArgs& a, const Shape& s, bool tile) { return tile && s.items * s.splits > kAttnGrid; }
int64_t workgroups_of(const AttnArgs& a, const Shape& s, bool tile) {
  if (!tiles_owned(a, s, tile)) return s.items * s.splits;
  return (a.Tq * (a.Hq / a.c.heads) / kTileRows + a.B) * a.c.heads * s.splits;
}
int64_t attn_workgroups(const AttnArgs& a, bool tile) { return workgroups_of(a, shape_of(a, tile), tile); }

hipError_t launch_attn(const AttnArgs& a, bool tile, hipStream_t st) {
  const Shape s = shape_of(a, tile);
  AttnLaunch L;
  L.a = a;
  L.pd = divisor((uint32_t)(a.c.page / 16));
  L.G = a.Hq / a.c.heads;
  L.gd = divisor((uint32_t)L.G);
  L.td = divisor((uint32_t)s.row_tiles);
  L.sd = divisor((uint32_t)s.splits);
  L.each = a.q_offsets ? 0 : a.Tq / a.B;
  L.row_tiles = s.row_tiles;
  L.owned = tiles_owned(a, s, tile);
  L.splits = s.splits;
  L.part_o = (float*)a.ws;
  L.part_ml = L.part_o + (s.splits > 1 ? s.items * s.splits * s.R * a.c.D : 0);
  const int D = a.c.D;
  if (tile) {
    const hipError_t e = launch_attn_tile(L, workgroups_of(a, s, tile), st);
    if (e != hipSuccess) return e;
  } else if (D == 64) launch<64, 64>(L, s, st);
  else if (D < 64) launch<64, 0>(L, s, st);
  else if (D == 128) launch<128, 128>(L, s, st);
  else if (D < 128) launch<128, 0>(L, s, st);
  else if (D == 256) launch<256, 256>(L, s, st);
  else launch<256, 0>(L, s, st);
  if (s.splits > 1) {
    const int max_rows = (int)(a.max_q * L.G);
    const int64_t rows = a.B * a.c.heads * max_rows;
    if (s.splits > 64) hipLaunchKernelGGL((k_attn_join<1024>), dim3((unsigned)rows), dim3(1024), 0, st, L, s.R, max_rows);
    else if (s.splits > 16) hipLaunchKernelGGL((k_attn_join<256>), dim3((unsigned)rows), dim3(256), 0, st, L, s.R, max_rows);
    else hipLaunchKernelGGL((k_attn_join<64>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, st, L, s.R, max_rows);
  }
  return hipGetLastError();
}

}  // namespace ssn
