// Attention over the 4-bit cache for many query rows to a key head: prompts and chunks of prompts.
//
// A workgroup takes 32 rows a wave and walks tiles of TK keys: all its threads decode a tile's keys and values once, to
// f16 in LDS, while the loads of the next tile are in flight; two buffers, one barrier a tile. With v_mfma_f32_32x32x16_f16, l the lane and h = l / 32:
//   S^T: A = keys from LDS (token l % 32, d = 16 s + 8 h ..), B = Q from registers. The result has token
//        8 (i / 4) + 4 h + i % 4 of 32 in register i, row l % 32.
//   O^T: B = P, the lane's own eight tokens of every 16 (8 (x / 4) + 4 h + x % 4); A = values, stored transposed and in
//        that order of tokens, so an operand is one 16-byte read. Row p of tile m is d = (DP / 32) p + m, which gives the
//        decoding threads, eight d of four tokens each, rows whose LDS banks do not meet (rows are 16 bytes longer than
//        their data for that), and a lane of the result runs of DP / 8 consecutive d.
//
// Measured: a prompt of 8192 tokens x 40 heads (8 of keys), D = 128, causal, 709 us (970 TFLOP/s; a large matrix product
// reaches 1145 to 1158 on this card), 7 chunks of 214 to 1500 queries over 2251 to 9001 keys, 16 heads (4), D = 256, 520 us (855).
// Bound by the matrix cores and the vector units together: at D = 128 a wave's tile of 32 keys has 16 matrix
// instructions, 526 clocks of a SIMD, and some 150 vector instructions (exponentials, maxima, the conversion of p, a
// quarter of the decoding), some 650; matrix cores 0.48 and vector units 0.63 of the time, a wave waits 0.29 of its own for
// its turn, and the clock falls to some 2.05 GHz under that load. Both products and the LDS rows run over DP, so widths
// between pay for the next of 64, 128 and 256: that prompt at D = 32 takes 412 us, 64 444 (773 TFLOP/s: half the matrix work
// for each exponential), 96 673, 160 1256, 192 1291, 224 1340, 256 1362 (1009). With tiles of 64 keys, where D = 128
// took 748 us, the next tile's logits before this one's softmax took 733; with tiles of 32, at 715, that was not tried
// again. Tried without gain: 256 rows (756), the overflow of sums in place of the maxima, LDS operands read ahead in a
// fixed order, 64 rows of two waves.
#include <algorithm>

#include "attn.hpp"
#include "device_once.hpp"
#include "pipeline.hpp"

namespace ssn {
namespace {

// LDS writes done before, LDS reads after; global loads stay in flight
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

template <int DP, int TK>
struct Lds {
  static constexpr int KS = DP * 2 + 16, VS = TK * 2 + 16;   // bytes of a row: of a token's keys, of a d's values
  uint8_t k[TK * KS];
  uint8_t v[DP * VS];
  uint32_t there[4];                                         // byte u % 4 of word u / 4: unit u of 16 tokens has a page
};

// The first token and d of lane l's piece of keys (one token, 32 d) or values (four tokens, eight d), the wave's first
// token being base: an order in which the rows that 8 and 16 lanes write together lie in different LDS banks.
template <int DP>
__device__ __forceinline__ void piece(bool values, int base, int l, int& tok, int& d) {
  if (values) {
    if constexpr (DP == 64) {
      tok = base + 4 * ((l >> 1) & 7);
      d = 8 * ((l & 1) | (l >> 4) << 1);
    } else if constexpr (DP == 128) {
      tok = base + 4 * ((l >> 2) & 3);
      d = 8 * ((l & 3) | (l >> 4) << 2);
    } else {                                       // tokens 8 apart, so that the two halves of a 16-byte piece are written together
      tok = (base & ~15) + (base & 8) / 2 + 8 * ((l >> 3) & 1);
      d = 8 * ((l & 7) | (l >> 4) << 3);
    }
  } else {
    if constexpr (DP == 64) {
      tok = base + ((l & 3) | (l & 8) | (l & 16) >> 2 | (l & 32) >> 1);
      d = 32 * ((l >> 2) & 1);
    } else if constexpr (DP == 128) {
      tok = base + ((l & 3) | (l >> 4) << 2);
      d = 32 * ((l >> 2) & 3);
    } else {
      tok = base + ((l & 3) | (l & 32) >> 3);
      d = 32 * ((l >> 2) & 7);
    }
  }
}

// the largest of the lanes' values, none below 0
__device__ __forceinline__ int wave_max(int x) {
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false));   // from one, two, four and eight lanes below
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false));
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false));   // the last of 16 lanes to the next 16
  x = max(x, __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false));   // the last of 32 to the next 32
  return __builtin_amdgcn_readlane(x, 63);
}

// Item t of the pairs (sequence, tile of rows), those with the most keys first: workgroups start in this order, so the
// long ones do not end alone. Tile j from the end of sequence b lies at level off_b + j of R rows below max_kv keys, so
// C(p) = sum over b of clamp(p - off_b, 0, tiles_b) items lie above level p; the last of the levels off_b and
// off_b + tiles_b with C <= t is found, a lane a sequence, and from there each level holds the same sequences. Beyond 64
// sequences: the last tiles of all, then those before. False behind the last item. 7 chunks of 214 to 1500 queries
// over 2251 to 9001 keys: 520 us, 775 in the order of the batch; 16 prompts of 512 72 and 73 to 79.
//
// Where row_tiles a sequence would be too many workgroups (a large batch whose max_q is all its queries), sequence b has
// the items from v_b = floor(q_offsets[b] G / R) + b on: v ascends, v_(b+1) - v_b holds the sequence's tiles, and all
// of them lie below Tq G / R + B. The last b with v_b <= t is found by 64 probes at once, three times for 65535.
__device__ __forceinline__ bool find_item(const AttnLaunch& L, int t, int lane, int& b, int& rt, Seq& seq) {
  const int B = (int)L.a.B;
  if (L.owned) {
    auto first = [&](int x) {
      const int64_t q0 = L.a.q_offsets ? max(L.a.q_offsets[x], 0) : x * L.each;
      return (int)min(q0 * L.G / kTileRows, (int64_t)1 << 30) + x;
    };
    b = 0;
    for (int n = B; n > 1;) {                            // b is in [b, b + n)
      const int step = (n + 63) / 64;
      const uint64_t in = __ballot(lane * step < n && first(b + min(lane * step, n - 1)) <= t);
      const int probe = max(__popcll(in) - 1, 0) * step;
      b += probe;
      n = min(step, n - probe);
    }
    b = __builtin_amdgcn_readfirstlane(b);
    rt = t - __builtin_amdgcn_readfirstlane(first(b));
    seq = find_seq(L, b);
    return rt >= 0;
  }
  if (B > 64 || B == 1) {
    const int j = B == 1 ? t : t / B;
    b = t - j * B;
    rt = L.row_tiles - 1 - j;
    seq = find_seq(L, b);
    return true;
  }
  const Seq s = find_seq(L, min(lane, B - 1));
  int off = 0, tiles = 0;
  if (lane < B && s.n > 0) {
    const int64_t keys = max(s.len - s.all + s.n, (int64_t)0);
    off = (int)min(((L.a.max_kv - keys) * L.G) / kTileRows, (int64_t)1 << 29);
    tiles = (int)((s.n * L.G + kTileRows - 1) / kTileRows);
  }
  const int off0 = __builtin_amdgcn_readfirstlane(off), tiles0 = __builtin_amdgcn_readfirstlane(tiles);
  if (!__any(lane < B && (off != off0 || tiles != tiles0))) {        // all alike
    const int j = t / B;
    b = t - j * B;
    rt = tiles0 - 1 - j;
    if (rt < 0) return false;
  } else {
    int c0 = 0, c1 = 0, total = 0;
    for (int x = 0; x < B; ++x) {
      const int o = __builtin_amdgcn_readlane(off, x), n = __builtin_amdgcn_readlane(tiles, x);
      c0 += min(max(off - o, 0), n);
      c1 += min(max(off + tiles - o, 0), n);
      total += n;
    }
    if (t >= total) return false;
    const int p = wave_max(c1 <= t ? off + tiles : c0 <= t ? off : 0), above = wave_max(c1 <= t ? c1 : c0 <= t ? c0 : 0);
    uint64_t in = __ballot(off <= p && p < off + tiles);
    const int m = __popcll(in), j = (t - above) / m;     // m > 0: t is above the next of those levels
    for (int x = t - above - j * m; x > 0; --x) in &= in - 1;
    b = __ffsll((unsigned long long)in) - 1;
    rt = __builtin_amdgcn_readlane(tiles, b) - 1 - (p + j - __builtin_amdgcn_readlane(off, b));
  }
  auto from = [&](int64_t v) {
    return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), b) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)v, b));
  };
  seq = {from(s.q0), from(s.all), from(s.n), __builtin_amdgcn_readlane(s.len, b)};
  return true;
}

template <int DP, int W, int TK, int WPS>
__global__ __launch_bounds__(64 * W, WPS) void k_attn_tile(AttnLaunch L) {
  static_assert(32 * W == kTileRows, "");
  constexpr int R = 32 * W, NTH = 64 * W, KS = DP / 16, MT = DP / 32, AT = TK / 32;
  constexpr int NK = TK * DP / 32, IT = 2 * NK / NTH;        // pieces of 16 bytes of keys, as many of values; a thread's
  static_assert(NK % 64 == 0 && 2 * NK % NTH == 0, "");
  using Buf = Lds<DP, TK>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds_raw[];
  Buf* const lds = (Buf*)lds_raw;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int id = div_by(L.sd, blockIdx.x), split = blockIdx.x - id * L.splits;
  const KvCache& c = L.a.c;
  const int D = c.D, item = id / c.heads, h = id - item * c.heads;
  int b, rt;
  Seq seq;
  Work w;
  if (!find_item(L, item, lane, b, rt, seq) || !find_work(L, seq, b, h, rt, R, w)) return;

  // What this thread brings of every tile: of each piece the first token and d. A wave's pieces lie in UW units of 16
  // tokens, so pages are found once a wave, in scalar registers, and a lane's offsets never change.
  constexpr int TW = 64 * 32 / DP, UW = (TW + 15) / 16;          // tokens and units of a wave
  int tok[IT], dd[IT];
  uint32_t at[IT], ats[IT];
  bool isv[IT];
#pragma unroll
  for (int it = 0; it < IT; ++it) {
    isv[it] = NK % NTH ? it * NTH + 64 * wave >= NK : it * NTH >= NK;
    piece<DP>(isv[it], wave * TW % TK, lane, tok[it], dd[it]);
    // beyond D an offset beyond the resource, which reads 0
    at[it] = dd[it] < D ? (tok[it] & 15) * (D / 2) + dd[it] / 2 : 0x80000000u;
    ats[it] = dd[it] >= D ? 0x80000000u : isv[it] ? dd[it] / 16 * c.page + (tok[it] & 15) : (tok[it] & 15) * (D / 16) + dd[it] / 16;
  }
  const int t0 = w.lo / TK, t1 = (w.hi + TK - 1) / TK;
  const int per = div_by(L.sd, max(t1 - t0, 0) + L.splits - 1);
  const int ta = t0 + split * per, tb = min(t1, ta + per);

  u32x4 raw[IT];
  uint32_t scl[IT];
  int pg[UW], place[UW];                             // of the tile to load next
  bool there[UW];                                    // of the tile loaded last
  const int first_unit = (wave * TW % TK) >> 4;      // the wave's first unit in a tile, the same for keys and values
  auto find_pages = [&](int t) {
#pragma unroll
    for (int u = 0; u < UW; ++u) pg[u] = page_of(L, b, t * (TK / 16) + first_unit + u, place[u]);
  };
  auto load_unit = [&](int u) {
    const int64_t head = (int64_t)(there[u] ? pg[u] : 0) * c.heads + h, row = head * c.page + place[u];
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if (isv[it]) {
        const auto vc = buf_rsrc(c.v_codes + row * (D / 2)), vs = buf_rsrc(c.v_scales + head * (D / 16) * c.page + place[u]);
#pragma unroll
        for (int i = 0; i < 4; ++i) raw[it][i] = __builtin_amdgcn_raw_buffer_load_b32(vc, at[it], i * (D / 2), 0);
        scl[it] = __builtin_amdgcn_raw_buffer_load_b32(vs, ats[it], 0, 0);
      } else {
        const auto kc = buf_rsrc(c.k_codes + row * (D / 2)), ks = buf_rsrc(c.k_scales + row * (D / 16));
        raw[it] = __builtin_amdgcn_raw_buffer_load_b128(kc, at[it], 0, 0);
        scl[it] = __builtin_amdgcn_raw_buffer_load_b16(ks, ats[it], 0, 0);
      }
    }
  };
  auto load = [&]() {
#pragma unroll
    for (int u = 0; u < UW; ++u) there[u] = is_page(L, pg[u]);
    if (UW == 1 || !(tok[0] & 16)) load_unit(0);
    else load_unit(UW - 1);
  };
  auto stage = [&](Buf& f, int t) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const bool ok = UW == 1 || !(tok[it] & 16) ? there[0] : there[UW - 1];
      if (isv[it]) {
        uint32_t s = scl[it];
        // what lies in a slot that no row keeps may be anything: its value's scale becomes 0
        const int x = t * TK + tok[it], lo = min(max(w.lo - x, 0), 4), hi = min(max((ok ? w.hi : 0) - x, 0), 4);
        s &= (hi == 4 ? ~0u : (1u << (8 * hi)) - 1u) & (lo == 4 ? 0u : ~0u << (8 * lo));
        const f16x2 s01 = e4m3x2_f16<false>(s), s23 = e4m3x2_f16<true>(s);
        uint32_t e01, o01, e23, o23;
        pair_tokens(raw[it][0], raw[it][1], e01, o01);
        pair_tokens(raw[it][2], raw[it][3], e23, o23);
        const u32x2 d[8] = {{fp4x2_f16<0>(e01, s01), fp4x2_f16<0>(e23, s23)}, {fp4x2_f16<0>(o01, s01), fp4x2_f16<0>(o23, s23)},
                            {fp4x2_f16<1>(e01, s01), fp4x2_f16<1>(e23, s23)}, {fp4x2_f16<1>(o01, s01), fp4x2_f16<1>(o23, s23)},
                            {fp4x2_f16<2>(e01, s01), fp4x2_f16<2>(e23, s23)}, {fp4x2_f16<2>(o01, s01), fp4x2_f16<2>(o23, s23)},
                            {fp4x2_f16<3>(e01, s01), fp4x2_f16<3>(e23, s23)}, {fp4x2_f16<3>(o01, s01), fp4x2_f16<3>(o23, s23)}};
        // token 16 s + 8 x + 4 h + e is at 16 s + 8 h + 4 x + e
        const int pos = (tok[it] & ~15) | (tok[it] & 4) << 1 | (tok[it] & 8) >> 1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int rho = (dd[it] + j) / MT, m = j % MT;
          *(u32x2*)(f.v + (m * 32 + rho) * Buf::VS + pos * 2) = d[j];
        }
      } else {
        const f16x2 s = e4m3x2_f16<false>(scl[it]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          *(f16x8*)(f.k + tok[it] * Buf::KS + (dd[it] + 8 * j) * 2) = fp4x8_f16(raw[it][j], s[j / 2]);
        if (dd[it] == 0 && !(tok[it] & 15)) ((uint8_t*)f.there)[tok[it] >> 4] = ok;
      }
    }
  };
  // queries: the lane's row, d = 16 s + 8 half ..
  const int r = w.row0 + 32 * wave + col;
  int lo_r, hi_r;
  row_keys(L, w, r, lo_r, hi_r);
  const Factor factor = factor_of(L.a.scale, c.k_ts[h]);
  f16x8 q[KS];
  Reference ref;
  {
    const int rr = min(r, w.rows - 1), i = div_by(L.gd, rr);
    const uint16_t* src = (const uint16_t*)L.a.Q + (w.q0 + i) * L.a.q_token + (int64_t)(h * L.G + (rr - i * L.G)) * L.a.q_head;
    u32x4 x[KS];
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int d = 16 * s + 8 * half;
      x[s] = *(const u32x4*)(src + (d < D ? d : 0));
      if (r >= w.rows || d >= D) x[s] = u32x4{0, 0, 0, 0};
      m = max_bits(m, x[s]);
    }
    float amax = max_of(m, L.a.q_type);
    amax = fmaxf(amax, __shfl_xor(amax, 32, 64));
    const RowScale scale = row_scale(amax, factor);
    if (L.a.q_type == kBF16) scale_rows<kBF16>(x, scale.by);
    else scale_rows<kF16>(x, scale.by);
#pragma unroll
    for (int s = 0; s < KS; ++s) q[s] = as_f16x8(x[s]);
    ref.c = scale.c;
  }
  if (ta < tb) {
    find_pages(ta);
    load();
    find_pages(ta + 1);
  }

  // keys that some row, and that every row, of this wave keeps (rows behind the last aside)
  const int first = w.row0 + 32 * wave, last = min(first + 31, w.rows - 1);
  int wlo, whi, wlo_all, whi_all;
  row_keys(L, w, min(first, w.rows - 1), wlo, whi_all);
  row_keys(L, w, max(last, 0), wlo_all, whi);
  wlo = max(wlo, 0);
  if (first >= w.rows) whi = 0;

  f32x16 o[MT] = {};
  float l = 0.f;

  for (int t = ta; t < tb; ++t) {
    Buf& f = lds[(t - ta) & 1];
    stage(f, t);
    if (t + 1 < tb) {
      load();
      find_pages(t + 2);
    }
    lds_barrier();
    const int k0 = t * TK;
    if (k0 >= whi || k0 + TK <= wlo) continue;       // nothing for this wave (it still brings its part)
    f32x16 s[AT];
#pragma unroll
    for (int a = 0; a < AT; ++a) {
      s[a] = f32x16{};
#pragma unroll
      for (int x = 0; x < KS; ++x) {
        const f16x8 k = *(const f16x8*)(f.k + (32 * a + col) * Buf::KS + (16 * x + 8 * half) * 2);
        s[a] = __builtin_amdgcn_mfma_f32_32x32x16_f16(k, q[x], s[a], 0, 0, 0);
      }
    }
    constexpr uint32_t all = TK == 64 ? 0x01010101u : 0x0101u;
    const uint32_t units = __builtin_amdgcn_readfirstlane(f.there[0]) & (TK == 64 ? ~0u : 0xFFFFu);
    if (k0 < wlo_all || k0 + TK > whi_all || units != all) {
      const int lo = lo_r - k0 - 4 * half, hi = hi_r - k0 - 4 * half;
#pragma unroll
      for (int a = 0; a < AT; ++a)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int x = 32 * a + 8 * (i / 4) + i % 4;
          const int page = (int)(units << (31 - 8 * (2 * a + i / 8))) >> 31;     // all ones where the unit has one
          s[a][i] = ((x >= lo) & (x < hi) & page) ? s[a][i] : -__builtin_inff();
        }
    }
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 16 * AT; ++i) top = fmaxf(top, s[i / 16][i % 16]);
    if (__any(top * ref.c - ref.m > kTop)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float by = ref.raise(top);
      l *= by;
#pragma unroll
      for (int m = 0; m < MT; ++m) o[m] *= by;
    }
    f16x8 p[2 * AT];
#pragma unroll
    for (int y = 0; y < 2 * AT; ++y) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        e[i] = exp2_hw(fmaf(s[y / 2][8 * (y & 1) + i], ref.c, -ref.m));
        l += e[i];
      }
      p[y] = as_f16x8(u32x4{pk_f16(e[0], e[1]), pk_f16(e[2], e[3]), pk_f16(e[4], e[5]), pk_f16(e[6], e[7])});
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int y = 0; y < 2 * AT; ++y) {
        const f16x8 v = *(const f16x8*)(f.v + (m * 32 + col) * Buf::VS + (16 * y + 8 * half) * 2);
        o[m] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v, p[y], o[m], 0, 0, 0);
      }
  }

  l += __shfl_xor(l, 32, 64);
  const float mc = ref.m * ref.up;
  if (r >= w.rows) return;
  const int64_t part = ((((int64_t)b * c.heads + h) * L.row_tiles + rt) * L.splits + split) * R + 32 * wave + col;
  const int i0 = div_by(L.gd, r);
  const int64_t head = (w.q0 + i0) * L.a.Hq + h * L.G + (r - i0 * L.G);
  if (L.splits > 1) {
    if (half == 0) *(f32x2*)(L.part_ml + 2 * part) = f32x2{mc, l};
    if (!(l != 0.f)) return;
  } else if (L.a.lse && half == 0) {
    L.a.lse[head] = l != 0.f ? (mc + log2f(l)) * kLn2 : -__builtin_inff();
  }
  Finish fin = finish(c.v_ts[h], l);
  if (L.splits > 1) fin = {1.f, 0};
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int d = MT * (8 * u + 4 * half);           // 4 MT consecutive d
    float x[4 * MT];
#pragma unroll
    for (int e = 0; e < 4 * MT; ++e) x[e] = fin(o[e % MT][4 * u + e / MT]);
#pragma unroll
    for (int e = 0; e < 4 * MT; e += 8) {
      if (d + e >= D) break;
      if (L.splits > 1) store_run<8>(L.part_o, kF32, part * D + d + e, x + e);
      else store_run<8>(L.a.out, L.a.out_type, head * D + d + e, x + e);
    }
  }
}

template <int DP, int W, int TK, int WPS>
hipError_t launch(const AttnLaunch& L, int64_t groups, hipStream_t st) {
  constexpr size_t bytes = 2 * sizeof(Lds<DP, TK>);
  static PerDeviceOnce once;
  const hipError_t e = once_per_device(once, [] {
    return hipFuncSetAttribute((const void*)k_attn_tile<DP, W, TK, WPS>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attn_tile<DP, W, TK, WPS>), dim3((unsigned)groups), dim3(64 * W), bytes, st, L);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_tile(const AttnLaunch& L, int64_t groups, hipStream_t st) {
  const int D = L.a.c.D;
  // 64 keys a tile at D = 64, as four waves need for their 16-byte pieces; 32 at D = 128, where 64 leave room for two waves
  // a SIMD (a prompt of 8192 tokens 715 us, 740 with 64; 16 of 512 73 and 88), and at 256, where LDS holds no more
  if (D <= 64) return launch<64, 4, 64, 2>(L, groups, st);
  if (D <= 128) return launch<128, 4, 32, 3>(L, groups, st);
  return launch<256, 4, 32, 2>(L, groups, st);
}

}  // namespace ssn
