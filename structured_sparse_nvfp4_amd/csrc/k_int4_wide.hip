// Integer 4-bit product for more rows of Y than k_int4.hip keeps in registers, or a longer K (the arithmetic
// is in int4.hpp).
//
// One workgroup of eight waves computes 16 MT rows of Y for 16 NT weight rows; each wave takes an eighth
// of K and keeps the whole tile's sums. Weights go straight to registers, one chunk ahead. The activations
// of a chunk come through the wave's own LDS by direct loads, which need no registers and read each row's
// 256 bytes together: they are read at the chunk's start and the next chunk's are sent for, a part after
// each tile, to arrive while this one is multiplied. No wave waits for another before the end, where the eight tiles of
// sums meet in the same LDS, one thread per output.
//
// Every weight is decoded once and multiplied by MT operands; every operand of activations serves NT
// tiles, so a workgroup reads 16 MT K activations from the L2 for 16 NT K weights. No one part bounds it:
// a wave goes through loads, LDS, decode and matrix instructions in turn, and two waves per SIMD hide little of
// that (M = 50, N = 4097, K = 5152, group 64 16.8 us; without any loads 12.7, without the decode 16.4; M = 64, N =
// 131072, group 128: vector units busy 0.41 of the time, matrix cores 0.26, a wave waits 0.33 of its own for memory or
// LDS and 0.38 for its turn). M = 64, group 128: N = 13824, K = 5120 25 us, N = 131072 183 us (2.1 TB/s, 470
// TFLOP/s); M = 16: N = 13824 16.6 us. The 4 x 4 tile spills 36 bytes a lane for groups of 32 and 16 for 64.
#include <algorithm>

#include "device_once.hpp"
#include "int4.hpp"

namespace ssn {
namespace {

constexpr int kWaves = 8;

template <bool F16X, int MT, int NT, int FOLD, bool GROUPED, bool SILU>
__global__ __launch_bounds__(kWaves * 64, !GROUPED && MT * NT <= 2 ? 4 : 2) void k_int4_wide(Int4GemvArgs a, int ngroups) {
  constexpr int SPANS = 4 / FOLD, H = SILU ? 2 : 1;
  // A wave's activations: 256 bytes per row, in 16 pieces, piece p of row r at place p ^ swizzle(r). The LDS
  // serves a 16-byte read in groups of lanes like 0-3, 12-15, 20-27: rows 0-3 and 12-15 of one piece and
  // rows 4-11 of the next lane group's. With r itself as the swizzle they meet no bank twice where the lane
  // groups' pieces follow one another (finer groups of k), with its bit pairs exchanged where they are four apart.
  __shared__ __attribute__((aligned(1024))) char lds[kWaves][16 * MT][256];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kq = lane >> 4;
  auto swizzle = [](int r) { return FOLD == 4 ? (r & 3) << 2 | (r >> 2 & 3) : r & 15; };
  const int No = (int)(a.N / H);
  const int K = (int)a.K, nch = (K + kChunk - 1) / kChunk, g32 = (int)(a.group / 32), groups = (int)a.groups;
  const int c_lo = nch * wave / kWaves, c_hi = nch * (wave + 1) / kWaves;
  const uint32_t one = F16X ? 0x3C003C00u : 0x3F803F80u;
  const u32x4 ones = {one, one, one, one};
  const f32x4 zero4 = {0.f, 0.f, 0.f, 0.f};
  const uint32_t z_add = a.zeros ? 0u : 8u;

  // Workgroups run over the sets of 16 MT rows (the grid's first axis, so that those that share weights run
  // side by side) and over groups of weight rows; with experts, a workgroup has one set.
  int e = 0, r0 = 16 * MT * blockIdx.x, cnt = 0, ng0 = blockIdx.y, ng_step = gridDim.y;
  if constexpr (GROUPED) {
    Slot sl;
    if (!find_slot(a.offsets, a.E, (int)a.M, 16 * MT, ngroups, sl)) return;
    e = sl.e; r0 = sl.r0; cnt = sl.cnt; ng0 = sl.part; ng_step = sl.parts;
  }
  for (int ng = ng0; ng < ngroups; ng += ng_step) {
    if constexpr (!GROUPED) cnt = min((int)a.M - r0, 16 * MT);
    // A direct load brings four rows' 256 bytes: lane l piece (l % 16) of row l / 16. Rows past the last come
    // as zeros or stay what they were; their sums are dropped.
    const int xrow = lane >> 4;
    const char* xp[GROUPED ? 4 : 1];          // with experts: a pointer per row, else an offset from the first
    uint32_t xo[GROUPED ? 1 : 4];
    const auto xr = buf_rsrc((const uint16_t*)a.X + (GROUPED ? 0 : (int64_t)r0 * K), GROUPED ? 0 : cnt * K * 2);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t piece = 16u * (uint32_t)(r16 ^ swizzle(4 * q + xrow));
      if constexpr (GROUPED) {
        const int m = r0 + min(4 * q + xrow, cnt - 1);
        const int src = min(max(a.row_token ? a.row_token[m] : m, 0), (int)a.x_rows - 1);
        xp[q] = (const char*)a.X + (int64_t)src * K * 2 + piece;
      } else {
        xo[q] = (uint32_t)(4 * q + xrow) * (uint32_t)K * 2u + piece;
      }
    }
    // first row, and rows, of a tile: those of one expert, gate tiles before up tiles
    auto tile_row = [&](int t) { return 16 * (SILU ? ng * (NT / H) + t % (NT / H) : ng * NT + t); };
    struct Loads {
      u32x4 w[NT];
    };
    auto tile_base = [&](int t) { return (int64_t)e * a.N + (SILU && t >= NT / H ? No : 0) + tile_row(t); };
    auto tile_rows = [&](int t) {
      // (not max(0, min(..)): the compiler makes v_med3 of it, and a resource in vector registers)
      const int n0 = tile_row(t);
      return n0 < No ? min(16, No - n0) : 0;
    };
    auto load = [&](Loads& o, int c) __attribute__((always_inline)) {
      const int k = kChunk * c + 32 * kq;
      const uint32_t ko = c < c_hi && k < K ? (uint32_t)(r16 * (K / 2) + k / 2) : kOutside;
#pragma unroll
      for (int t = 0; t < NT; ++t)
        o.w[t] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                               buf_rsrc(a.codes + tile_base(t) * (K / 2), tile_rows(t) * (K / 2)), ko, 0, 0));
    };
    // Scales and zero points: lane group g loads span g of the four spans from chunk c on, FOLD chunks' worth
    // (a load of its own for every chunk costs the address unit as much as the codes)
    uint32_t sc[NT], zp[NT], sz[NT] = {};
    auto load_sz = [&](int c) __attribute__((always_inline)) {
      const int k = kChunk * c + 32 * FOLD * kq;
      const uint32_t go = c < c_hi && k < K ? (uint32_t)(r16 * groups + k / 32 / g32) : kOutside / 2;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int rows = tile_rows(t) * groups;
        sc[t] = __builtin_amdgcn_raw_buffer_load_b16(buf_rsrc(a.scales + tile_base(t) * groups, rows * 2), 2 * go, 0, 0);
        zp[t] = __builtin_amdgcn_raw_buffer_load_b8(buf_rsrc(a.zeros + tile_base(t) * groups, a.zeros ? rows : 0), go, 0, 0);
      }
    };
    // part j of the kParts of the direct loads of chunk c
    constexpr int kParts = SPANS * NT;
    auto send_x = [&](int c, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 4 * MT * j / kParts; i < 4 * MT * (j + 1) / kParts; ++i) {
        if constexpr (GROUPED) {
          // a piece past the end of K: the row's first
          const int piece = r16 ^ swizzle(4 * i + xrow);
          lds_dma16(xp[i] + (kChunk * c + 8 * piece < K ? 2 * c * kChunk : -16 * piece), lds[wave][4 * i]);
        } else {
          lds_dma16(xr, xo[i % 4] + (uint32_t)(i / 4 * 16) * (uint32_t)K * 2u + (uint32_t)(2 * c * kChunk), 0u, lds[wave][4 * i]);
        }
      }
    };
    f32x4 tot[NT][MT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) tot[t][mt] = zero4;
    // chunk c, whose weights are on their way to cur; the next chunk's go to nxt
    auto chunk = [&](const Loads& cur, Loads& nxt, int c) __attribute__((always_inline)) {
      wait_vmcnt<0>();                        // this chunk's activations are in LDS
      asm volatile("" ::: "memory");
      u32x4 x[MT][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int s = 0; s < 4; ++s)
          x[mt][s] = *(const u32x4*)(lds[wave][16 * mt + r16] + 16 * ((FOLD == 4 ? 4 * kq + s : 4 * s + kq) ^ swizzle(r16)));
      __builtin_amdgcn_s_waitcnt(0xC07F);     // read, before they are written over
      asm volatile("" ::: "memory");
      const int phase = (c - c_lo) % FOLD;    // of the chunks that share a load of scales
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t fresh = sc[t] | (zp[t] + z_add) << 16;
        sz[t] = phase == 0 ? fresh : sz[t];
      }
      if (phase == FOLD - 1) load_sz(c + 1);
      load(nxt, c + 1);
      __builtin_amdgcn_sched_barrier(0);
      if (kChunk * (c + 1) > K) {
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = kChunk * c + (FOLD == 4 ? 32 * kq : 32 * s);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
            if (k >= K) x[mt][s] = u32x4{0u, 0u, 0u, 0u};
        }
      }
      u32x4 w[NT], szs[NT];                   // codes, and scales and zero points of the chunk's spans, in every lane
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        w[t] = FOLD == 4 ? cur.w[t] : transpose4(cur.w[t]);
        if (FOLD == 1) szs[t] = spread4(sz[t]);
        else
#pragma unroll
          for (int v = 0; v < SPANS; ++v)
            szs[t][v] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * (16 * (phase * SPANS + v) + r16), (int)sz[t]);
      }
      // Span by span, so that only one span's sums of x are held (M = 64, N = 131072, K = 5120 182 us; with all
      // of them held 190). Activations sent straight to registers come in pieces of 64 bytes and were slower than
      // through LDS: 21.6 against 18.6 us at M = 20, N = 13824, K = 5120, 24.0 against 20.0 at M = 50, N = 4097.
#pragma unroll
      for (int v = 0; v < SPANS; ++v) {
        f32x4 sum[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          sum[mt] = zero4;
#pragma unroll
          for (int i = 0; i < FOLD; ++i) sum[mt] = mfma16<F16X>(x[mt][v * FOLD + i], ones, sum[mt]);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          u32x4 op[FOLD];
#pragma unroll
          for (int i = 0; i < FOLD; ++i) op[i] = codes_operand_natural<F16X>(w[t][v * FOLD + i]);
          const float s = float16_of((uint16_t)(szs[t][v] & 0xFFFFu), a.s_type), z = (float)(szs[t][v] >> 16);
          f32x4 acc[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) acc[mt] = zero4;
#pragma unroll
          for (int i = 0; i < FOLD; ++i)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) acc[mt] = mfma16<F16X>(x[mt][v * FOLD + i], op[i], acc[mt]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tot[t][mt][i] = __builtin_fmaf(s, __builtin_fmaf(-z, sum[mt][i], acc[mt][i]), tot[t][mt][i]);
          // the next chunk's activations, a part at a time; past the share its last chunk again, not used
          __builtin_amdgcn_sched_barrier(0);
          send_x(min(c + 1, c_hi - 1), v * NT + t);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    if (c_lo < c_hi) {
      Loads buf[2];
#pragma unroll
      for (int j = 0; j < kParts; ++j) send_x(c_lo, j);
      load_sz(c_lo);
      load(buf[0], c_lo);
      __builtin_amdgcn_sched_barrier(0);
      for (int c = c_lo;; c += 2) {
        chunk(buf[0], buf[1], c);
        if (c + 1 >= c_hi) break;
        chunk(buf[1], buf[0], c + 1);
        if (c + 2 >= c_hi) break;
      }
      wait_vmcnt<0>();                        // the last direct loads have written LDS
      asm volatile("" ::: "memory");
    }
    // the eight waves' tiles meet in LDS, each in its wave's own part (NT MT KB of MT 4 KB)
    static_assert(NT <= 4, "a wave's sums fit its part of LDS");
    float* const red = (float*)lds;
    constexpr int kPart = MT * 4 * 256;       // floats per wave
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) *(f32x4*)(red + wave * kPart + (t * MT + mt) * 256 + 4 * lane) = tot[t][mt];
    __syncthreads();
    constexpr int kOuts = NT / H * MT * 256;
    for (int o = threadIdx.x; o < kOuts; o += kWaves * 64) {
      // output o: weight row o % 16 of its tile, row o / 16 % 16 of its row tile
      const int n16 = o & 15, m16 = (o >> 4) & 15, j = o >> 8, mt = j % MT, t = j / MT;
      const int m = 16 * mt + m16, n = tile_row(t) + n16;
      if (m >= cnt || n >= No) continue;
      const float* p = red + j * 256 + (16 * (m16 >> 2) + n16) * 4 + (m16 & 3);
      float y = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        y += p[w * kPart];
        if (SILU) u += p[w * kPart + NT / H * MT * 256];
      }
      if (SILU) y = silu(y) * u;
      store_elem(a.Y, a.y_type, (int64_t)(r0 + m) * No + n, y);
    }
    __syncthreads();
  }
}

template <bool F16X, int MT, int NT, int FOLD, bool GROUPED, bool SILU>
hipError_t launch_wide(const Int4GemvArgs& a, hipStream_t s) {
  constexpr int H = SILU ? 2 : 1;
  const int64_t No = a.N / H;
  const int ngroups = (int)((No + 16 * NT / H - 1) / (16 * NT / H));
  dim3 grid((unsigned)((a.M + 16 * MT - 1) / (16 * MT)), (unsigned)std::min(ngroups, 65535));
  if (GROUPED) grid = dim3((unsigned)std::max<int64_t>(4 * cu_count(), std::min<int64_t>(a.E, a.M) + a.M / (16 * MT)));
  hipLaunchKernelGGL((k_int4_wide<F16X, MT, NT, FOLD, GROUPED, SILU>), grid, dim3(kWaves * 64), 0, s, a, ngroups);
  return hipGetLastError();
}

// The tile of a product: the time is taken to be the number of rounds of cu_count() workgroups times a
// round's own, which grows with the tile. Measured at K = 5120, in tenths of a us per round:
//   NT            1    2    3    4
//   16 rows      65   97  125  149
//   32 rows      80  115  144  172
//   64 rows           167  198  230
// The larger tiles cost less per output, the smaller ones leave less of a last round empty: M = 50, N = 5120 takes
// 14.4 us in one round of 2 x 3 tiles, 16.1 in one of 4 x 2, 19.4 in two of 2 x 2, 22.2 in a third of one of 4 x 4.
// Two things it leaves out. A compute unit holds two workgroups of the tiles 1 x 2, 1 x 3 and 2 x 1 (of 2 x 2
// too for groups of a multiple of 128) and three of 1 x 1, so that their second round is often the shorter one (1 x 1
// 6.5 us and 3.5 more, 2 x 1 8.3 and 5.3, 1 x 3 13.0 and 9.3); one of each other tile. And K changes the
// proportions where it is short: one round of 4 x 4, 2 x 2 and 1 x 1 takes 10.6, 5.8 and 4.6 us at K = 1024, 27.5,
// 10.7 and 6.5 at 5120, 67, 33 and 17.5 at 16384.
struct Tile {
  int mt, nt, cost;
};
constexpr Tile kTiles[] = {{4, 4, 230}, {4, 3, 198}, {4, 2, 167}, {2, 4, 172}, {2, 3, 144}, {2, 2, 115},
                           {2, 1, 80},  {1, 4, 149}, {1, 3, 125}, {1, 2, 97},  {1, 1, 65}};

template <bool F16X, int FOLD>
hipError_t launch_wide_m(const Int4GemvArgs& a, hipStream_t s) {
  if (a.offsets)
    return a.silu ? launch_wide<F16X, 1, 2, FOLD, true, true>(a, s) : launch_wide<F16X, 1, 2, FOLD, true, false>(a, s);
  const int64_t cus = cu_count();
  const Tile* best = nullptr;
  int64_t least = 0;
  for (const Tile& t : kTiles) {
    const int64_t wgs = (a.M + 16 * t.mt - 1) / (16 * t.mt) * ((a.N + 16 * t.nt - 1) / (16 * t.nt));
    const int64_t cost = (wgs + cus - 1) / cus * t.cost;
    if (!best || cost < least) best = &t, least = cost;
  }
  switch (4 * best->mt + best->nt) {
    case 20: return launch_wide<F16X, 4, 4, FOLD, false, false>(a, s);
    case 19: return launch_wide<F16X, 4, 3, FOLD, false, false>(a, s);
    case 18: return launch_wide<F16X, 4, 2, FOLD, false, false>(a, s);
    case 12: return launch_wide<F16X, 2, 4, FOLD, false, false>(a, s);
    case 11: return launch_wide<F16X, 2, 3, FOLD, false, false>(a, s);
    case 10: return launch_wide<F16X, 2, 2, FOLD, false, false>(a, s);
    case 9: return launch_wide<F16X, 2, 1, FOLD, false, false>(a, s);
    case 8: return launch_wide<F16X, 1, 4, FOLD, false, false>(a, s);
    case 7: return launch_wide<F16X, 1, 3, FOLD, false, false>(a, s);
    case 6: return launch_wide<F16X, 1, 2, FOLD, false, false>(a, s);
    default: return launch_wide<F16X, 1, 1, FOLD, false, false>(a, s);
  }
}

template <bool F16X>
hipError_t launch_wide_f(const Int4GemvArgs& a, hipStream_t s) {
  switch (int4_fold(a.group)) {
    case 4: return launch_wide_m<F16X, 4>(a, s);
    case 2: return launch_wide_m<F16X, 2>(a, s);
    default: return launch_wide_m<F16X, 1>(a, s);
  }
}

}  // namespace

hipError_t launch_int4_wide(const Int4GemvArgs& a, hipStream_t s) {
  return a.x_type == kF16 ? launch_wide_f<true>(a, s) : launch_wide_f<false>(a, s);
}

}  // namespace ssn
