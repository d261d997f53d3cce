// Host-side launchers of the gfx950 kernels (internal to the library; the public C ABI is
// declared in include/ssnvfp4.h and implemented in api.hip). Every launcher assumes its
// arguments were validated by the caller and returns the launch status.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssn {

// quantisation / producer side
hipError_t launch_quantize(const void* W, int w_bf16, int64_t N, int64_t K, const float* ts_in,
                           uint8_t* codes, uint8_t* scales, float* ts_out, hipStream_t s);
hipError_t launch_dequantize(const uint8_t* codes, const uint8_t* scales, const float* ts, int64_t N,
                             int64_t K, void* out, int out_bf16, hipStream_t s);
// ts_out nullable: when given, receives s_t = fl32(amax|W| / 2688) gathered during the prune
hipError_t launch_prune(const void* W, int w_bf16, int64_t N, int64_t K, void* out, float* ts_out, hipStream_t s);
// prune -> quantise -> compress in one pass; codes (the pruned tensor's codes) nullable; bad device
hipError_t launch_produce24(const void* W, int w_bf16, int64_t N, int64_t K, const float* ts_in, uint8_t* vals,
                            uint8_t* meta, uint8_t* scales, float* ts_out, uint8_t* codes, int64_t* bad,
                            hipStream_t s);

// 2:4 codec
hipError_t launch_check(const uint8_t* codes, int64_t N, int64_t K, int64_t* bad, int64_t* first,
                        hipStream_t s);
hipError_t launch_compress(const uint8_t* codes, int64_t N, int64_t K, uint8_t* vals, uint8_t* meta,
                           int64_t* bad, hipStream_t s);
hipError_t launch_decompress(const uint8_t* vals, const uint8_t* meta, int64_t N, int64_t K,
                             uint8_t* codes, hipStream_t s);

// products. `w0`/`w1` are (codes, -) for dense and (vals, meta) for 2:4.
struct GemmArgs {
  const uint16_t* X;
  int64_t M, N, K;
  const uint8_t* w0;      // codes [N,K/2] or vals [N,K/4]
  const uint8_t* w1;      // meta [N,K/8] or nullptr
  const uint8_t* scales;  // [N,K/16]
  const float* ts;        // [1]
  void* Y;
  int y_bf16;
};

hipError_t launch_gemv_dense_mfma(const GemmArgs& a, hipStream_t s);     // M <= 16
hipError_t launch_gemv_sp24_smfmac(const GemmArgs& a, hipStream_t s);    // M <= 16, K % 64
hipError_t launch_gemv_sp24_decomp(const GemmArgs& a, hipStream_t s);    // M <= 16
hipError_t launch_gemm_dense_valu(const GemmArgs& a, hipStream_t s);     // any M
hipError_t launch_gemm_sp24_valu(const GemmArgs& a, hipStream_t s);      // any M (skip-and-gather)
hipError_t launch_gemm_dense_mfma(const GemmArgs& a, hipStream_t s);     // 256x256 tiles, any M
hipError_t launch_gemm_sp24_decomp(const GemmArgs& a, hipStream_t s);    // 256x256 tiles, any M
hipError_t launch_gemm_sp24_smfmac(const GemmArgs& a, hipStream_t s);    // 256x256 tiles, any M

// grouped-expert (MoE) path
struct MoeGemmArgs {
  const uint16_t* X;        // activations [x_rows, K] bf16
  int64_t x_rows, K;
  const int32_t* row_token; // [R] source row of each expert-ordered row, or nullptr (identity)
  const int32_t* offsets;   // [E + 1] device
  int E;
  int64_t R, N;             // rows of Y; weight rows per expert (2I for the SiLU-gate form)
  const uint8_t* w0;        // codes [E, N, K/2] or vals [E, N, K/4]
  const uint8_t* w1;        // meta [E, N, K/8] or nullptr
  const uint8_t* scales;    // [E, N, K/16]
  const float* ts;          // [E]
  void* Y;                  // [R, N] (or [R, N/2] for the SiLU-gate form)
  int y_bf16, sparse, silu;
  int ktiled;               // weights (all three arrays) in the 64-k tiled layout [E][K/64][N][piece]
  int smfmac = 0;           // 2:4 tiles on the sparse matrix cores (else expanded to dense)
};

size_t moe_route_workspace(int64_t F, int E);
hipError_t launch_moe_route(const int32_t* ids, int64_t T, int k, int E, int32_t* offsets, int32_t* row_token,
                            int32_t* row_slot, int32_t* row_of, int64_t* bad, void* ws, hipStream_t s);
hipError_t launch_moe_gemm(const MoeGemmArgs& a, hipStream_t s);
// one wave per (expert, 32 weight rows, <= 32 routed rows); N % 32 == 0, K % 64 == 0
hipError_t launch_moe_stream(const MoeGemmArgs& a, hipStream_t s);
hipError_t launch_moe_pack_ktiles(const uint8_t* src, int64_t E, int64_t N, int64_t row_bytes, int64_t piece,
                                  uint8_t* dst, hipStream_t s);
hipError_t launch_moe_combine(const void* Yd, int yd_bf16, int64_t R, const int32_t* row_of, const float* w,
                              int64_t T, int k, int64_t D, float* out, hipStream_t s);

// W4A4 variant (MXFP4 operands on the block-scaled matrix cores)
int64_t mx_tiled_code_bytes(int64_t R, int64_t K);
int64_t mx_tiled_scale_bytes(int64_t R, int64_t K);
hipError_t launch_mx_quantize(const void* V, int v_bf16, int64_t R, int64_t K, int tiled, uint8_t* codes,
                              uint8_t* scales, hipStream_t s);
hipError_t launch_gemm_mx(const uint8_t* xc, const uint8_t* xs, int64_t M, const uint8_t* wc, const uint8_t* ws,
                          int64_t N, int64_t K, void* Y, int y_bf16, hipStream_t s);

// integer 4-bit weights with group scales. Types are the codes of include/ssnvfp4.h (f32 0, bf16 1, f16 2);
// scales are 16-bit (s_type bf16 or f16), zeros nullable (then every zero point is 8)
hipError_t launch_int4_quantize(const void* W, int w_type, int64_t N, int64_t K, int64_t group, uint8_t* codes,
                                uint16_t* scales, int s_type, uint8_t* zeros, hipStream_t s);
hipError_t launch_int4_dequantize(const uint8_t* codes, const uint16_t* scales, int s_type, const uint8_t* zeros,
                                  int64_t N, int64_t K, int64_t group, void* out, int out_type, hipStream_t s);
struct Int4GemvArgs {
  const void* X;            // [x_rows, K] bf16 or f16
  int64_t x_rows, M, N, K;  // M: rows of Y; N: weight rows (per expert)
  int64_t group, groups;    // groups = ceil(K / group)
  const uint8_t* codes;     // [E, N, K/2]
  const uint16_t* scales;   // [E, N, groups]
  const uint8_t* zeros;     // [E, N, groups] or nullptr
  const int32_t* row_token; // grouped: source row of each row, or nullptr (identity)
  const int32_t* offsets;   // grouped: [E + 1] device; nullptr: one weight for every row
  void* Y;                  // [M, N] (or [M, N/2] for the SiLU-gate form)
  int E, x_type, s_type, y_type, silu;
};
hipError_t launch_int4_gemv(const Int4GemvArgs& a, hipStream_t s);
hipError_t launch_int4_wide(const Int4GemvArgs& a, hipStream_t s);   // its part for many rows or a long K

// tokens to expert order and back: row_of[t k + j] is the row of entry (t, j), none outside [0, R)
struct PermuteArgs {
  int64_t T, D, R;
  int k, a_type, b_type;
  const int32_t* row_of;    // [T k]
  const float* w;           // [T k] or nullptr (every weight 1)
  const void* A;            // token side [T, D]: scatter's input; gather: only for dw
  const void* B;            // row side [R, D]: gather's input; scatter: only for dw
  void* A_out;              // gather's output
  void* B_out;              // scatter's output
  float* dw;                // [T k] or nullptr: <A[t], B[row]> of every entry, 0 without a row
};
hipError_t launch_moe_scatter(const PermuteArgs& a, hipStream_t s);
hipError_t launch_moe_gather(const PermuteArgs& a, hipStream_t s);

// 4-bit cache of keys and values in pages (layout in include/ssnvfp4.h), and attention over it
struct KvCache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales;
  const float *k_ts, *v_ts;   // [heads]
  int64_t pages;
  int page, heads, D;         // tokens of a page (a multiple of 16), key heads, width (a multiple of 32, <= 256)
};
struct KvAppendArgs {
  const void *K, *V;          // [T, heads, D] of type, a head's D values contiguous
  int64_t T, k_token, k_head, v_token, v_head;   // strides in elements
  const int64_t* slots;       // [T]: page * tokens of a page + place; negative: no slot
  int64_t* bad;               // [1] or nullptr: slots beyond the cache
  KvCache c;
  int type;
};
struct KvReadArgs {
  const int64_t* slots;
  int64_t T;
  void *K, *V;                // [T, heads, D] contiguous
  KvCache c;
  int type;
};
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);
hipError_t launch_kv_read(const KvReadArgs& a, hipStream_t s);
struct AttnArgs {
  const void* Q;              // [Tq, Hq, D] of q_type, a head's D values contiguous
  int64_t q_token, q_head;    // strides in elements
  void* out;                  // [Tq, Hq, D] contiguous
  float* lse;                 // [Tq, Hq] or nullptr
  KvCache c;
  const int32_t* table;       // [B, max_blocks]
  const int32_t* lens;        // [B]
  const int32_t* q_offsets;   // [B + 1] or nullptr: Tq / B queries each
  int64_t Tq, B, max_blocks, max_q, max_kv;
  int Hq, q_type, out_type, causal, window;
  float scale;
  void* ws;                   // attn_workspace() bytes
};
int64_t attn_workspace(const AttnArgs& a);              // bytes for the partial results, 0 if none are made
bool attn_takes_tile(const AttnArgs& a);                // AUTO's choice
constexpr int64_t kAttnGrid = (int64_t)1 << 23;         // workgroups of 512 threads at most
int64_t attn_workgroups(const AttnArgs& a, bool tile);
hipError_t launch_attn(const AttnArgs& a, bool tile, hipStream_t s);

// calibration: register-resident matrix ops on random operands (cu_count() * waves_per_simd
// workgroups of 256 threads; sink holds one float per thread)
hipError_t launch_mfma_probe(int kind, int waves_per_simd, int iters, uint32_t seed, float* sink, hipStream_t s);

}  // namespace ssn
