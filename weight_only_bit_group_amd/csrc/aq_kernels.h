// Internal launch functions of libaq (host side).  Each enqueues its kernels on
// `stream` and returns the launch status; arguments are validated by the C ABI
// layer before these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace aq {

// sym: the symmetric variant (S = max |v| / 7, codes q + 8, zero point 8)
hipError_t launch_quant_pack(const void* W, bool w_bf16, const float* chan_scale, uint8_t* packed, float* scales,
                             uint8_t* zeros, int64_t N, int64_t K, int group, bool sym, hipStream_t stream);
// E = (q - z) S * chan_rcp - W as two bf16 planes; chan_rcp[k] = fl32(1 / chan_scale[k])
hipError_t launch_quant_error(const void* W, bool w_bf16, const float* chan_scale, const float* chan_rcp, uint16_t* E,
                              int64_t N, int64_t K, int group, hipStream_t stream);
hipError_t launch_w4a16_gemv(const uint16_t* X, int M, int K, const uint8_t* P, const float* S, const uint8_t* Z,
                             int N, int group, float* Y, hipStream_t stream);
// the same products on the matrix cores, M <= 16 (used by the launch_*_gemv dispatchers
// from a few rows up); FP4 needs K % 64 == 0
// true where the LDS-staged matrix-core decode kernel serves a W4A16 product (K = 2048, N >= 8192, M >= 4)
bool w4a16_lds_decode(int M, int N, int K);
hipError_t launch_w4a16_gemv_mfma(const uint16_t* X, int M, int K, const uint8_t* P, const float* S,
                                  const uint8_t* Z, int N, int group, float* Y, hipStream_t stream);
hipError_t launch_w8a16_gemv_mfma(const uint16_t* X, int M, int K, const uint8_t* C, const float* S,
                                  const uint8_t* Z, int N, int group, float* Y, hipStream_t stream);
hipError_t launch_fp4_gemv_mfma(const uint16_t* X, int M, int K, const uint8_t* codes, const uint8_t* bscale,
                                float ts, int N, float* Y, hipStream_t stream);
// the VALU kernels only (any M <= 16)
hipError_t launch_w8a16_gemv_valu(const uint16_t* X, int M, int K, const uint8_t* C, const float* S,
                                  const uint8_t* Z, int N, int group, float* Y, hipStream_t stream);
hipError_t launch_fp4_gemv_valu(const uint16_t* X, int M, int K, const uint8_t* codes, const uint8_t* bscale,
                                float ts, int N, float* Y, hipStream_t stream);
// the VALU kernel only (any M <= 16)
hipError_t launch_w4a16_gemv_valu(const uint16_t* X, int M, int K, const uint8_t* P, const float* S,
                                  const uint8_t* Z, int N, int group, float* Y, hipStream_t stream);
// `staged`: NULL for the fused kernel, else N * K bf16 of device memory that first
// receives the dequantized weights (the staged GEMM then loads them like activations)
// K slices of a W4A16 GEMM with few output tiles (1: none); *kslice = k per slice.  The
// split GEMM writes slices x M x N fp32 partials to `partial` and adds them in order.
int gemm_k_slices(int64_t M, int64_t N, int64_t K, int group, int* kslice);
hipError_t launch_w4a16_gemm(const uint16_t* X, int M, int K, const uint8_t* P, const float* S,
                             const uint8_t* Z, int N, int group, float* Y, uint16_t* staged, float* partial,
                             hipStream_t stream);
// 8-bit codes [N, K] (one byte per weight), S / z as the INT4 format
hipError_t launch_quant_pack8(const void* W, bool w_bf16, const float* chan_scale, uint8_t* codes, float* scales,
                              uint8_t* zeros, int64_t N, int64_t K, int group, hipStream_t stream);
hipError_t launch_w8a16_gemv(const uint16_t* X, int M, int K, const uint8_t* C, const float* S, const uint8_t* Z,
                             int N, int group, float* Y, hipStream_t stream);
// `staged`: N * K bf16 of device memory (always used)
hipError_t launch_w8a16_gemm(const uint16_t* X, int M, int K, const uint8_t* C, const float* S, const uint8_t* Z,
                             int N, int group, float* Y, uint16_t* staged, hipStream_t stream);
hipError_t launch_fp4_gemv(const uint16_t* X, int M, int K, const uint8_t* codes, const uint8_t* bscale, float ts,
                           int N, float* Y, hipStream_t stream);
hipError_t launch_fp4_gemm(const uint16_t* X, int M, int K, const uint8_t* codes, const uint8_t* bscale, float ts,
                           int N, float* Y, uint16_t* staged, hipStream_t stream);
size_t fp4_quantize_workspace_bytes(int64_t N, int64_t K);
// ts: one fp32 on the device (written); partial: fp4_quantize_workspace_bytes of device memory
hipError_t launch_fp4_quantize(const void* W, bool w_bf16, int64_t N, int64_t K, uint8_t* codes, uint8_t* bscale,
                               float* ts, float* partial, hipStream_t stream);
// MXFP4: x_bf16 / y_bf16 false means fp32; ldx in elements
hipError_t launch_mxfp4_quantize(const void* X, bool x_bf16, int64_t M, int64_t K, int64_t ldx, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream);
hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t K, void* Y,
                                   bool y_bf16, hipStream_t stream);
// XS == NULL: X is bf16, else X holds MXFP4 codes and XS their scale bytes; xrow = bytes
// between rows of X.  Grouped: M rows of Y, T rows of X, rows NULL or [M]
hipError_t launch_mxfp4_gemm(const void* X, const uint8_t* XS, int64_t xrow, int M, int K, const uint8_t* codes,
                             const uint8_t* scales, int N, void* Y, bool y_bf16, hipStream_t stream);
hipError_t launch_mxfp4_grouped_gemm(const void* X, const uint8_t* XS, int64_t xrow, int T, int K,
                                     const uint8_t* codes, const uint8_t* scales, int E, int N, const int32_t* offsets,
                                     const int32_t* rows, int M, void* Y, bool y_bf16, hipStream_t stream);
// The kernel form that such a product takes on a device of `cus` compute units (E = 1: dense), and a
// form's description (empty for one that the product does not have, negative past the last): the
// tests hold that every form is run.
extern "C" int mxfp4_form(bool a4, bool grouped, int M, int K, int N, int E, int cus);
extern "C" int mxfp4_form_name(bool a4, bool grouped, int form, char* to, size_t n);
// FP8 blocks: E matrices of N rows, rows ldx elements apart; blocks: one scale for 128 x 128, else for 128 k of a row
hipError_t launch_fp8_quantize(const void* X, bool x_bf16, int64_t E, int64_t N, int64_t K, int64_t ldx, bool blocks,
                               uint8_t* codes, float* scales, hipStream_t stream);
hipError_t launch_fp8_dequantize(const uint8_t* codes, const float* scales, int64_t E, int64_t N, int64_t K, bool blocks,
                                 void* Y, bool y_bf16, hipStream_t stream);
// Products of FP8 rows X [T, K] with scales XS [T, ceil(K / 128)] and weights in 128 x 128 blocks.  offsets NULL: dense
// (E = 1, T = M); else grouped by expert, rows NULL or [M].  bf16 Y is computed by the FP8 matrix instructions, fp32 Y by
// the bf16 ones, or grouped with `fast` by the FP8 ones too
hipError_t launch_fp8_gemm(const uint8_t* X, const float* XS, int T, int K, const uint8_t* codes, const float* scales, int E,
                           int N, const int32_t* offsets, const int32_t* rows, int M, void* Y, bool y_bf16, bool fast,
                           hipStream_t stream);
// The dense product with rows of fp32 or bf16, ldx elements apart, rounded on the way in; room for their codes and scales
hipError_t launch_fp8_linear(const void* X, bool x_bf16, int64_t ldx, int M, int K, const uint8_t* codes, const float* scales,
                             int N, void* Y, bool y_bf16, uint8_t* x_codes, float* x_scales, hipStream_t stream);
// The kernel form that such a product takes on a device of `cus` compute units (E = 1: dense), and a form's
// description (negative past the last): the tests hold that every form is run.
extern "C" int fp8_form(bool y_bf16, bool grouped, int M, int K, int N, int E, int cus);
extern "C" int fp8_form_name(bool y_bf16, int form, char* to, size_t n);
// (of the product with the gated activation: negative where the activation is a kernel of its own)
extern "C" int fp8_gated_form(int M, int K, int I, int E, int cus);
// The first product of an expert's gated MLP with its activation: h = silu(g) u of [g | u] = X times weights [E, 2 I, K]
// by expert with fp32 sums, rounded to FP8 rows (codes [M, I], scales [M, I / 128]); where fp8_gated_fused holds.
bool fp8_gated_fused(int M, int K, int I, int E);
hipError_t launch_fp8_gated(const uint8_t* X, const float* XS, int T, int K, const uint8_t* codes, const float* scales, int E,
                            int I, const int32_t* offsets, const int32_t* rows, int M, uint8_t* h_codes, float* h_scales,
                            hipStream_t stream);
// Routing: T tokens, rows of logits ld elements apart
struct RouteArgs {
  const void* logits;
  const float* bias;   // [E] or NULL
  int64_t T, ld;
  int E, top;
  int groups, top_groups;
  int lanes;           // of a wave for each group (set by the launch)
  uint32_t magic;      // 2^20 over the experts of a group, rounded up (set by the launch)
  bool sigmoid, renormalize;
  float scale;
  int32_t* ids;        // [T, top]
  float* weights;      // [T, top]
};
hipError_t launch_moe_route(RouteArgs a, bool l_bf16, hipStream_t stream);
// dlogits [T, E] in the logits' type
hipError_t launch_moe_route_backward(const RouteArgs& a, bool l_bf16, const float* grad, void* dlogits, hipStream_t stream);
// C choices of experts 0 .. E - 1 (others: none) sorted by expert; work: moe_group_workspace_bytes of device memory
size_t moe_group_workspace_bytes(int64_t C, int E);
hipError_t launch_moe_group(const int32_t* ids, int64_t C, int top, int E, int32_t* offsets, int32_t* rows, int32_t* slots,
                            uint32_t* work, hipStream_t stream);
// the same and, beside it, the T rows X [T, K] of the choices' tokens as FP8 rows
hipError_t launch_moe_group_quantize(const int32_t* ids, int64_t C, int top, int E, int32_t* offsets, int32_t* rows,
                                     int32_t* slots, uint32_t* work, const void* X, bool x_bf16, int64_t T, int64_t K,
                                     int64_t ldx, uint8_t* codes, float* scales, hipStream_t stream);
// rows [gate | up] of 2 I values -> FP8 rows of I; end NULL or the device's count of rows that matter
hipError_t launch_fp8_swiglu_quantize(const void* H, bool h_bf16, int64_t M, int I, const int32_t* end, uint8_t* codes,
                                      float* scales, hipStream_t stream);
hipError_t launch_moe_combine(const void* Y, bool y_bf16, int64_t R, int64_t K, const int32_t* slots, const float* weights,
                              int64_t T, int top, void* out, bool out_bf16, hipStream_t stream);
hipError_t launch_moe_combine_backward(const void* Y, bool y_bf16, int64_t R, int64_t K, const int32_t* slots, int64_t T,
                                       int top, const void* dout, bool dout_bf16, float* dweights, hipStream_t stream);
// compute units of the current device (cached per device)
int device_cu_count();
int64_t sumsq_gemm_blocks(int64_t M, int64_t N);
hipError_t launch_sumsq_gemm(const uint16_t* X, int M, int K, const uint16_t* E, int N, double* partial,
                             hipStream_t stream);
// Gram form of the search's error GEMM: E = the [2][M, K] error planes, H = the [2][K, K]
// bf16 planes of X^T X; partial[sumsq_gemm_blocks(M, K)] gets each tile's sum of
// (E_hi H)[m, j] (E_hi + 2 E_lo)[m, j]
hipError_t launch_gram_gemm(const uint16_t* E, int M, int K, const uint16_t* H, double* partial, hipStream_t stream);
// Y[M, N] = A[M, K] Bm[N, K]^T, bf16 operands (K contiguous, K % 32 == 0), fp32 output
hipError_t launch_bf16_gemm(const uint16_t* A, int M, int K, const uint16_t* Bm, int N, float* Y, hipStream_t stream);
// Xt[K, Tp] = X[T, K]^T with rows T .. Tp - 1 of X taken as zero (Tp % 64 == 0, K % 8 == 0)
hipError_t launch_transpose_pad(const uint16_t* X, int64_t T, int64_t K, int64_t Tp, uint16_t* Xt, hipStream_t stream);
// H[n] (fp32) -> planes[0][n] = bf16(H), planes[1][n] = bf16(H - planes[0]), n < count (count % 4 == 0)
hipError_t launch_split_planes(const float* H, int64_t count, uint16_t* planes, hipStream_t stream);
int absmean_row_slices(int64_t T, int64_t K);
// the allocation-free entry point's scratch: its size, and its device address on the
// current device (looked up once per device)
size_t absmean_scratch_bytes();
hipError_t absmean_scratch(double** ptr);
hipError_t launch_act_absmean(const uint16_t* X, int64_t T, int64_t K, double* sum_abs, float* mean, int64_t count,
                              double* work, hipStream_t stream);
hipError_t launch_fold_norm(const void* w, bool w_bf16, const float* s, int K, float* out, hipStream_t stream);
hipError_t launch_search_select(const double* partial, int nblocks, int n_grid, double count, const float* sgrid,
                                int K, double* mse, int32_t* best, float* best_scale, hipStream_t stream);

}  // namespace aq
