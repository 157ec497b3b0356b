// bl_kernels.h -- launchers of the BitLinear kernels (internal to the library).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "bitlinear.h"

namespace bl {

// Launch with programmatic stream serialization (see pdl_enter): the kernel
// may be scheduled while the previous kernel in the stream finishes.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_pdl(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                              Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...);
}

// absmean: the last CTA folds 2^lgR chunk sums per lane (lgR <= 11 allows
// 2^19 chunks of 8192 elements, so N*K <= 2^32).
constexpr int kFinishMaxLevels = 11;

// What follows the dequantization of an output: bias [N], act (bl_act; negative:
// nothing follows), residual and kept pre-activation [M, N] of y's type.
struct Epilogue {
  const float* bias;
  const void* res;
  void* pre;
  int act;
};
inline Epilogue no_epilogue() { return Epilogue{nullptr, nullptr, nullptr, -1}; }

// Number of SMs of the current device (cached per device).
constexpr int kMaxDevices = 64;
int device_sms();

// decode GEMV: shared memory for activations, tokens per launch.
constexpr int64_t kGemvSmemBudget = 200 * 1024;
constexpr int kGemvMaxTokens = 4;

// ws: a workspace whose header ticket is zero; partial sums follow the header.
// alpha: when given, the mean of the weights in the same order (the 1-bit
// variant; then the partial sums take 2 C doubles).
cudaError_t launch_absmean(const void* W, int wdt, int64_t N, int64_t K, void* ws, float* gamma,
                           cudaStream_t st, float* alpha = nullptr);
cudaError_t launch_binarize_pack(const void* W, int wdt, int64_t N, int64_t K, const float* alpha, uint8_t* packed,
                                 int8_t* codes, int64_t rowbytes, cudaStream_t st);
cudaError_t launch_b1_to_i2(const uint8_t* b1, int64_t N, int64_t K, int64_t rb1, uint8_t* i2, int64_t rb2,
                            cudaStream_t st);
// ws: a workspace header for device flags, or nullptr (then a bounded wait
// that runs out goes unreported).
cudaError_t launch_ternarize_pack(const void* W, int wdt, int64_t N, int64_t K, const float* gamma,
                                  float eps, int fmt, uint8_t* packed, int8_t* codes, int64_t rowbytes, void* ws,
                                  cudaStream_t st);
cudaError_t launch_pack(const int8_t* codes, int64_t N, int64_t K, int fmt, uint8_t* packed,
                        int64_t rowbytes, void* ws, cudaStream_t st);
cudaError_t launch_ln_quant(const void* x, int xdt, const float* g, const float* b, float eps, int64_t M, int64_t K,
                            uint16_t* y, int8_t* xq, float* scale, cudaStream_t st);
cudaError_t launch_act_quant(const void* x, int xdt, int64_t M, int64_t K, int8_t* xq, float* scale,
                             cudaStream_t st);
int gemv_max_tokens(int fmt, int64_t rowbytes);
bool gemv_epilogue_fits(int64_t M, int64_t N, int64_t rowbytes);
// tcgen05 GEMM on 2-bit weights; limit_cycles <= 0 uses the default wait limit.
int gemm_token_tile(int64_t M);
// y: row t of the output at y + t ldy (ldy >= N).  part: ks x M x N INT32
// partial sums for the split-K one-SM path (ks = gemm_split_k(M, N, K)), or
// nullptr to keep every tile whole.
cudaError_t launch_gemm_i2(const int8_t* xq, const uint8_t* w, int64_t rb, const float* gamma, const float* scale,
                           void* y, int ydt, int64_t M, int64_t N, int64_t K, int64_t ldy, int32_t* part, void* ws,
                           long long limit_cycles, int skip_producer, cudaStream_t st);
int gemm_split_k(int64_t M, int64_t N, int64_t K);
// The product with an epilogue on weights expanded to int8 rows of ldw bytes.
// Its operands: weights as int8 rows of gemm_i8_row bytes, codes in rows of ldx
// bytes (xq null: the codes are there already).
int64_t gemm_i8_row(int64_t K, int fmt);
cudaError_t launch_gemm_operands(const uint8_t* packed, int fmt, int64_t rowbytes, int64_t N, int64_t K, int8_t* w,
                                 const void* x, int xdt, int64_t M, int64_t ldx, int8_t* xq, float* scale,
                                 cudaStream_t st);
cudaError_t launch_gemm_i8(const int8_t* xq, int64_t ldx, const int8_t* w, int64_t ldw, const float* gamma,
                           const float* scale, void* y, int ydt, int64_t M, int64_t N, int64_t K, const Epilogue& ep,
                           int32_t* part, void* ws, long long limit, int skip_producer, cudaStream_t st);
int gemm_i8_parts(int64_t M, int64_t N, int64_t K);  // part: [this][M][N], or unused when 1
// The product with an epilogue of up to 64 tokens, from packed weights; scratch
// of gemm_few_bytes for the tokens' codes.
constexpr int64_t kFewTokens = 64;
size_t gemm_few_bytes(int64_t M, int64_t rowbytes, int fmt);
cudaError_t launch_gemm_few(const uint8_t* packed, int fmt, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, int64_t M, void* y, int ydt, const Epilogue& ep,
                            void* scratch, cudaStream_t st);
cudaError_t launch_t5_to_i2(const uint8_t* t5, int64_t N, int64_t K, int64_t rb5, uint8_t* i2, int64_t rb2,
                            cudaStream_t st);
// Output rows in up to kMaxRowGroups consecutive groups, each with its own
// gamma (row n belongs to the first group g with n < end[g]).
constexpr int kMaxRowGroups = 8;
struct RowGroups {
  int n;
  int64_t end[kMaxRowGroups];
};
// And what follows their dequantization.  Kernels without an epilogue take the
// groups alone: those that look a group up in their argument copy it to local
// memory first, and 32 bytes more took 0.25 to 0.4 us (four tokens, 3200 -> 8640:
// 13.2 us against 13.4).
struct RowGroupsEp : RowGroups {
  Epilogue ep;
};
template <bool EP>
using KernelGroups = typename std::conditional<EP, RowGroupsEp, RowGroups>::type;
__host__ __device__ inline int row_group(const RowGroups& rg, int64_t row) {
  int g = 0;
  while (g + 1 < rg.n && row >= rg.end[g]) ++g;
  return g;
}
inline RowGroupsEp one_group(int64_t N, const Epilogue& ep = no_epilogue()) {
  RowGroupsEp rg{};
  rg.n = 1;
  rg.end[0] = N;
  rg.ep = ep;
  return rg;
}

// STE backward: dx through fp64 partial sums part [chunks][2][K] (chunks =
// backward_dx_chunks(N)); dW straight into dw [N, K].
int64_t backward_dx_chunks(int64_t N);
int backward_dx_tokens_per_pass();
cudaError_t launch_backward_dx(const uint8_t* packed, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                               const void* dy, int dydt, int64_t M, float* dx, double* part, cudaStream_t st);
cudaError_t launch_backward_dw(const void* dy, int dydt, const int8_t* xq, const float* scale, const float* gamma,
                               int64_t M, int64_t N, int64_t K, float* dw, cudaStream_t st);

// Gradients through the forward's epilogue; part: act_grad_row_blocks(M, N)
// rows of N fp32 partial sums (dbias without them when there is one block).
int64_t act_grad_row_blocks(int64_t M, int64_t N);
cudaError_t launch_act_grad(const void* dy, int dydt, const void* z, int zdt, int act, int64_t M, int64_t N, void* dz,
                            float* dbias, float* part, cudaStream_t st);

// The gradient products on the tensor cores.  grad_ld: row stride (elements)
// of a scratch array of n columns.  dx: dz bf16 with row stride lddz (a
// multiple of 8), w the codes in bf16 with row stride ldw; part: ks M K fp32
// where ks = grad_dx_parts(M, N, K) > 1.
int64_t grad_ld(int64_t n);
int grad_dx_parts(int64_t M, int64_t N, int64_t K);
int64_t grad_rowmax_ranges(int64_t M, int64_t N);
cudaError_t launch_i2_to_bf16(const uint8_t* i2, int64_t N, int64_t rowbytes, uint16_t* w, cudaStream_t st);
cudaError_t launch_pad_rows(const uint16_t* src, int64_t M, int64_t N, int64_t ld, uint16_t* dst, cudaStream_t st);
cudaError_t launch_grad_dx(const uint16_t* dz, int64_t lddz, const uint16_t* w, int64_t ldw, const float* gamma,
                           int64_t M, int64_t N, int64_t K, void* dx, int dxdt, float* part, void* ws,
                           cudaStream_t st);
// out = gamma times the ks parts of n values, added in order.
cudaError_t launch_grad_parts(const float* part, int ks, int64_t n, const float* gamma, void* out, int odt,
                              cudaStream_t st);
// dx of a few tokens from 2-bit rows; part: [dx_few_parts(N, K)][M][K] when more than one.
bool dx_few_fits(int64_t M, int64_t N);
int64_t dx_few_parts(int64_t N, int64_t K);
cudaError_t launch_dx_few(const uint8_t* packed, int64_t rowbytes, const uint16_t* dz, const float* gamma, int64_t M,
                          int64_t N, int64_t K, void* dx, int dxdt, float* part, cudaStream_t st);
struct GradDwScratch {
  uint32_t* maxes;  // [grad_rowmax_ranges(M, N)][N]
  float* rowinv;    // [N]
  void *hi, *lo;    // fp16 [M][grad_ld(N)]
  void* x;          // fp16 [M][grad_ld(K)]
};
cudaError_t launch_grad_dw(const uint16_t* dz, const int8_t* xq, const float* scale, const float* gamma, int64_t M,
                           int64_t N, int64_t K, float* dw, const GradDwScratch& s, void* ws, cudaStream_t st);
// Both products on 2 KB at op with their producers switched off (the self test).
cudaError_t launch_grad_selftest(void* op, void* ws, long long limit, cudaStream_t st);

// The norms around a block's end.  Backward scratch: part [norm_grad_blocks(M, K)]
// [4][K], gpart [norm_grad_blocks(M, K) + gate rows][K], stats [M][8] fp32.
using NormParams = bl_residual_norm_params;
cudaError_t launch_residual_norm(const NormParams& p, const void* b, int bdt, const void* r, int rdt, int64_t M,
                                 int64_t K, void* h, void* y, int ydt, int8_t* xq, float* scale, cudaStream_t st);
int64_t norm_grad_blocks(int64_t M, int64_t K);
cudaError_t launch_residual_norm_grad(const NormParams& p, const void* dy, int dydt, const void* dh, const void* b,
                                      int bdt, const void* h, int rdt, int64_t M, int64_t K, void* dr, void* db,
                                      float* dw1, float* db1, float* dgate, float* dw2, float* db2, float* part,
                                      float* gpart, void* stats, cudaStream_t st);

// One-token 2-bit GEMV (column-stationary, early start): K % 16 == 0, rows of
// at most 8192 bytes, and fp32 tokens only when K is small enough for the raw
// token words of a thread to fit (see gemv1_fits).
bool gemv1_fits(int64_t N, int64_t K, int64_t rowbytes, int xdt);
// ws: a workspace header for the device flags (a bounded wait that runs out).
cudaError_t launch_gemv1(const uint8_t* packed, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                         const void* x, int xdt, float* scale, void* y, int ydt, const RowGroupsEp& rg, void* ws,
                         cudaStream_t st);
// The same for one token on base-3 rows (80 weights per 16-byte segment,
// digits decoded by a per-lane shared table): K % 16 == 0 and the table,
// token, ring and row sums within the two-CTAs-per-SM budget.
bool gemv1_t5_fits(int64_t N, int64_t K, int64_t rowbytes, int xdt);
cudaError_t launch_gemv1_t5(const uint8_t* packed, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, void* y, int ydt, const RowGroupsEp& rg, void* ws,
                            cudaStream_t st);
// And on 1-bit rows (128 weights per 16-byte segment, the codes of a column
// in registers in bit-plane order), within the same budget.
bool gemv1_b1_fits(int64_t N, int64_t K, int64_t rowbytes, int xdt);
cudaError_t launch_gemv1_b1(const uint8_t* packed, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, void* y, int ydt, const RowGroupsEp& rg, void* ws,
                            cudaStream_t st);

cudaError_t launch_gemv(const uint8_t* packed, int fmt, const float* gamma, int64_t N, int64_t K,
                        const void* x, int xdt, float* scale, int64_t M, void* y, int ydt,
                        const RowGroupsEp& rg, void* ws, cudaStream_t st);

}  // namespace bl
