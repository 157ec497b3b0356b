// bl_api.cu -- the C ABI declared in include/bitlinear.h: argument checks on the
// host, workspace carving, and kernel selection.  Nothing here computes.
#include <cmath>
#include <cstring>

#include "bitlinear.h"
#include "bl_common.cuh"
#include "bl_kernels.h"

namespace {

constexpr int64_t kMaxK = int64_t{1} << 20;
constexpr int64_t kMaxNK = int64_t{1} << 32;
// Rows of W (N) and tokens (M) stay below 2^31: the kernels count rows,
// tokens and per-row work items in 32-bit integers (with K = 1, N up to
// 2^32 would satisfy N K <= 2^32 but overflow those counts).
constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int kVersion = 100;  // 0.1.0

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t round256(size_t v) { return (v + 255) / 256 * 256; }
inline bool float_dt(int dt) { return dt == BL_F32 || dt == BL_BF16; }
inline bool fmt_ok(int fmt) { return fmt == BL_PACK_I2 || fmt == BL_PACK_T5 || fmt == BL_PACK_B1; }
inline bool tern_fmt_ok(int fmt) { return fmt == BL_PACK_I2 || fmt == BL_PACK_T5; }  // ternary formats

inline bool act_ok(int act) { return act >= BL_ACT_NONE && act <= BL_ACT_GELU; }
inline bool norm_ok(int kind) { return kind >= BL_NORM_NONE && kind <= BL_NORM_LAYER; }

inline bl_status cuda_status(cudaError_t e) { return e == cudaSuccess ? BL_OK : BL_ERR_CUDA; }

bool nk_ok(int64_t N, int64_t K) {
  if (N < 0 || N > kMaxRows || K < 1 || K > kMaxK) return false;
  return N <= kMaxNK / K;
}

inline bool m_ok(int64_t M) { return M >= 0 && M <= kMaxRows; }

}  // namespace

extern "C" {

int bitlinear_version(void) { return kVersion; }

const char* bitlinear_status_string(int status) {
  switch (status) {
    case BL_OK: return "BL_OK: success";
    case BL_ERR_INVALID_VALUE: return "BL_ERR_INVALID_VALUE: a size, dtype, format or pointer is invalid";
    case BL_ERR_UNSUPPORTED: return "BL_ERR_UNSUPPORTED: valid arguments, but not supported on this device";
    case BL_ERR_MISALIGNED: return "BL_ERR_MISALIGNED: an array pointer is not 16-byte aligned";
    case BL_ERR_WORKSPACE_TOO_SMALL: return "BL_ERR_WORKSPACE_TOO_SMALL: workspace below the queried size";
    case BL_ERR_CUDA: return "BL_ERR_CUDA: a CUDA runtime call failed";
    case BL_ERR_DEVICE_TIMEOUT: return "BL_ERR_DEVICE_TIMEOUT: a bounded wait in a kernel ran out";
    case BL_ERR_BAD_CODE: return "BL_ERR_BAD_CODE: a weight code outside {-1, 0, 1} was packed";
    case BL_ERR_SCRATCH_LIMIT:
      return "BL_ERR_SCRATCH_LIMIT: N*K exceeds the fixed scratch of bitlinear_absmean_noalloc (2^28 elements)";
    default: return "unknown bitlinear status";
  }
}

int64_t bitlinear_packed_row_bytes(int64_t K, int fmt) {
  if (K < 1 || K > kMaxK || !fmt_ok(fmt)) return -1;
  const int64_t per = fmt == BL_PACK_I2 ? 4 : (fmt == BL_PACK_T5 ? 5 : 8);
  return ((K + per - 1) / per + 15) / 16 * 16;
}

size_t bitlinear_quantize_weights_workspace_bytes(int64_t N, int64_t K) {
  if (N < 1 || !nk_ok(N, K)) return 0;
  const int64_t chunks = (N * K + bl::kChunk - 1) / bl::kChunk;
  return BL_WS_HEADER_BYTES + round256(static_cast<size_t>(chunks) * sizeof(double));
}

// The tensor-core path serves more tokens than one GEMV launch holds, when the
// x_q rows can be a TMA tensor (row stride a multiple of 16 bytes).
bool uses_gemm(int64_t M, int64_t K) { return M > bl::kGemvMaxTokens && (K % 16) == 0; }
// 1-bit rows longer than the 1-bit GEMV takes (4096 bytes: K > 32768) are
// transcoded to 2 bits in the workspace for the decode path too.
bool b1_via_i2(int fmt, int64_t K) { return fmt == BL_PACK_B1 && (K + 7) / 8 > 4096; }

size_t bitlinear_forward_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt, int xdt) {
  if (!m_ok(M) || !nk_ok(N, K) || !fmt_ok(fmt)) return 0;
  size_t bytes = BL_WS_HEADER_BYTES;
  if (uses_gemm(M, K)) {
    if (xdt != BL_I8) bytes += round256(static_cast<size_t>(M * K));
    if (fmt != BL_PACK_I2) bytes += round256(static_cast<size_t>(N * bitlinear_packed_row_bytes(K, BL_PACK_I2)));
    const int ks = bl::gemm_split_k(M, N, K);
    if (ks > 1) bytes += round256(static_cast<size_t>(ks) * M * N * sizeof(int32_t));
  } else if (b1_via_i2(fmt, K)) {
    bytes += round256(static_cast<size_t>(N * bitlinear_packed_row_bytes(K, BL_PACK_I2)));
  }
  return bytes;
}

bl_status bitlinear_workspace_init(void* ws, size_t ws_bytes, void* stream) {
  if (ws == nullptr || ws_bytes < BL_WS_HEADER_BYTES) return BL_ERR_INVALID_VALUE;
  return cuda_status(cudaMemsetAsync(ws, 0, BL_WS_HEADER_BYTES, static_cast<cudaStream_t>(stream)));
}

bl_status bitlinear_quantize_weights(const void* W, int wdt, int64_t N, int64_t K, float eps, int fmt,
                                     uint8_t* packed, int8_t* codes, float* gamma, void* ws,
                                     size_t ws_bytes, void* stream) {
  if (W == nullptr || gamma == nullptr || ws == nullptr || (packed == nullptr && codes == nullptr))
    return BL_ERR_INVALID_VALUE;
  if (!float_dt(wdt) || !tern_fmt_ok(fmt) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return BL_ERR_INVALID_VALUE;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(codes, 16) || !aligned(gamma, 4) ||
      !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_quantize_weights_workspace_bytes(N, K)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = bl::launch_absmean(W, wdt, N, K, ws, gamma, st);
  if (e != cudaSuccess) return BL_ERR_CUDA;
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  return cuda_status(bl::launch_ternarize_pack(W, wdt, N, K, gamma, eps, fmt, packed, codes, rb, ws, st));
}

bl_status bitlinear_absmean(const void* W, int wdt, int64_t N, int64_t K, float* gamma, void* ws,
                            size_t ws_bytes, void* stream) {
  if (W == nullptr || gamma == nullptr || ws == nullptr) return BL_ERR_INVALID_VALUE;
  if (!float_dt(wdt) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (!aligned(W, 16) || !aligned(gamma, 4) || !aligned(ws, 16)) return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_quantize_weights_workspace_bytes(N, K)) return BL_ERR_WORKSPACE_TOO_SMALL;
  return cuda_status(bl::launch_absmean(W, wdt, N, K, ws, gamma, static_cast<cudaStream_t>(stream)));
}

bl_status bitlinear_ternarize_pack(const void* W, int wdt, int64_t N, int64_t K, const float* gamma,
                                   float eps, int fmt, uint8_t* packed, int8_t* codes, void* stream) {
  if (W == nullptr || gamma == nullptr || (packed == nullptr && codes == nullptr)) return BL_ERR_INVALID_VALUE;
  if (!float_dt(wdt) || !tern_fmt_ok(fmt) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return BL_ERR_INVALID_VALUE;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(codes, 16) || !aligned(gamma, 4))
    return BL_ERR_MISALIGNED;
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  return cuda_status(bl::launch_ternarize_pack(W, wdt, N, K, gamma, eps, fmt, packed, codes, rb, nullptr,
                                               static_cast<cudaStream_t>(stream)));
}

size_t bitlinear_binarize_weights_workspace_bytes(int64_t N, int64_t K) {
  if (N < 1 || !nk_ok(N, K)) return 0;
  const int64_t chunks = (N * K + bl::kChunk - 1) / bl::kChunk;
  return BL_WS_HEADER_BYTES + round256(static_cast<size_t>(2 * chunks) * sizeof(double));
}

bl_status bitlinear_binarize_weights(const void* W, int wdt, int64_t N, int64_t K, uint8_t* packed, int8_t* codes,
                                     float* beta, float* alpha, void* ws, size_t ws_bytes, void* stream) {
  if (W == nullptr || beta == nullptr || alpha == nullptr || ws == nullptr || (packed == nullptr && codes == nullptr))
    return BL_ERR_INVALID_VALUE;
  if (!float_dt(wdt) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (!aligned(W, 16) || !aligned(packed, 16) || !aligned(codes, 16) || !aligned(beta, 4) || !aligned(alpha, 4) ||
      !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_binarize_weights_workspace_bytes(N, K)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (bl::launch_absmean(W, wdt, N, K, ws, beta, st, alpha) != cudaSuccess) return BL_ERR_CUDA;
  const int64_t rb = bitlinear_packed_row_bytes(K, BL_PACK_B1);
  return cuda_status(bl::launch_binarize_pack(W, wdt, N, K, alpha, packed, codes, rb, st));
}

bl_status bitlinear_pack(const int8_t* codes, int64_t N, int64_t K, int fmt, uint8_t* packed, void* ws,
                         size_t ws_bytes, void* stream) {
  if (!fmt_ok(fmt) || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (N == 0) return BL_OK;
  if (codes == nullptr || packed == nullptr || ws == nullptr) return BL_ERR_INVALID_VALUE;
  if (!aligned(codes, 16) || !aligned(packed, 16) || !aligned(ws, 16)) return BL_ERR_MISALIGNED;
  if (ws_bytes < BL_WS_HEADER_BYTES) return BL_ERR_WORKSPACE_TOO_SMALL;
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  return cuda_status(bl::launch_pack(codes, N, K, fmt, packed, rb, ws, static_cast<cudaStream_t>(stream)));
}

bl_status bitlinear_quantize_acts(const void* x, int xdt, int64_t M, int64_t K, int8_t* xq, float* scale,
                                  void* stream) {
  if (!float_dt(xdt) || !m_ok(M) || K < 1 || K > kMaxK) return BL_ERR_INVALID_VALUE;
  if (M == 0) return BL_OK;
  if (x == nullptr || xq == nullptr || scale == nullptr) return BL_ERR_INVALID_VALUE;
  if (!aligned(x, 16) || !aligned(xq, 16) || !aligned(scale, 4)) return BL_ERR_MISALIGNED;
  return cuda_status(bl::launch_act_quant(x, xdt, M, K, xq, scale, static_cast<cudaStream_t>(stream)));
}

bl_status bitlinear_layernorm_quantize_acts(const void* x, int xdt, const float* ln_w, const float* ln_b, float eps,
                                            int64_t M, int64_t K, uint16_t* y, int8_t* xq, float* scale,
                                            void* stream) {
  if (!float_dt(xdt) || !m_ok(M) || K < 1 || K > kMaxK) return BL_ERR_INVALID_VALUE;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return BL_ERR_INVALID_VALUE;
  if (M == 0) return BL_OK;
  if (x == nullptr || ln_w == nullptr || ln_b == nullptr || xq == nullptr || scale == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(x, 16) || !aligned(ln_w, 4) || !aligned(ln_b, 4) || !aligned(y, 2) || !aligned(scale, 4))
    return BL_ERR_MISALIGNED;
  return cuda_status(bl::launch_ln_quant(x, xdt, ln_w, ln_b, eps, M, K, y, xq, scale, static_cast<cudaStream_t>(stream)));
}

bl_status bitlinear_forward(const uint8_t* packed, int fmt, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, int64_t M, void* y, int ydt, void* ws,
                            size_t ws_bytes, void* stream) {
  if (!fmt_ok(fmt) || !(float_dt(xdt) || xdt == BL_I8) || !(float_dt(ydt) || ydt == BL_I32))
    return BL_ERR_INVALID_VALUE;
  if (!m_ok(M) || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return BL_OK;  // empty output: nothing to read or write
  if (packed == nullptr || gamma == nullptr || x == nullptr || scale == nullptr || y == nullptr ||
      ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scale, 4) ||
      !aligned(gamma, 4) || !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_forward_workspace_bytes(M, N, K, fmt, xdt)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!uses_gemm(M, K)) {
    if (b1_via_i2(fmt, K)) {
      uint8_t* w2 = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
      const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
      if (bl::launch_b1_to_i2(packed, N, K, bitlinear_packed_row_bytes(K, fmt), w2, rb2, st) != cudaSuccess)
        return BL_ERR_CUDA;
      packed = w2;
      fmt = BL_PACK_I2;
    }
    if (bl::gemv_max_tokens(fmt, bitlinear_packed_row_bytes(K, fmt)) < 1) return BL_ERR_UNSUPPORTED;
    return cuda_status(bl::launch_gemv(packed, fmt, gamma, N, K, x, xdt, scale, M, y, ydt,
                                       bl::one_group(N, bl::no_epilogue()), ws, st));
  }
  uint8_t* scratch = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const int8_t* xq = static_cast<const int8_t*>(x);
  if (xdt != BL_I8) {
    if (bl::launch_act_quant(x, xdt, M, K, reinterpret_cast<int8_t*>(scratch), scale, st) != cudaSuccess)
      return BL_ERR_CUDA;
    xq = reinterpret_cast<const int8_t*>(scratch);
    scratch += round256(static_cast<size_t>(M * K));
  }
  const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
  const uint8_t* w2 = packed;
  if (fmt != BL_PACK_I2) {
    const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
    const cudaError_t e = fmt == BL_PACK_T5 ? bl::launch_t5_to_i2(packed, N, K, rb, scratch, rb2, st)
                                            : bl::launch_b1_to_i2(packed, N, K, rb, scratch, rb2, st);
    if (e != cudaSuccess) return BL_ERR_CUDA;
    w2 = scratch;
    scratch += round256(static_cast<size_t>(N * rb2));
  }
  int32_t* part = bl::gemm_split_k(M, N, K) > 1 ? reinterpret_cast<int32_t*>(scratch) : nullptr;
  return cuda_status(bl::launch_gemm_i2(xq, w2, rb2, gamma, scale, y, ydt, M, N, K, N, part, ws, 0, 0, st));
}

// The product with its epilogue has three forms: the decode kernels, the product
// on packed weights (gemm_few) and the product on int8 weights (gemm_i8).
//  - One token: the one-token decode kernel of the format where it takes the
//    shape (3200 -> 8640: 5.5 us against 9.0), else gemm_few.  The base-3 decode
//    kernel first fills a table, so small layers are gemm_few's (512 -> 512: 22.6
//    us against 6.0; 3200 -> 3200: 7.0 and 7.0).
//  - 2 to 4 tokens of 2-bit weights: the decode kernel's time grows with tokens,
//    gemm_few's with the weights (2 tokens: 8.9 us against 9.0 for 3200 -> 8640,
//    7.8 against 5.8 for 3200 -> 3200; 3 tokens: 26.7 against 30.3 for 8192 ->
//    28672, 14.1 against 9.3 for 8640 -> 3200).
//  - Up to 64 tokens, MB of them in groups of 8, 16, 32 or 64: gemm_few takes some
//    3 us + (1.5 + MB / 20 + 0.45 K / 1000) us for each turn of its blocks of 16
//    rows on the SMs (two fit up to MB = 16), gemm_i8 some 11 us (8 more for odd
//    rows) + 2.6 NK / 10^7 us (writing and reading the int8 weights) + 0.27 us a
//    k-block of the busiest SM pair (16 tokens, 3200 -> 8640: 13.0 us against 24.4;
//    64 tokens: 31 against 21.3; 64 tokens, 8192 -> 8192: 38 against 43.6).
enum class ForwardPath { kGemv, kFew, kMany };
static ForwardPath epilogue_path(int64_t M, int64_t N, int64_t K, int fmt, int xdt) {
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  const double nk = static_cast<double>(N) * static_cast<double>(K) * 1e-7;
  if (M == 1) {
    const bool fits = fmt == BL_PACK_I2   ? bl::gemv1_fits(N, K, rb, xdt)
                      : fmt == BL_PACK_T5 ? bl::gemv1_t5_fits(N, K, rb, xdt)
                                          : bl::gemv1_b1_fits(N, K, rb, xdt);
    return fits && (fmt != BL_PACK_T5 || nk >= 0.84) ? ForwardPath::kGemv : ForwardPath::kFew;
  }
  if (M <= bl::kGemvMaxTokens && fmt == BL_PACK_I2 && bl::gemv_epilogue_fits(M, N, rb) &&
      nk * 1e7 >= static_cast<double>(int64_t{1} << (20 + 2 * M)))
    return ForwardPath::kGemv;
  if (M > bl::kFewTokens) return ForwardPath::kMany;
  const int64_t tiles = (N + 255) / 256, ks = bl::gemm_i8_parts(M, N, K), pairs = bl::device_sms() / 2;
  const double mb = M <= 8 ? 8 : M <= 16 ? 16 : M <= 32 ? 32 : 64;
  const int64_t fit = bl::device_sms() * (mb <= 16 ? 2 : 1), turns = ((N + 15) / 16 + fit - 1) / fit;
  const double few = 3 + static_cast<double>(turns) * (1.5 + mb / 20 + 0.00045 * static_cast<double>(K));
  const double many = 11 + (N % 8 != 0 || K % 16 != 0 ? 8 : 0) + 2.6 * nk +
                      0.27 * static_cast<double>((tiles * ks + pairs - 1) / pairs * ((K + 127) / 128 / ks));
  return few <= many ? ForwardPath::kFew : ForwardPath::kMany;
}
static int64_t padded_codes(int64_t K) { return (K + 15) / 16 * 16; }  // TMA rows

size_t bitlinear_forward_epilogue_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt, int xdt) {
  if (!m_ok(M) || !nk_ok(N, K) || !fmt_ok(fmt)) return 0;
  size_t bytes = BL_WS_HEADER_BYTES;
  if (M == 0 || N == 0) return bytes;
  switch (epilogue_path(M, N, K, fmt, xdt)) {
    case ForwardPath::kGemv: return bytes;
    case ForwardPath::kFew: return bytes + bl::gemm_few_bytes(M, bitlinear_packed_row_bytes(K, fmt), fmt);
    default: break;
  }
  if (xdt != BL_I8 || K % 16 != 0) bytes += round256(static_cast<size_t>(M * padded_codes(K)));
  bytes += round256(static_cast<size_t>(N * bl::gemm_i8_row(K, fmt)));
  const int ks = bl::gemm_i8_parts(M, N, K);
  return ks > 1 ? bytes + round256(static_cast<size_t>(ks) * M * N * sizeof(int32_t)) : bytes;
}

bl_status bitlinear_forward_epilogue(const uint8_t* packed, int fmt, const float* gamma, int64_t N, int64_t K,
                                     const void* x, int xdt, float* scale, int64_t M, const float* bias, int act,
                                     const void* residual, void* preact, void* y, int ydt, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!fmt_ok(fmt) || !(float_dt(xdt) || xdt == BL_I8) || !float_dt(ydt) || !act_ok(act)) return BL_ERR_INVALID_VALUE;
  if (preact != nullptr && (preact == y || preact == residual)) return BL_ERR_INVALID_VALUE;
  if (!aligned(bias, 4) || !aligned(residual, 16) || !aligned(preact, 16)) return BL_ERR_MISALIGNED;
  if (!m_ok(M) || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (M == 0 || N == 0) return BL_OK;
  if (packed == nullptr || gamma == nullptr || x == nullptr || scale == nullptr || y == nullptr || ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scale, 4) || !aligned(gamma, 4) ||
      !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_forward_epilogue_workspace_bytes(M, N, K, fmt, xdt)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* scratch = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  const bl::Epilogue ep{bias, residual, preact, act};
  const ForwardPath path = epilogue_path(M, N, K, fmt, xdt);
  if (path == ForwardPath::kFew)
    return cuda_status(bl::launch_gemm_few(packed, fmt, rb, gamma, N, K, x, xdt, scale, M, y, ydt, ep, scratch, st));
  if (path == ForwardPath::kGemv)
    return cuda_status(bl::launch_gemv(packed, fmt, gamma, N, K, x, xdt, scale, M, y, ydt, bl::one_group(N, ep), ws, st));
  const int8_t* xq = static_cast<const int8_t*>(x);
  int8_t* codes = nullptr;
  if (xdt != BL_I8 || K % 16 != 0) {
    xq = codes = reinterpret_cast<int8_t*>(scratch);
    scratch += round256(static_cast<size_t>(M * padded_codes(K)));
  }
  int8_t* w8 = reinterpret_cast<int8_t*>(scratch);
  scratch += round256(static_cast<size_t>(N * bl::gemm_i8_row(K, fmt)));
  if (bl::launch_gemm_operands(packed, fmt, rb, N, K, w8, x, xdt, M, padded_codes(K), codes, scale, st) != cudaSuccess)
    return BL_ERR_CUDA;
  return cuda_status(bl::launch_gemm_i8(xq, padded_codes(K), w8, bl::gemm_i8_row(K, fmt), gamma, scale, y, ydt, M, N, K,
                                        ep, reinterpret_cast<int32_t*>(scratch), ws, 0, 0, st));
}

// Several weight matrices sharing one token batch (for example a block's Q, K
// and V projections): their packed rows are concatenated, each group has its
// own gamma, and y holds the groups' outputs side by side.
static int64_t group_total(int64_t ngroups, const int64_t* group_rows) {
  if (ngroups < 1 || ngroups > bl::kMaxRowGroups || group_rows == nullptr) return -1;
  int64_t n = 0;
  for (int64_t g = 0; g < ngroups; ++g) {
    if (group_rows[g] < 1) return -1;
    n += group_rows[g];
  }
  return n;
}

size_t bitlinear_forward_grouped_workspace_bytes(int64_t M, int64_t ngroups, const int64_t* group_rows, int64_t K,
                                                 int fmt, int xdt) {
  const int64_t N = group_total(ngroups, group_rows);
  if (N < 1 || !m_ok(M) || !nk_ok(N, K) || !fmt_ok(fmt)) return 0;
  size_t bytes = BL_WS_HEADER_BYTES;
  if (uses_gemm(M, K)) {
    if (xdt != BL_I8) bytes += round256(static_cast<size_t>(M * K));
    size_t most = 0;  // the groups run one after another and share the rest
    for (int64_t g = 0; g < ngroups; ++g) {
      const int64_t Ng = group_rows[g];
      size_t e = 0;
      if (fmt != BL_PACK_I2) e += round256(static_cast<size_t>(Ng * bitlinear_packed_row_bytes(K, BL_PACK_I2)));
      const int ks = bl::gemm_split_k(M, Ng, K);
      if (ks > 1) e += round256(static_cast<size_t>(ks) * M * Ng * sizeof(int32_t));
      if (e > most) most = e;
    }
    bytes += most;
  } else if (b1_via_i2(fmt, K)) {
    bytes += round256(static_cast<size_t>(N * bitlinear_packed_row_bytes(K, BL_PACK_I2)));
  }
  return bytes;
}

bl_status bitlinear_forward_grouped(const uint8_t* packed, int fmt, const float* gammas, int64_t ngroups,
                                    const int64_t* group_rows, int64_t K, const void* x, int xdt, float* scale,
                                    int64_t M, void* y, int ydt, void* ws, size_t ws_bytes, void* stream) {
  if (!fmt_ok(fmt) || !(float_dt(xdt) || xdt == BL_I8) || !(float_dt(ydt) || ydt == BL_I32))
    return BL_ERR_INVALID_VALUE;
  const int64_t N = group_total(ngroups, group_rows);
  if (N < 1 || !m_ok(M) || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (M == 0) return BL_OK;
  if (packed == nullptr || gammas == nullptr || x == nullptr || scale == nullptr || y == nullptr || ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 16) || !aligned(scale, 4) || !aligned(gammas, 4) ||
      !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_forward_grouped_workspace_bytes(M, ngroups, group_rows, K, fmt, xdt))
    return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
  if (!uses_gemm(M, K)) {  // one GEMV launch over every group's rows
    if (b1_via_i2(fmt, K)) {
      uint8_t* w2 = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
      if (bl::launch_b1_to_i2(packed, N, K, rb, w2, bitlinear_packed_row_bytes(K, BL_PACK_I2), st) != cudaSuccess)
        return BL_ERR_CUDA;
      packed = w2;
      fmt = BL_PACK_I2;
    }
    if (bl::gemv_max_tokens(fmt, bitlinear_packed_row_bytes(K, fmt)) < 1) return BL_ERR_UNSUPPORTED;
    bl::RowGroupsEp rg{};
    rg.n = static_cast<int>(ngroups);
    rg.ep = bl::no_epilogue();
    int64_t end = 0;
    for (int64_t g = 0; g < ngroups; ++g) rg.end[g] = (end += group_rows[g]);
    return cuda_status(bl::launch_gemv(packed, fmt, gammas, N, K, x, xdt, scale, M, y, ydt, rg, ws, st));
  }
  // one activation quantization, then each group's product into its columns of y
  uint8_t* scratch = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const int8_t* xq = static_cast<const int8_t*>(x);
  if (xdt != BL_I8) {
    if (bl::launch_act_quant(x, xdt, M, K, reinterpret_cast<int8_t*>(scratch), scale, st) != cudaSuccess)
      return BL_ERR_CUDA;
    xq = reinterpret_cast<const int8_t*>(scratch);
    scratch += round256(static_cast<size_t>(M * K));
  }
  const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
  const size_t ysize = (ydt == BL_BF16) ? 2 : 4;
  int64_t off = 0;
  for (int64_t g = 0; g < ngroups; ++g) {
    const int64_t Ng = group_rows[g];
    uint8_t* s2 = scratch;
    const uint8_t* w2 = packed + off * rb;
    if (fmt != BL_PACK_I2) {
      const cudaError_t ce = fmt == BL_PACK_T5 ? bl::launch_t5_to_i2(w2, Ng, K, rb, s2, rb2, st)
                                               : bl::launch_b1_to_i2(w2, Ng, K, rb, s2, rb2, st);
      if (ce != cudaSuccess) return BL_ERR_CUDA;
      w2 = s2;
      s2 += round256(static_cast<size_t>(Ng * rb2));
    }
    int32_t* part = bl::gemm_split_k(M, Ng, K) > 1 ? reinterpret_cast<int32_t*>(s2) : nullptr;
    const bl_status e = cuda_status(bl::launch_gemm_i2(xq, w2, rb2, gammas + g, scale, static_cast<uint8_t*>(y) + off * ysize,
                                                       ydt, M, Ng, K, N, part, ws, 0, 0, st));
    if (e != BL_OK) return e;
    off += Ng;
  }
  return BL_OK;
}

// STE backward.
size_t bitlinear_backward_dx_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt) {
  if (N < 1 || !m_ok(M) || !nk_ok(N, K) || !fmt_ok(fmt)) return 0;
  size_t bytes = BL_WS_HEADER_BYTES;
  if (fmt != BL_PACK_I2) bytes += round256(static_cast<size_t>(N * bitlinear_packed_row_bytes(K, BL_PACK_I2)));
  const int64_t mt = M < bl::backward_dx_tokens_per_pass() ? M : bl::backward_dx_tokens_per_pass();
  bytes += round256(static_cast<size_t>(bl::backward_dx_chunks(N) * mt * K) * sizeof(double));
  return bytes;
}

bl_status bitlinear_backward_dx(const uint8_t* packed, int fmt, const float* gamma, int64_t N, int64_t K,
                                const void* dy, int dydt, int64_t M, float* dx, void* ws, size_t ws_bytes,
                                void* stream) {
  if (!fmt_ok(fmt) || !float_dt(dydt) || !m_ok(M) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (M == 0) return BL_OK;
  if (packed == nullptr || gamma == nullptr || dy == nullptr || dx == nullptr || ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(packed, 16) || !aligned(dy, 16) || !aligned(dx, 16) || !aligned(gamma, 4) || !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_backward_dx_workspace_bytes(M, N, K, fmt)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* scratch = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
  const uint8_t* w2 = packed;
  if (fmt != BL_PACK_I2) {
    const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
    const cudaError_t e = fmt == BL_PACK_T5 ? bl::launch_t5_to_i2(packed, N, K, rb, scratch, rb2, st)
                                            : bl::launch_b1_to_i2(packed, N, K, rb, scratch, rb2, st);
    if (e != cudaSuccess) return BL_ERR_CUDA;
    w2 = scratch;
    scratch += round256(static_cast<size_t>(N * rb2));
  }
  return cuda_status(bl::launch_backward_dx(w2, rb2, gamma, N, K, dy, dydt, M, dx, reinterpret_cast<double*>(scratch), st));
}

bl_status bitlinear_backward_dw(const void* dy, int dydt, const int8_t* xq, const float* scale, const float* gamma,
                                int64_t M, int64_t N, int64_t K, float* dw, void* stream) {
  if (!float_dt(dydt) || !m_ok(M) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (dw == nullptr || gamma == nullptr || (M > 0 && (dy == nullptr || xq == nullptr || scale == nullptr)))
    return BL_ERR_INVALID_VALUE;
  if (!aligned(dy, 16) || !aligned(xq, 16) || !aligned(dw, 16) || !aligned(scale, 4) || !aligned(gamma, 4))
    return BL_ERR_MISALIGNED;
  return cuda_status(bl::launch_backward_dw(dy, dydt, xq, scale, gamma, M, N, K, dw, static_cast<cudaStream_t>(stream)));
}

// Gradients through the epilogue of bitlinear_forward_epilogue.
size_t bitlinear_epilogue_backward_workspace_bytes(int64_t M, int64_t N) {
  if (!m_ok(M) || N < 1 || N > kMaxRows) return 0;
  return BL_WS_HEADER_BYTES + round256(static_cast<size_t>(bl::act_grad_row_blocks(M, N)) * N * sizeof(float));
}

bl_status bitlinear_epilogue_backward(const void* dy, int dydt, const void* z, int zdt, int act, int64_t M, int64_t N,
                                      void* dz, float* dbias, void* ws, size_t ws_bytes, void* stream) {
  if (!float_dt(dydt) || !float_dt(zdt) || !act_ok(act) || !m_ok(M) || N < 1 || N > kMaxRows)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(dbias, 4)) return BL_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) return dbias == nullptr ? BL_OK : cuda_status(cudaMemsetAsync(dbias, 0, N * sizeof(float), st));
  if (dz == nullptr && dbias == nullptr) return BL_ERR_INVALID_VALUE;
  if (dy == nullptr || (act != BL_ACT_NONE && z == nullptr) || ws == nullptr) return BL_ERR_INVALID_VALUE;
  if (z != nullptr && dz == z) return BL_ERR_INVALID_VALUE;
  if (!aligned(dy, 16) || !aligned(z, 16) || !aligned(dz, 16) || !aligned(ws, 16)) return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_epilogue_backward_workspace_bytes(M, N)) return BL_ERR_WORKSPACE_TOO_SMALL;
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES);
  return cuda_status(bl::launch_act_grad(dy, dydt, z, zdt, act, M, N, dz, dbias, part, st));
}

// The gradient products on the tensor cores.
size_t bitlinear_backward_dx_bf16_workspace_bytes(int64_t M, int64_t N, int64_t K, int fmt) {
  if (N < 1 || !m_ok(M) || !nk_ok(N, K) || !fmt_ok(fmt)) return 0;
  const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
  size_t bytes = BL_WS_HEADER_BYTES;
  if (fmt != BL_PACK_I2) bytes += round256(static_cast<size_t>(N) * rb2);
  if (bl::dx_few_fits(M, N)) {
    const int64_t parts = bl::dx_few_parts(N, K);
    return parts > 1 ? bytes + round256(static_cast<size_t>(parts) * M * K * sizeof(float)) : bytes;
  }
  bytes += round256(static_cast<size_t>(N) * bl::grad_ld(K) * 2);
  if (N % 8 != 0) bytes += round256(static_cast<size_t>(M) * bl::grad_ld(N) * 2);
  const int ks = bl::grad_dx_parts(M, N, K);
  if (ks > 1) bytes += round256(static_cast<size_t>(ks) * M * K * sizeof(float));
  return bytes;
}

bl_status bitlinear_backward_dx_bf16(const uint8_t* packed, int fmt, const float* gamma, int64_t N, int64_t K,
                                     const void* dz, int64_t M, void* dx, int dxdt, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!fmt_ok(fmt) || !float_dt(dxdt) || !m_ok(M) || N < 1 || !nk_ok(N, K)) return BL_ERR_INVALID_VALUE;
  if (M == 0) return BL_OK;
  if (packed == nullptr || gamma == nullptr || dz == nullptr || dx == nullptr || ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(packed, 16) || !aligned(dz, 16) || !aligned(dx, 16) || !aligned(gamma, 4) || !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_backward_dx_bf16_workspace_bytes(M, N, K, fmt)) return BL_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint8_t* scratch = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const int64_t rb2 = bitlinear_packed_row_bytes(K, BL_PACK_I2);
  const uint8_t* w2 = packed;
  if (fmt != BL_PACK_I2) {
    const int64_t rb = bitlinear_packed_row_bytes(K, fmt);
    const cudaError_t e = fmt == BL_PACK_T5 ? bl::launch_t5_to_i2(packed, N, K, rb, scratch, rb2, st)
                                            : bl::launch_b1_to_i2(packed, N, K, rb, scratch, rb2, st);
    if (e != cudaSuccess) return BL_ERR_CUDA;
    w2 = scratch;
    scratch += round256(static_cast<size_t>(N) * rb2);
  }
  if (bl::dx_few_fits(M, N))
    return cuda_status(bl::launch_dx_few(w2, rb2, static_cast<const uint16_t*>(dz), gamma, M, N, K, dx, dxdt,
                                         reinterpret_cast<float*>(scratch), st));
  const int64_t ldw = bl::grad_ld(K);
  uint16_t* w16 = reinterpret_cast<uint16_t*>(scratch);
  if (bl::launch_i2_to_bf16(w2, N, rb2, w16, st) != cudaSuccess) return BL_ERR_CUDA;
  scratch += round256(static_cast<size_t>(N) * ldw * 2);
  const uint16_t* g = static_cast<const uint16_t*>(dz);
  int64_t ldg = N;
  if (N % 8 != 0) {  // TMA rows are multiples of 16 bytes
    ldg = bl::grad_ld(N);
    uint16_t* padded = reinterpret_cast<uint16_t*>(scratch);
    if (bl::launch_pad_rows(g, M, N, ldg, padded, st) != cudaSuccess) return BL_ERR_CUDA;
    g = padded;
    scratch += round256(static_cast<size_t>(M) * ldg * 2);
  }
  return cuda_status(bl::launch_grad_dx(g, ldg, w16, ldw, gamma, M, N, K, dx, dxdt, reinterpret_cast<float*>(scratch),
                                        ws, st));
}

size_t bitlinear_backward_dw_bf16_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (N < 1 || !m_ok(M) || !nk_ok(N, K)) return 0;
  return BL_WS_HEADER_BYTES + round256(static_cast<size_t>(bl::grad_rowmax_ranges(M, N)) * N * 4) +
         round256(static_cast<size_t>(N) * 4) + 2 * round256(static_cast<size_t>(M) * bl::grad_ld(N) * 2) +
         round256(static_cast<size_t>(M) * bl::grad_ld(K) * 2);
}

bl_status bitlinear_backward_dw_bf16(const void* dz, const int8_t* xq, const float* scale, const float* gamma,
                                     int64_t M, int64_t N, int64_t K, float* dw, void* ws, size_t ws_bytes,
                                     void* stream) {
  if (!m_ok(M) || N < 1 || !nk_ok(N, K) || dw == nullptr) return BL_ERR_INVALID_VALUE;
  if (!aligned(dw, 16)) return BL_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) return cuda_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(N) * K * sizeof(float), st));
  if (dz == nullptr || xq == nullptr || scale == nullptr || gamma == nullptr || ws == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(dz, 16) || !aligned(xq, 16) || !aligned(scale, 4) || !aligned(gamma, 4) || !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  if (ws_bytes < bitlinear_backward_dw_bf16_workspace_bytes(M, N, K)) return BL_ERR_WORKSPACE_TOO_SMALL;
  uint8_t* p = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  auto take = [&p](size_t bytes) {
    uint8_t* q = p;
    p += round256(bytes);
    return q;
  };
  bl::GradDwScratch s;
  s.maxes = reinterpret_cast<uint32_t*>(take(static_cast<size_t>(bl::grad_rowmax_ranges(M, N)) * N * 4));
  s.rowinv = reinterpret_cast<float*>(take(static_cast<size_t>(N) * 4));
  s.hi = take(static_cast<size_t>(M) * bl::grad_ld(N) * 2);
  s.lo = take(static_cast<size_t>(M) * bl::grad_ld(N) * 2);
  s.x = take(static_cast<size_t>(M) * bl::grad_ld(K) * 2);
  return cuda_status(bl::launch_grad_dw(static_cast<const uint16_t*>(dz), xq, scale, gamma, M, N, K, dw, s, ws, st));
}

// The norms around a block's end.
static bl_status residual_norm_params_ok(const bl_residual_norm_params* p) {
  if (p == nullptr || !norm_ok(p->post) || !norm_ok(p->pre)) return BL_ERR_INVALID_VALUE;
  if (p->post != BL_NORM_NONE && (!(p->post_eps > 0.0f) || !std::isfinite(p->post_eps))) return BL_ERR_INVALID_VALUE;
  if (p->pre != BL_NORM_NONE && (!(p->pre_eps > 0.0f) || !std::isfinite(p->pre_eps))) return BL_ERR_INVALID_VALUE;
  if (!std::isfinite(p->res_scale) || !std::isfinite(p->branch_scale)) return BL_ERR_INVALID_VALUE;
  if (p->gate != nullptr && p->gate_rows < 1) return BL_ERR_INVALID_VALUE;
  if (!aligned(p->post_w, 4) || !aligned(p->post_b, 4) || !aligned(p->gate, 4) || !aligned(p->pre_w, 4) ||
      !aligned(p->pre_b, 4))
    return BL_ERR_MISALIGNED;
  return BL_OK;
}
// gate rows past the last token are not looked at: counts beyond M act as M
static bl_residual_norm_params clamp_gate(const bl_residual_norm_params& p, int64_t M) {
  bl_residual_norm_params q = p;
  if (q.gate == nullptr || q.gate_rows > M) q.gate_rows = M;
  return q;
}

bl_status bitlinear_residual_norm(const bl_residual_norm_params* p, const void* b, int bdt, const void* r, int rdt,
                                  int64_t M, int64_t K, void* h, void* y, int ydt, int8_t* xq, float* scale,
                                  void* stream) {
  if (!float_dt(bdt) || !float_dt(rdt) || (y != nullptr && !float_dt(ydt)) || !m_ok(M) || K < 1 || K > kMaxK)
    return BL_ERR_INVALID_VALUE;
  const bl_status ps = residual_norm_params_ok(p);
  if (ps != BL_OK) return ps;
  if (M == 0) return BL_OK;
  if ((h == nullptr && y == nullptr && xq == nullptr) || (xq == nullptr) != (scale == nullptr))
    return BL_ERR_INVALID_VALUE;
  if (b == nullptr || r == nullptr || y == b || y == r || (y != nullptr && y == h) || h == b)
    return BL_ERR_INVALID_VALUE;
  if (!aligned(b, 16) || !aligned(r, 16) || !aligned(h, 16) || !aligned(y, 16) || !aligned(xq, 16) ||
      !aligned(scale, 4))
    return BL_ERR_MISALIGNED;
  return cuda_status(bl::launch_residual_norm(clamp_gate(*p, M), b, bdt, r, rdt, M, K, h, y, ydt, xq, scale,
                                              static_cast<cudaStream_t>(stream)));
}

size_t bitlinear_residual_norm_backward_workspace_bytes(int64_t M, int64_t K, int64_t gate_rows) {
  if (!m_ok(M) || K < 1 || K > kMaxK || gate_rows < 0) return 0;
  if (M == 0) return BL_WS_HEADER_BYTES;
  const int64_t blocks = bl::norm_grad_blocks(M, K);
  const int64_t per = gate_rows > M ? M : gate_rows;
  const int64_t gates = per > 0 ? blocks + (M + per - 1) / per : 0;
  return BL_WS_HEADER_BYTES + round256(static_cast<size_t>(blocks) * 4 * K * sizeof(float)) +
         round256(static_cast<size_t>(gates) * K * sizeof(float)) + round256(static_cast<size_t>(M) * 8 * sizeof(float));
}

bl_status bitlinear_residual_norm_backward(const bl_residual_norm_params* p, const void* dy, int dydt, const void* dh,
                                           const void* b, int bdt, const void* h, int rdt, int64_t M, int64_t K,
                                           void* dr, void* db, const bl_residual_norm_grads* g, void* ws,
                                           size_t ws_bytes, void* stream) {
  if (!float_dt(dydt) || !float_dt(bdt) || !float_dt(rdt) || !m_ok(M) || K < 1 || K > kMaxK || g == nullptr)
    return BL_ERR_INVALID_VALUE;
  const bl_status ps = residual_norm_params_ok(p);
  if (ps != BL_OK) return ps;
  if (g->dgate != nullptr && p->gate == nullptr) return BL_ERR_INVALID_VALUE;
  if (!aligned(g->dpost_w, 4) || !aligned(g->dpost_b, 4) || !aligned(g->dgate, 4) || !aligned(g->dpre_w, 4) ||
      !aligned(g->dpre_b, 4))
    return BL_ERR_MISALIGNED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {
    float* const sums[5] = {g->dpost_w, g->dpost_b, g->dgate, g->dpre_w, g->dpre_b};  // (one gate row)
    for (float* s : sums)
      if (s != nullptr && cudaMemsetAsync(s, 0, K * sizeof(float), st) != cudaSuccess) return BL_ERR_CUDA;
    return BL_OK;
  }
  if (dr == nullptr && db == nullptr && g->dpost_w == nullptr && g->dpost_b == nullptr && g->dgate == nullptr &&
      g->dpre_w == nullptr && g->dpre_b == nullptr)
    return BL_ERR_INVALID_VALUE;
  if (dy == nullptr || b == nullptr || h == nullptr || ws == nullptr) return BL_ERR_INVALID_VALUE;
  // in place: dr over dh, and db over dy of the same type; an output over anything else is refused
  if (dr != nullptr && (dr == dy || dr == b || dr == h || dr == db)) return BL_ERR_INVALID_VALUE;
  if (db != nullptr && (db == dh || db == b || db == h || (db == dy && bdt != dydt))) return BL_ERR_INVALID_VALUE;
  if (!aligned(dy, 16) || !aligned(dh, 16) || !aligned(b, 16) || !aligned(h, 16) || !aligned(dr, 16) ||
      !aligned(db, 16) || !aligned(ws, 16))
    return BL_ERR_MISALIGNED;
  const int64_t gate_rows = p->gate != nullptr ? (p->gate_rows > M ? M : p->gate_rows) : 0;
  const size_t need = bitlinear_residual_norm_backward_workspace_bytes(M, K, gate_rows);
  if (ws_bytes < need) return BL_ERR_WORKSPACE_TOO_SMALL;
  const int64_t blocks = bl::norm_grad_blocks(M, K);
  const int64_t gates = gate_rows > 0 ? blocks + (M + gate_rows - 1) / gate_rows : 0;
  uint8_t* s = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  float* part = reinterpret_cast<float*>(s);
  s += round256(static_cast<size_t>(blocks) * 4 * K * sizeof(float));
  float* gpart = reinterpret_cast<float*>(s);
  s += round256(static_cast<size_t>(gates) * K * sizeof(float));
  return cuda_status(bl::launch_residual_norm_grad(clamp_gate(*p, M), dy, dydt, dh, b, bdt, h, rdt, M, K, dr, db,
                                                   g->dpost_w, g->dpost_b, g->dgate, g->dpre_w, g->dpre_b, part, gpart,
                                                   s, st));
}

bl_status bitlinear_selftest_wait_timeout(void* ws, size_t ws_bytes, void* stream) {
  // 16 tokens x 128 rows x 128 K: the header plus 8 KB, whose first floats the kernels may read as gamma and
  // scales; the operands are never touched
  if (ws == nullptr || ws_bytes < BL_WS_HEADER_BYTES + 8192) return BL_ERR_INVALID_VALUE;
  if (!aligned(ws, 16)) return BL_ERR_MISALIGNED;
  uint8_t* op = static_cast<uint8_t*>(ws) + BL_WS_HEADER_BYTES;
  const float* g = reinterpret_cast<const float*>(op);
  const int8_t* x = reinterpret_cast<const int8_t*>(op);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  constexpr long long kLimit = 1ll << 20;
  cudaError_t e = bl::launch_gemm_i2(x, op, 32, g, g, op, BL_I32, 16, 128, 128, 128, nullptr, ws, kLimit, 1, st);
  if (e == cudaSuccess)
    e = bl::launch_gemm_i8(x, 128, x, 128, g, g, op, BL_F32, 16, 64, 128, bl::Epilogue{nullptr, nullptr, nullptr, BL_ACT_NONE},
                           nullptr, ws, kLimit, 1, st);
  return cuda_status(e == cudaSuccess ? bl::launch_grad_selftest(op, ws, kLimit, st) : e);
}

bl_status bitlinear_device_status(void* ws, void* stream) {
  if (ws == nullptr) return BL_ERR_INVALID_VALUE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint32_t h[2] = {0, 0};
  if (cudaMemcpyAsync(h, ws, sizeof h, cudaMemcpyDeviceToHost, st) != cudaSuccess) return BL_ERR_CUDA;
  if (cudaStreamSynchronize(st) != cudaSuccess) return BL_ERR_CUDA;
  if (h[0] != 0) {
    if (cudaMemsetAsync(ws, 0, sizeof h, st) != cudaSuccess) return BL_ERR_CUDA;
    if (cudaStreamSynchronize(st) != cudaSuccess) return BL_ERR_CUDA;
  }
  if (h[0] & bl::kFlagTimeout) return BL_ERR_DEVICE_TIMEOUT;
  if (h[0] & bl::kFlagBadCode) return BL_ERR_BAD_CODE;
  return BL_OK;
}

}  // extern "C"
