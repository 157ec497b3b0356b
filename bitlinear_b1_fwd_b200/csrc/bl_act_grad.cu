// bl_act_grad.cu -- gradients through the forward product's epilogue.
//
//   dz[m, n] = dy[m, n] act'(z[m, n]),   dbias[n] = sum_m dz[m, n]
//
// One pass over dy and z: bound by HBM (3 values moved per element against
// some 10 operations).  A thread takes 8 neighbouring columns (16-byte loads of
// bf16) and keeps some of its rows in flight, their column sums in registers;
// the activation is a template argument, so the inner loop has no choice in it.
// A block is 32 column threads x 8 row threads over a range of rows; all blocks
// are resident at once (one wave).  A block's 8 row sums meet in shared memory
// and go to a partial row, and column_sum_kernel adds the partial rows in a
// fixed order (no atomics: the same bits on every call).  4096 x 8640 bf16, SiLU:
// 39 us for both kernels, 0.85 of the copy rate; 578 blocks of 64 registers a
// thread (one wave) against 1190 at 72 (three waves at 89 %): 49 us.
#include "bl_common.cuh"
#include "bl_epilogue.cuh"
#include "bl_kernels.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kAgCols = 32, kAgRows = 8;  // threads of a block along columns and rows
constexpr int kAgResident = 4;            // blocks that fit an SM together (64 registers a thread)
// rows a thread has in flight: what its 64 registers hold
constexpr int ag_unroll(int dyt, int zt, int vec) {
  return vec == 1 ? 8 : dyt == BL_F32 || zt == BL_F32 ? 2 : 4;
}

// act'(z), s = 1 / (1 + exp(-z)) and Phi, phi the normal distribution:
//   SiLU  s + z s (1 - s)   within (3 + |z|) 2^-22 s (1 + |z|)
//   GELU  Phi + z phi       within (4 + z^2 / 2) 2^-22 (Phi + |z| phi)
// which is relative to the terms, since they cancel near the slope's zero.  For bf16
// gradients the fast exponential, divide and normal tail: what grows with z is the
// rounding of the exponent, and slopes below 2^-118 may be 0.  That is far under half a
// step of dz, and dbias, an fp32 sum, does not see it (4096 tokens: 1.43e-7 off in the
// 2-norm for SiLU and 1.49e-7 for GELU, with the other forms 1.44e-7 and 1.41e-7: the
// sum's own roundings).  An exponent with its rounding made good took 46 us against
// 38 for SiLU (4096 x 8640) and 55 against 43.5 for GELU, 43 and 54 in packed pairs.
template <int ACT, bool FAST>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (ACT == BL_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == BL_ACT_RELU2) return z > 0.0f ? 2.0f * z : 0.0f;
  if constexpr (ACT == BL_ACT_SILU) {
    if constexpr (FAST) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-z));
      return s * (1.0f + z * (1.0f - s));
    } else {  // e = exp(-|z|) does not overflow: s is q, or e q for z < 0, and s (1 - s) is e q^2
      const float e = expf(-fabsf(z)), q = __fdiv_rn(1.0f, 1.0f + e), eq = e * q;
      return fmaf(z * eq, q, z < 0.0f ? eq : q);
    }
  }
  if constexpr (ACT == BL_ACT_GELU) {  // Phi(z) + z phi(z)
    if constexpr (FAST) {
      float e;
      const float tail = normal_tail(z, &e);
      return fmaf(z, 0.39894228040143268f * e, z < 0.0f ? tail : 1.0f - tail);
    } else {
      return 0.5f * erfcf(-0.70710678118654752f * z) + z * (0.39894228040143268f * expf(-0.5f * z * z));
    }
  }
  return 1.0f;
}

template <int DYT, int ZT, int VEC, int ACT>
__global__ void __launch_bounds__(kAgCols* kAgRows, kAgResident)
    act_grad_kernel(const void* __restrict__ dy, const void* __restrict__ z, int64_t M, int64_t N, int64_t rows_per,
                    void* __restrict__ dz, float* __restrict__ part) {
  pdl_enter(dy, z, dz, part);
  constexpr int kAgUnroll = ag_unroll(DYT, ZT, VEC);
  __shared__ float sums[kAgRows][kAgCols * VEC + 1];
  const int tx = threadIdx.x % kAgCols, ty = threadIdx.x / kAgCols;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * kAgCols + tx) * VEC;
  const int64_t m0 = blockIdx.y * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  float sum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
  auto one = [&](const Raw<DYT, VEC>& rg, const Raw<ZT, VEC>& rz, int64_t e) {
    float g[VEC], v[VEC];
    rg.get(g);
    if constexpr (ACT != BL_ACT_NONE) rz.get(v);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if constexpr (ACT != BL_ACT_NONE) g[j] = __fmul_rn(g[j], act_slope<ACT, DYT == BL_BF16>(v[j]));
      sum[j] += g[j];
    }
    if (dz != nullptr) store_vec<DYT, VEC>(dz, e, g);
  };
  if (n0 < N) {
    int64_t m = m0 + ty;
    const int64_t step = kAgRows * N;
    for (; m + (kAgUnroll - 1) * kAgRows < m1; m += kAgRows * kAgUnroll) {
      Raw<DYT, VEC> rg[kAgUnroll];
      Raw<ZT, VEC> rz[kAgUnroll];
      const int64_t e = m * N + n0;
#pragma unroll
      for (int u = 0; u < kAgUnroll; ++u) {
        rg[u].load(dy, e + u * step);
        if constexpr (ACT != BL_ACT_NONE) rz[u].load(z, e + u * step);
      }
#pragma unroll
      for (int u = 0; u < kAgUnroll; ++u) one(rg[u], rz[u], e + u * step);
    }
    for (; m < m1; m += kAgRows) {
      Raw<DYT, VEC> rg;
      Raw<ZT, VEC> rz;
      rg.load(dy, m * N + n0);
      if constexpr (ACT != BL_ACT_NONE) rz.load(z, m * N + n0);
      one(rg, rz, m * N + n0);
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int j = 0; j < VEC; ++j) sums[ty][tx * VEC + j] = sum[j];
  __syncthreads();
  for (int c = threadIdx.x; c < kAgCols * VEC; c += kAgCols * kAgRows) {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kAgCols * VEC + c;
    if (n < N) {
      float s = 0.0f;
#pragma unroll
      for (int r = 0; r < kAgRows; ++r) s += sums[r][c];
      part[blockIdx.y * N + n] = s;
    }
  }
}

// out[n] = sum over the partial rows in a fixed order: 8 threads per column
// each add every eighth row, their sums meet in order
__global__ void __launch_bounds__(256)
    column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t N, float* __restrict__ out) {
  pdl_enter(part, out);
  __shared__ float sums[8][33];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t n = static_cast<int64_t>(blockIdx.x) * 32 + tx;
  float s = 0.0f;
  if (n < N) {
#pragma unroll 8
    for (int64_t r = ty; r < rows; r += 8) s += __ldcg(part + r * N + n);
  }
  sums[ty][tx] = s;
  __syncthreads();
  if (ty == 0 && n < N) {
    s = 0.0f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += sums[r][tx];
    out[n] = s;
  }
}

int64_t col_blocks(int64_t N, int vec) { return (N + kAgCols * vec - 1) / (kAgCols * vec); }

template <int DYT, int ZT, int VEC>
cudaError_t launch_t(const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz, float* part,
                     int64_t blocks, cudaStream_t st) {
  const int64_t rows_per = (M + blocks - 1) / blocks;
  const dim3 grid(static_cast<unsigned>(col_blocks(N, VEC)), static_cast<unsigned>(blocks));
  auto run = [&](auto kern) { return launch_pdl(kern, grid, kAgCols * kAgRows, 0, st, dy, z, M, N, rows_per, dz, part); };
  switch (act) {
    case BL_ACT_RELU: return run(act_grad_kernel<DYT, ZT, VEC, BL_ACT_RELU>);
    case BL_ACT_RELU2: return run(act_grad_kernel<DYT, ZT, VEC, BL_ACT_RELU2>);
    case BL_ACT_SILU: return run(act_grad_kernel<DYT, ZT, VEC, BL_ACT_SILU>);
    case BL_ACT_GELU: return run(act_grad_kernel<DYT, ZT, VEC, BL_ACT_GELU>);
    default: return run(act_grad_kernel<DYT, DYT, VEC, BL_ACT_NONE>);
  }
}

}  // namespace

// Row blocks: one wave of kAgResident blocks per SM, each of at least kAgRows rows.
int64_t act_grad_row_blocks(int64_t M, int64_t N) {
  const int vec = N % 8 == 0 ? 8 : 1;
  const int64_t want = kAgResident * static_cast<int64_t>(device_sms()) / col_blocks(N, vec);
  const int64_t most = (M + kAgRows - 1) / kAgRows;
  int64_t b = want < most ? want : most;
  if (b > 65535) b = 65535;  // grid.y
  if (b < 1) b = 1;
  const int64_t rows_per = (M + b - 1) / b;  // no block is empty
  return rows_per > 0 ? (M + rows_per - 1) / rows_per : 1;
}

cudaError_t launch_act_grad(const void* dy, int dydt, const void* z, int zdt, int act, int64_t M, int64_t N, void* dz,
                            float* dbias, float* part, cudaStream_t st) {
  const int64_t blocks = act_grad_row_blocks(M, N);
  float* sums = dbias == nullptr ? nullptr : (blocks == 1 ? dbias : part);
  const bool wide = N % 8 == 0;
  cudaError_t e;
#define BL_AG(DYT, ZT)                                                                            \
  e = wide ? launch_t<DYT, ZT, 8>(dy, z, act, M, N, dz, sums, blocks, st)                         \
           : launch_t<DYT, ZT, 1>(dy, z, act, M, N, dz, sums, blocks, st)
  if (dydt == BL_F32 && zdt == BL_F32) {
    BL_AG(BL_F32, BL_F32);
  } else if (dydt == BL_F32) {
    BL_AG(BL_F32, BL_BF16);
  } else if (zdt == BL_F32) {
    BL_AG(BL_BF16, BL_F32);
  } else {
    BL_AG(BL_BF16, BL_BF16);
  }
#undef BL_AG
  if (e != cudaSuccess) return e;
  if (dbias != nullptr && blocks > 1)
    e = launch_pdl(column_sum_kernel, static_cast<unsigned>((N + 31) / 32), 256, 0, st,
                   static_cast<const float*>(part), blocks, N, dbias);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
