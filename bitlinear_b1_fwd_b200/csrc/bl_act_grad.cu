// bl_act_grad.cu -- gradients through the forward product's epilogue.
//
//   dz[m, n] = dy[m, n] act'(z[m, n]),   dbias[n] = sum_m dz[m, n]
//
// One pass over dy and z: bound by HBM (3 values moved per element against
// some 20 operations), so a thread takes 8 neighbouring columns (16-byte loads
// of bf16) of several rows and keeps their column sums in registers.  A block
// is 32 column threads x 8 row threads over a range of rows; its 8 row sums
// meet in shared memory and go to a partial row, and column_sum_kernel adds
// the partial rows in order (no atomics: the same bits on every call).
#include "bl_common.cuh"
#include "bl_epilogue.cuh"
#include "bl_kernels.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kAgCols = 32, kAgRows = 8;  // threads of a block along columns and rows
constexpr int kAgUnroll = 4;              // rows a thread has in flight

// act'(z).  For bf16 gradients the fast exponential and divide: their errors
// (below 2^-20 for |z| < 30) are far under half a bf16 step, 2^-9.
template <bool FAST>
__device__ __forceinline__ float act_slope(int act, float z) {
  switch (act) {
    case BL_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
    case BL_ACT_RELU2: return z > 0.0f ? 2.0f * z : 0.0f;
    case BL_ACT_SILU: {
      const float s = FAST ? __fdividef(1.0f, 1.0f + __expf(-z)) : __fdiv_rn(1.0f, 1.0f + expf(-z));
      return s * (1.0f + z * (1.0f - s));
    }
    case BL_ACT_GELU: {
      const float t = -0.5f * z * z;
      const float pdf = 0.39894228040143268f * (FAST ? __expf(t) : expf(t));
      return 0.5f * erfcf(-0.70710678118654752f * z) + z * pdf;
    }
    default: return 1.0f;
  }
}

template <int DYT, int ZT, int VEC>
__global__ void __launch_bounds__(kAgCols* kAgRows)
    act_grad_kernel(const void* __restrict__ dy, const void* __restrict__ z, int act, int64_t M, int64_t N,
                    int64_t rows_per, void* __restrict__ dz, float* __restrict__ part) {
  pdl_enter(dy, z, dz, part);
  __shared__ float sums[kAgRows][kAgCols * VEC + 1];
  const int tx = threadIdx.x % kAgCols, ty = threadIdx.x / kAgCols;
  const int64_t n0 = (static_cast<int64_t>(blockIdx.x) * kAgCols + tx) * VEC;
  const int64_t m0 = blockIdx.y * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  const bool live = n0 < N;
  float sum[VEC];
#pragma unroll
  for (int j = 0; j < VEC; ++j) sum[j] = 0.0f;
  if (live) {
    for (int64_t m = m0 + ty; m < m1; m += kAgRows * kAgUnroll) {
      float g[kAgUnroll][VEC], v[kAgUnroll][VEC];
#pragma unroll
      for (int u = 0; u < kAgUnroll; ++u) {
        const int64_t e = (m + u * kAgRows) * N + n0;
        if (m + u * kAgRows < m1) {
          load_vec<DYT, VEC>(dy, e, g[u]);
          if (act != BL_ACT_NONE) load_vec<ZT, VEC>(z, e, v[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kAgUnroll; ++u) {
        if (m + u * kAgRows < m1) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            if (act != BL_ACT_NONE) g[u][j] *= act_slope<DYT == BL_BF16>(act, v[u][j]);
            sum[j] += g[u][j];
          }
          if (dz != nullptr) store_vec<DYT, VEC>(dz, (m + u * kAgRows) * N + n0, g[u]);
        }
      }
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

// out[n] = sum over the partial rows, in order
__global__ void __launch_bounds__(128)
    column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t N, float* __restrict__ out) {
  pdl_enter(part, out);
  const int64_t n = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (n >= N) return;
  float s = 0.0f;
#pragma unroll 8
  for (int64_t r = 0; r < rows; ++r) s += __ldcg(part + r * N + n);
  out[n] = s;
}

int64_t col_blocks(int64_t N, int vec) { return (N + kAgCols * vec - 1) / (kAgCols * vec); }

template <int DYT, int ZT, int VEC>
cudaError_t launch_t(const void* dy, const void* z, int act, int64_t M, int64_t N, void* dz, float* part,
                     int64_t blocks, cudaStream_t st) {
  const int64_t rows_per = (M + blocks - 1) / blocks;
  return launch_pdl(act_grad_kernel<DYT, ZT, VEC>,
                    dim3(static_cast<unsigned>(col_blocks(N, VEC)), static_cast<unsigned>(blocks)), kAgCols * kAgRows,
                    0, st, dy, z, act, M, N, rows_per, dz, part);
}

}  // namespace

// Row blocks: enough for eight blocks per SM, each of at least kAgRows rows.
int64_t act_grad_row_blocks(int64_t M, int64_t N) {
  const int vec = N % 8 == 0 ? 8 : 1;
  const int64_t want = (8 * static_cast<int64_t>(device_sms()) + col_blocks(N, vec) - 1) / col_blocks(N, vec);
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
    e = launch_pdl(column_sum_kernel, static_cast<unsigned>((N + 127) / 128), 128, 0, st,
                   static_cast<const float*>(part), blocks, N, dbias);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
