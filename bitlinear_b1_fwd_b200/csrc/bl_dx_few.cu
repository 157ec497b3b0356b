// bl_dx_few.cu -- dx = gamma dz W_q for up to 32 tokens, straight from 2-bit weights.
//
//   dx[m, k] = gamma sum_n dz[m, n] W_q[n, k]        dz bf16, codes exact in bf16
//
// The tensor-memory product (bl_gemm_grad.cu) pays for a bf16 copy of the weights
// and tiles of 256 tokens: 16 tokens, 3200 x 8640, 35 us against
// 18 here, 3200 x 3200 23 against 9.  Here packed words go
// from memory to registers and from there into mma.sync (m16n8k16) as its B
// fragment.  A packed word holds 16 neighbouring columns k of one row n; the
// fragment wants rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9 of a column, so lane (g, t)
// keeps word g of those four rows, and digit j of each gives the fragment of
// column 16 g + j: 16 MMAs for four words, 128 columns x 16 rows.  Digits of two
// rows sit in the halves of a register (a shift and a mask with 0x4300, the bf16
// 128 + d, and one subtraction of 129: exact).
//
// A block has 128 columns and a range of rows, which its 8 warps share 16 rows at a
// time, at most kMaxSteps each (short fp32 runs, as in bl_gemm_grad.cu); the
// warps' sums meet in shared memory in warp order, and the blocks' sums of a column
// in a second kernel in block order: the same bits on every call.
#include <cuda_bf16.h>

#include "bl_common.cuh"
#include "bl_kernels.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kDxWarps = 8, kDxThreads = 32 * kDxWarps;
constexpr int kDxCols = 128;     // columns of a block: 8 packed words
constexpr int kMaxSteps = 32;    // steps of 16 rows a warp adds up

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Digit j (2-bit codes q + 1 at bits 2 j of both halves) as two bf16 weights.
__device__ __forceinline__ uint32_t two_weights(uint32_t pair, int j) {
  const uint32_t v = (pair >> (2 * j) & 0x00030003u) | 0x43004300u;  // 128 + d
  const __nv_bfloat162 m = __halves2bfloat162(__ushort_as_bfloat16(0x4301), __ushort_as_bfloat16(0x4301));  // 129
  const __nv_bfloat162 w = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&v), m);
  return *reinterpret_cast<const uint32_t*>(&w);
}

// MB groups of 16 tokens.  Row range of block (x, y): steps [y per, (y + 1) per).
// out: dx (odt) when there is one range, else part[range][m][k] in fp32.
template <int MB>
__global__ void __launch_bounds__(kDxThreads)
    dx_few_kernel(const uint8_t* __restrict__ packed, int64_t rowbytes, const uint16_t* __restrict__ dz,
                  const float* __restrict__ gamma, int M, int64_t N, int64_t K, int steps, int per,
                  void* __restrict__ out, int odt, float* __restrict__ part) {
  pdl_enter(packed, dz, gamma, out, part);
  extern __shared__ __align__(16) float slab[];  // [kDxWarps][16 MB][kDxCols + 1]
  constexpr int kRow = kDxCols + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t word0 = static_cast<int64_t>(blockIdx.x) * (kDxCols / 16);
  const bool has_word = 4 * (word0 + g) < rowbytes;
  const bool even = N % 2 == 0;
  const int s0 = blockIdx.y * per, s1 = s0 + per < steps ? s0 + per : steps;
  float acc[MB][16][4];
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 16; ++j) acc[b][j][0] = acc[b][j][1] = acc[b][j][2] = acc[b][j][3] = 0.0f;
  struct Step {
    uint32_t w[4];       // rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9
    uint32_t a[MB][4];   // (token g, rows 2 t), (g + 8, 2 t), (g, 2 t + 8), (g + 8, 2 t + 8)
  };
  auto fetch = [&](int s, Step& f) {
    const int64_t n0 = 16 * static_cast<int64_t>(s) + 2 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = n0 + (i & 1) + 8 * (i >> 1);
      f.w[i] = 0x55555555u;  // weights 0
      if (s < s1 && has_word && n < N)
        f.w[i] = __ldcg(reinterpret_cast<const uint32_t*>(packed + n * rowbytes) + word0 + g);
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = 16 * b + g + 8 * (i & 1);
        const int64_t n = n0 + 8 * (i >> 1);
        const uint16_t* p = dz + m * N + n;
        f.a[b][i] = 0u;
        if (s < s1 && m < M) {
          if (even) {
            if (n < N) f.a[b][i] = __ldcg(reinterpret_cast<const uint32_t*>(p));
          } else {
            if (n < N) f.a[b][i] = __ldcg(p);
            if (n + 1 < N) f.a[b][i] |= static_cast<uint32_t>(__ldcg(p + 1)) << 16;
          }
        }
      }
  };
  Step next;
  fetch(s0 + warp, next);
  for (int s = s0 + warp; s < s1; s += kDxWarps) {
    const Step f = next;
    fetch(s + kDxWarps, next);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // digits 0..7, then 8..15: two rows' halves of the words side by side
      const uint32_t sel = h == 0 ? 0x5410u : 0x7632u;
      const uint32_t lo = __byte_perm(f.w[0], f.w[1], sel), hi = __byte_perm(f.w[2], f.w[3], sel);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t b0 = two_weights(lo, j), b1 = two_weights(hi, j);
#pragma unroll
        for (int b = 0; b < MB; ++b) mma_bf16(acc[b][8 * h + j], f.a[b], b0, b1);
      }
    }
  }
  // column of acc[.][j][0]: digit j of word 2 t; [1]: of word 2 t + 1; [2], [3]: token g + 8
  float* mine = slab + static_cast<int64_t>(warp) * 16 * MB * kRow;
#pragma unroll
  for (int b = 0; b < MB; ++b)
#pragma unroll
    for (int j = 0; j < 16; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        mine[(16 * b + g + 8 * (c >> 1)) * kRow + 16 * (2 * t + (c & 1)) + j] = acc[b][j][c];
  __syncthreads();
  const float gm = __ldcg(gamma);
  for (int e = threadIdx.x; e < M * kDxCols; e += kDxThreads) {
    const int m = e / kDxCols, c = e % kDxCols;
    const int64_t k = static_cast<int64_t>(blockIdx.x) * kDxCols + c;
    if (k >= K) continue;
    float s = slab[m * kRow + c];
#pragma unroll
    for (int w = 1; w < kDxWarps; ++w) s += slab[(w * 16 * MB + m) * kRow + c];
    if (gridDim.y > 1) {
      part[(static_cast<int64_t>(blockIdx.y) * M + m) * K + k] = s;
    } else {
      s = __fmul_rn(s, gm);
      store_vec_dt<1>(out, odt, m * K + k, &s);
    }
  }
}

template <int MB>
cudaError_t launch_t(const uint8_t* packed, int64_t rowbytes, const uint16_t* dz, const float* gamma, int64_t M, int64_t N,
                     int64_t K, void* dx, int dxdt, float* part, cudaStream_t st) {
  const int64_t steps = (N + 15) / 16, ranges = dx_few_parts(N, K), per = (steps + ranges - 1) / ranges;
  auto kern = dx_few_kernel<MB>;
  const size_t smem = static_cast<size_t>(kDxWarps) * 16 * MB * (kDxCols + 1) * sizeof(float);
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(static_cast<unsigned>((K + kDxCols - 1) / kDxCols), static_cast<unsigned>(ranges)),
                    kDxThreads, smem, st, packed, rowbytes, dz, gamma, static_cast<int>(M), N, K,
                    static_cast<int>(steps), static_cast<int>(per), dx, dxdt, part);
}

}  // namespace

// Row ranges: a block on every SM, no warp with more than kMaxSteps steps, none
// without any.
int64_t dx_few_parts(int64_t N, int64_t K) {
  const int64_t steps = (N + 15) / 16, cols = (K + kDxCols - 1) / kDxCols;
  int64_t r = (device_sms() + cols - 1) / cols;
  const int64_t least = (steps + kDxWarps * kMaxSteps - 1) / (kDxWarps * kMaxSteps);
  const int64_t most = (steps + kDxWarps - 1) / kDxWarps;
  if (r > most) r = most;
  if (r < least) r = least;
  const int64_t per = (steps + r - 1) / r;
  return (steps + per - 1) / per;
}

bool dx_few_fits(int64_t M, int64_t N) { return M <= 32 && N <= int64_t{16} * kDxWarps * kMaxSteps * 65535; }

cudaError_t launch_dx_few(const uint8_t* packed, int64_t rowbytes, const uint16_t* dz, const float* gamma, int64_t M,
                          int64_t N, int64_t K, void* dx, int dxdt, float* part, cudaStream_t st) {
  cudaError_t e = M <= 16 ? launch_t<1>(packed, rowbytes, dz, gamma, M, N, K, dx, dxdt, part, st)
                          : launch_t<2>(packed, rowbytes, dz, gamma, M, N, K, dx, dxdt, part, st);
  const int64_t ranges = dx_few_parts(N, K);
  if (e == cudaSuccess && ranges > 1)
    e = launch_grad_parts(part, static_cast<int>(ranges), M * K, gamma, dx, dxdt, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
