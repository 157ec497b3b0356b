// bl_gemm_few.cu -- the forward product of a few tokens (5 to 64) with its
// epilogue, straight from packed weights of every format.
//
//   acc[t, n] = sum_k x_q[t, k] W_q[n, k];  z = acc c_t + bias_n;  y = act(z) + residual
//
// With this few tokens a layer is its weights' bytes and the latency of getting
// at them, so the kernel keeps them on the shortest way: packed words go from
// memory to registers, are expanded there to int8 and enter mma.sync (m16n8k32)
// as its A fragment; no shared memory, no transcoded copy, no split of K over
// blocks (the tensor-memory kernel of bl_gemm_sm100.cu needs all three: 16
// tokens, 8640 -> 3200 in base 3 took a transcoding, a product and a reduction,
// 28 us; this takes X us).  The order of k within an MMA is free as long as both
// operands agree, so a lane simply owns one 16-byte segment of a row: lanes t =
// 0..3 of a group take segments 4 c + t, and packed word w of it (16 weights)
// feeds two MMAs.  The tokens' codes are laid out to match by act_pieces_kernel:
// pieces of 16 codes in the order [chunk][word][token][t], one coalesced 16-byte
// load per lane for two MMAs of eight tokens.
//
// A block has 16 weight rows; its 16 warps share the chunks of K (and, when
// there are fewer chunks than warps, the token groups), and their INT32 sums meet
// in shared memory by integer adds, whose order does not matter.  Each block
// reads all codes, M K bytes through L2, which is what limits the number of
// tokens it serves well.
#include "bl_common.cuh"
#include "bl_epilogue.cuh"
#include "bl_gemv.cuh"
#include "bl_kernels.h"
#include "bl_sm100.cuh"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewRows = 16;

// 16-weight words in a 16-byte packed segment
__host__ __device__ constexpr int few_words(int fmt) { return fmt == BL_PACK_I2 ? 4 : fmt == BL_PACK_T5 ? 5 : 8; }

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The int8 weights of word w of a segment.  For base 3, seg holds the segment's
// 2-bit words already (see few_segment).
template <int FMT>
struct Segment {
  uint32_t w[FMT == BL_PACK_T5 ? 5 : 4];
  __device__ __forceinline__ void set(const uint4& v) {
    if constexpr (FMT == BL_PACK_T5) {
      t5_segment(v, w);
    } else {
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    }
  }
  __device__ __forceinline__ uint4 weights(int i) const {
    if constexpr (FMT == BL_PACK_B1)
      return expand16_bits((i & 1) ? w[i >> 1] >> 16 : w[i >> 1]);
    else
      return expand16(w[i]);
  }
};

// NB groups of 8 tokens; ns of the 16 warps share a chunk's groups.
template <int FMT, int NB>
__global__ void __launch_bounds__(kFewThreads)
    gemm_few_kernel(const uint8_t* __restrict__ packed, int64_t rowbytes, const float* __restrict__ gamma, int64_t N,
                    const uint4* __restrict__ pieces, const float* __restrict__ scale, void* __restrict__ y, int ydt,
                    int M, int ns, const Epilogue ep_arg) {
  constexpr int W = few_words(FMT);
  constexpr int MB = 8 * NB;
  __shared__ int acc_s[kFewRows][MB + 1];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kFewRows;
  const int rows = N - row0 < kFewRows ? static_cast<int>(N - row0) : kFewRows;
  pdl_launch_dependents();
  l2_prefetch_bulk(packed + row0 * rowbytes, rows * rowbytes);
  for (int i = threadIdx.x; i < kFewRows * (MB + 1); i += kFewThreads) (&acc_s[0][0])[i] = 0;
  pdl_wait(packed, gamma, pieces, scale, y);
  const Epilogue ep = epilogue_after_wait(ep_arg);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int segs = static_cast<int>(rowbytes >> 4), chunks = (segs + 3) >> 2;
  const int kparts = kFewWarps / ns, kp = warp / ns, tp = warp % ns;
  const uint4 pad = FMT == BL_PACK_T5 ? make_uint4(0x79797979u, 0x79797979u, 0x79797979u, 0x79797979u)
                                      : make_uint4(0u, 0u, 0u, 0u);  // (against codes of 0)
  auto fetch = [&](int c, uint4 (&v)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      v[r] = pad;
      if (c < chunks && g + 8 * r < rows && 4 * c + t < segs)
        v[r] = ld_stream(reinterpret_cast<const uint4*>(packed + (row0 + g + 8 * r) * rowbytes) + 4 * c + t);
    }
  };
  int acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b) acc[b][0] = acc[b][1] = acc[b][2] = acc[b][3] = 0;
  uint4 next[2];
  fetch(kp, next);
  for (int c = kp; c < chunks; c += kparts) {
    Segment<FMT> s0, s1;
    s0.set(next[0]);
    s1.set(next[1]);
    fetch(c + kparts, next);
    const uint4* px = pieces + static_cast<int64_t>(c) * W * MB * 4 + 4 * g + t;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 x[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (b % ns == tp) x[b] = __ldcg(px + (w * NB + b) * 32);
      const uint4 a = s0.weights(w), e = s1.weights(w);  // rows g and g + 8
      const uint32_t lo[4] = {a.x, e.x, a.y, e.y}, hi[4] = {a.z, e.z, a.w, e.w};
#pragma unroll
      for (int b = 0; b < NB; ++b)
        if (b % ns == tp) {
          mma_s8(acc[b], lo, x[b].x, x[b].y);
          mma_s8(acc[b], hi, x[b].z, x[b].w);
        }
    }
  }
  if (kp < chunks) {
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (b % ns == tp) {
        atomicAdd(&acc_s[g][8 * b + 2 * t], acc[b][0]);
        atomicAdd(&acc_s[g][8 * b + 2 * t + 1], acc[b][1]);
        atomicAdd(&acc_s[g + 8][8 * b + 2 * t], acc[b][2]);
        atomicAdd(&acc_s[g + 8][8 * b + 2 * t + 1], acc[b][3]);
      }
  }
  __syncthreads();
  const float gm = __ldcg(gamma);
  for (int i = threadIdx.x; i < kFewRows * M; i += kFewThreads) {
    const int r = i % kFewRows, m = i / kFewRows;
    if (r < rows)
      epilogue_store(ep, y, ydt, m * N + row0 + r, row0 + r, acc_s[r][m], dequant_factor(gm, __ldcg(scale + m)));
  }
}

// One token per block: its scale (unless the codes are given, XDT = I8) and its
// codes as pieces of 16, zeros past K: piece s W + w of a row goes to [s / 4][w]
// [token][s % 4].
template <int XDT>
__global__ void __launch_bounds__(512)
    act_pieces_kernel(const void* __restrict__ x, int64_t K, float* __restrict__ scale, uint4* __restrict__ pieces,
                      int words, int64_t chunks, int mb) {
  pdl_enter(x, scale, pieces);
  __shared__ __align__(16) float sum_mem[2][4][32];
  const int64_t m = blockIdx.x;
  const bool wide = K % 8 == 0;
  float s = 1.0f, c127 = 0.0f;
  if constexpr (XDT != BL_I8) {
    BlockSum sum(sum_mem);
    float amax = 0.0f;
    if (wide) {
#pragma unroll 4
      for (int64_t k = 8 * threadIdx.x; k < K; k += 8 * blockDim.x) {
        float v[8];
        load_vec<XDT, 8>(x, m * K + k, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      }
    } else {
#pragma unroll 8
      for (int64_t k = threadIdx.x; k < K; k += blockDim.x) amax = fmaxf(amax, fabsf(load_elem<XDT>(x, m * K + k)));
    }
    s = fmaxf(sum.max(amax), 1e-6f);
    c127 = __fdiv_rn(127.0f, s);
    if (threadIdx.x == 0) scale[m] = s;
  }
  const int64_t total = 4 * chunks * words;
  for (int64_t p = threadIdx.x; p < total; p += blockDim.x) {
    uint32_t o[4];
#pragma unroll
    for (int hv = 0; hv < 2; ++hv) {
      const int64_t k = 16 * p + 8 * hv;
      int q[8];
      if (wide && k < K) {
        if constexpr (XDT == BL_I8) {
          const uint2 raw = __ldcg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(x) + m * K + k));
          o[2 * hv] = raw.x;
          o[2 * hv + 1] = raw.y;
          continue;
        } else {
          float v[8];
          load_vec<XDT, 8>(x, m * K + k, v);
          quant_act_fast_n<8>(v, s, c127, q);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if constexpr (XDT == BL_I8)
            q[j] = k + j < K ? static_cast<int>(__ldcg(static_cast<const signed char*>(x) + m * K + k + j)) : 0;
          else
            q[j] = k + j < K ? quant_act_fast(load_elem<XDT>(x, m * K + k + j), s, c127) : 0;
        }
      }
      o[2 * hv] = pack4(q);
      o[2 * hv + 1] = pack4(q + 4);
    }
    const int64_t sg = p / words;
    const int w = static_cast<int>(p - sg * words);
    pieces[(((sg >> 2) * words + w) * mb + m) * 4 + (sg & 3)] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

int few_groups(int64_t M) { return M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8; }
int64_t few_chunks(int64_t rowbytes) { return (rowbytes / 16 + 3) / 4; }

template <int FMT, int NB>
cudaError_t launch_few(const uint8_t* packed, int64_t rb, const float* gamma, int64_t N, const void* pieces,
                       const float* scale, void* y, int ydt, int64_t M, const Epilogue& ep, cudaStream_t st) {
  const int64_t chunks = few_chunks(rb);
  int ns = 1;  // warps that share a chunk: while some would have none
  while (2 * ns <= NB && kFewWarps / ns > chunks) ns *= 2;
  return launch_pdl(gemm_few_kernel<FMT, NB>, static_cast<unsigned>((N + kFewRows - 1) / kFewRows), kFewThreads, 0, st,
                    packed, rb, gamma, N, static_cast<const uint4*>(pieces), scale, y, ydt, static_cast<int>(M), ns, ep);
}

template <int FMT>
cudaError_t launch_few_fmt(const uint8_t* packed, int64_t rb, const float* gamma, int64_t N, const void* pieces,
                           const float* scale, void* y, int ydt, int64_t M, const Epilogue& ep, cudaStream_t st) {
  switch (few_groups(M)) {
    case 1: return launch_few<FMT, 1>(packed, rb, gamma, N, pieces, scale, y, ydt, M, ep, st);
    case 2: return launch_few<FMT, 2>(packed, rb, gamma, N, pieces, scale, y, ydt, M, ep, st);
    case 4: return launch_few<FMT, 4>(packed, rb, gamma, N, pieces, scale, y, ydt, M, ep, st);
    default: return launch_few<FMT, 8>(packed, rb, gamma, N, pieces, scale, y, ydt, M, ep, st);
  }
}

}  // namespace

size_t gemm_few_bytes(int64_t M, int64_t rowbytes, int fmt) {
  return static_cast<size_t>(few_chunks(rowbytes)) * few_words(fmt) * 8 * few_groups(M) * 4 * 16;
}

cudaError_t launch_gemm_few(const uint8_t* packed, int fmt, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, int64_t M, void* y, int ydt, const Epilogue& ep,
                            void* scratch, cudaStream_t st) {
  auto pieces_kern = xdt == BL_F32 ? act_pieces_kernel<BL_F32> : xdt == BL_BF16 ? act_pieces_kernel<BL_BF16>
                                                                                : act_pieces_kernel<BL_I8>;
  cudaError_t e = launch_pdl(pieces_kern, static_cast<unsigned>(M), 512, 0, st, x, K, scale,
                             static_cast<uint4*>(scratch), few_words(fmt), few_chunks(rowbytes), 8 * few_groups(M));
  if (e != cudaSuccess) return e;
  e = fmt == BL_PACK_I2   ? launch_few_fmt<BL_PACK_I2>(packed, rowbytes, gamma, N, scratch, scale, y, ydt, M, ep, st)
      : fmt == BL_PACK_T5 ? launch_few_fmt<BL_PACK_T5>(packed, rowbytes, gamma, N, scratch, scale, y, ydt, M, ep, st)
                          : launch_few_fmt<BL_PACK_B1>(packed, rowbytes, gamma, N, scratch, scale, y, ydt, M, ep, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
