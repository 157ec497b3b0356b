// bl_gemm_few.cu -- the forward product of a few tokens (up to 64) with its
// epilogue, straight from packed weights of every format.
//
//   acc[t, n] = sum_k x_q[t, k] W_q[n, k];  z = acc c_t + bias_n;  y = act(z) + residual
//
// With this few tokens a layer is its weights' bytes and the latency of getting
// at them, so the kernel keeps them on the shortest way: packed words go from
// memory to registers, are taken apart there and enter mma.sync (m16n8k32) as its
// A fragment; no shared memory, no transcoded copy, no split of K over blocks (the
// tensor-memory kernel of bl_gemm_sm100.cu needs all three: 16 tokens, 8640 ->
// 3200 in base 3 took a transcoding, a product and a reduction, 28 us; this takes
// 12.5).  A lane owns 16-byte segments of two rows: lanes t = 0..3 of a group take
// segments 4 c + t.  The order of k within an MMA is free as long as both operands
// agree, so a register of A holds whatever four weights one instruction yields,
// as digits d >= 0 with q = d - 1 (2-bit: the four codes at one position of a
// word's bytes; base 3: one digit of its four bytes; 1-bit: one bit of them, q =
// 2 d - 1); sum q x = sum d x - sum x, with sum x of each token formed once.  The
// tokens' codes are laid out to match by act_pieces_kernel: pieces of 16 codes (four
// registers) in the order [chunk][piece][token][t], one coalesced 16-byte load per
// lane for two MMAs of eight tokens.
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

// pieces of 16 weights in a 16-byte packed segment
__host__ __device__ constexpr int few_pieces(int fmt) { return fmt == BL_PACK_I2 ? 4 : fmt == BL_PACK_T5 ? 5 : 8; }

__device__ __forceinline__ void mma_s8(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The digits of a segment; piece(i) is four registers of them.
template <int FMT>
struct Segment {
  uint32_t w[4];
  __device__ __forceinline__ void set(const uint4& v) {
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
  __device__ __forceinline__ uint4 piece(int i) const {
    if constexpr (FMT == BL_PACK_I2) {  // byte b of register j: code 4 b + j of word i
      const uint32_t v = w[i], m = 0x03030303u;
      return make_uint4(v & m, v >> 2 & m, v >> 4 & m, v >> 6 & m);
    } else {  // byte b of register j: bit 8 b + 4 (i mod 2) + j of word i / 2
      const uint32_t v = w[i >> 1] >> (4 * (i & 1)), m = 0x01010101u;
      return make_uint4(v & m, v >> 1 & m, v >> 2 & m, v >> 3 & m);
    }
  }
};
// Base 3: byte b of register 5 w + j is digit j of byte b of word w.  d_j = q_j -
// 3 q_{j+1} with q_j = floor(byte / 3^j) by multiplies (see t5_pair), two bytes in
// the halves of a register; bytes 243..255 are five zero weights.
template <>
struct Segment<BL_PACK_T5> {
  uint32_t d[20];
  __device__ __forceinline__ void set(const uint4& v) {
    const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t q[2][6];
#pragma unroll
      for (int h = 0; h < 2; ++h) {  // bytes 0 and 2, then 1 and 3
        uint32_t x = wd[i] >> (8 * h) & 0x00ff00ffu;
        const uint32_t over = ((x + 0x000d000du) >> 8 & 0x00010001u) * 0xffu;
        q[h][0] = (x & ~over) | (0x00790079u & over);
#pragma unroll
        for (int j = 0; j < 4; ++j) q[h][j + 1] = (q[h][j] * 171u >> 9) & 0x007f007fu;
        q[h][5] = 0;
      }
#pragma unroll
      for (int j = 0; j < 5; ++j) {
        const uint32_t lo = q[0][j] - 3u * q[0][j + 1], hi = q[1][j] - 3u * q[1][j + 1];
        d[5 * i + j] = lo + (hi << 8);
      }
    }
  }
  __device__ __forceinline__ uint4 piece(int i) const { return make_uint4(d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]); }
};

// NB groups of 8 tokens; ns of the 16 warps share a chunk's groups.
template <int FMT, int NB>
__global__ void __launch_bounds__(kFewThreads)
    gemm_few_kernel(const uint8_t* __restrict__ packed, int64_t rowbytes, const float* __restrict__ gamma, int64_t N,
                    const uint4* __restrict__ pieces, const int* __restrict__ sums, const float* __restrict__ scale,
                    void* __restrict__ y, int ydt, int M, int ns, const Epilogue ep_arg) {
  constexpr int W = few_pieces(FMT);
  constexpr int MB = 8 * NB;
  __shared__ int acc_s[kFewRows][MB + 1];
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * kFewRows;
  const int rows = N - row0 < kFewRows ? static_cast<int>(N - row0) : kFewRows;
  pdl_launch_dependents();
  l2_prefetch_bulk(packed + row0 * rowbytes, rows * rowbytes);
  for (int i = threadIdx.x; i < kFewRows * (MB + 1); i += kFewThreads) (&acc_s[0][0])[i] = 0;
  pdl_wait(packed, gamma, pieces, sums, scale, y);
  const Epilogue ep = epilogue_after_wait(ep_arg);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int segs = static_cast<int>(rowbytes >> 4), chunks = (segs + 3) >> 2;
  const int kparts = kFewWarps / ns, kp = warp / ns, tp = warp % ns;
  auto fetch = [&](int c, uint4 (&v)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      v[r] = make_uint4(0u, 0u, 0u, 0u);  // (against codes of 0)
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
      const uint4 a = s0.piece(w), e = s1.piece(w);  // rows g and g + 8
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
      epilogue_store(ep, y, ydt, m * N + row0 + r, row0 + r,
                     (FMT == BL_PACK_B1 ? 2 * acc_s[r][m] : acc_s[r][m]) - __ldcg(sums + m),
                     dequant_factor(gm, __ldcg(scale + m)));
  }
}

// One token per block: its scale (unless the codes are given, XDT = I8), its codes
// as pieces of 16 (zeros past K), piece i of segment sg at [sg / 4][i][token][sg %
// 4], and their sum.  The codes of 128 segments at a time turn around in shared
// memory; a row's first such part is read once and kept in registers.
constexpr int kPieceThreads = 512, kPartSegs = 128;

template <int XDT, int FMT>
__global__ void __launch_bounds__(kPieceThreads)
    act_pieces_kernel(const void* __restrict__ x, int64_t K, float* __restrict__ scale, uint4* __restrict__ pieces,
                      int* __restrict__ sums, int64_t chunks, int mb) {
  pdl_enter(x, scale, pieces, sums);
  constexpr int W = few_pieces(FMT), kPart = kPartSegs * 16 * W;  // codes of a part
  constexpr int kKeep = (kPart / 8 + kPieceThreads - 1) / kPieceThreads;
  __shared__ __align__(16) uint8_t codes[kPart];
  __shared__ __align__(16) float sum_mem[2][4][32];
  __shared__ int total;
  const int64_t m = blockIdx.x;
  const bool wide = K % 8 == 0;
  constexpr int RDT = XDT == BL_I8 ? BL_BF16 : XDT;  // (raw values are not used for given codes)
  Raw<RDT, 8> keep[kKeep];
  if (threadIdx.x == 0) total = 0;
  float s = 1.0f, c127 = 0.0f;
  if constexpr (XDT != BL_I8) {
    BlockSum sum(sum_mem);
    float amax = 0.0f;
    if (wide) {
      auto take = [&](const Raw<RDT, 8>& r) {
        float v[8];
        r.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      };
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int k = 8 * (i * kPieceThreads + static_cast<int>(threadIdx.x));
        keep[i].zero();
        if (k < kPart && k < K) keep[i].load(x, m * K + k);
      }
#pragma unroll
      for (int i = 0; i < kKeep; ++i) take(keep[i]);
      for (int64_t k = kPart + 8 * threadIdx.x; k < K; k += 8 * kPieceThreads) {
        Raw<RDT, 8> r;
        r.load(x, m * K + k);
        take(r);
      }
    } else {
#pragma unroll 8
      for (int64_t k = threadIdx.x; k < K; k += kPieceThreads) amax = fmaxf(amax, fabsf(load_elem<XDT>(x, m * K + k)));
    }
    s = fmaxf(sum.max(amax), 1e-6f);
    c127 = __fdiv_rn(127.0f, s);
    if (threadIdx.x == 0) scale[m] = s;
  }
  int part_sum = 0;
  const int64_t segs = 4 * chunks;
  for (int64_t g0 = 0; g0 < segs; g0 += kPartSegs) {
    const int64_t k0 = g0 * 16 * W;
    __syncthreads();  // the previous part's pieces have been formed (and `total` is 0)
    if (wide) {
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int at = 8 * (i * kPieceThreads + static_cast<int>(threadIdx.x));
        if (at >= kPart) continue;
        const int64_t k = k0 + at;
        uint2 o = make_uint2(0u, 0u);
        if (k < K) {
          if constexpr (XDT == BL_I8) {
            o = __ldcg(reinterpret_cast<const uint2*>(static_cast<const int8_t*>(x) + m * K + k));
          } else {
            if (g0 != 0) keep[i].load(x, m * K + k);
            float v[8];
            int q[8];
            keep[i].get(v);
            quant_act_fast_n<8>(v, s, c127, q);
            o = make_uint2(pack4(q), pack4(q + 4));
          }
        }
        part_sum = __dp4a(static_cast<int>(o.x), 0x01010101, part_sum);
        part_sum = __dp4a(static_cast<int>(o.y), 0x01010101, part_sum);
        *reinterpret_cast<uint2*>(codes + at) = o;
      }
    } else {
#pragma unroll 4
      for (int i = 0; i < kPart / kPieceThreads; ++i) {
        const int at = i * kPieceThreads + threadIdx.x;
        const int64_t k = k0 + at;
        int q = 0;
        if (k < K) {
          if constexpr (XDT == BL_I8)
            q = __ldcg(static_cast<const signed char*>(x) + m * K + k);
          else
            q = quant_act_fast(load_elem<XDT>(x, m * K + k), s, c127);
        }
        part_sum += q;
        codes[at] = static_cast<uint8_t>(q);
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < kPartSegs * W; e += kPieceThreads) {
      const int sg = e / W, i = e - sg * W;
      if (g0 + sg >= segs) break;
      uint4 o;
      if constexpr (FMT == BL_PACK_T5) {
        const uint8_t* c = codes + 80 * sg;
        uint32_t r4[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * i + j, word = r / 5, digit = r - 5 * word;
          const uint8_t* q = c + 20 * word + digit;
          r4[j] = q[0] | static_cast<uint32_t>(q[5]) << 8 | static_cast<uint32_t>(q[10]) << 16 |
                  static_cast<uint32_t>(q[15]) << 24;
        }
        o = make_uint4(r4[0], r4[1], r4[2], r4[3]);
      } else if constexpr (FMT == BL_PACK_I2) {
        const uint4 q = *reinterpret_cast<const uint4*>(codes + 64 * sg + 16 * i);
        o = i2_slot(q.x, q.y, q.z, q.w);
      } else {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(codes + 128 * sg + 32 * (i >> 1) + 4 * (i & 1));
        o = i2_slot(q[0], q[2], q[4], q[6]);
      }
      const int64_t at = g0 + sg;
      pieces[(((at >> 2) * W + i) * mb + m) * 4 + (at & 3)] = o;
    }
  }
  part_sum = __reduce_add_sync(0xffffffffu, part_sum);
  if ((threadIdx.x & 31) == 0) atomicAdd(&total, part_sum);
  __syncthreads();
  if (threadIdx.x == 0) sums[m] = total;
}

int few_groups(int64_t M) { return M <= 8 ? 1 : M <= 16 ? 2 : M <= 32 ? 4 : 8; }
int64_t few_chunks(int64_t rowbytes) { return (rowbytes / 16 + 3) / 4; }

template <int FMT, int NB>
cudaError_t launch_few(const uint8_t* packed, int64_t rb, const float* gamma, int64_t N, const uint4* pieces,
                       const int* sums, const float* scale, void* y, int ydt, int64_t M, const Epilogue& ep, cudaStream_t st) {
  const int64_t chunks = few_chunks(rb);
  int ns = 1;  // warps that share a chunk: while some would have none
  while (2 * ns <= NB && kFewWarps / ns > chunks) ns *= 2;
  return launch_pdl(gemm_few_kernel<FMT, NB>, static_cast<unsigned>((N + kFewRows - 1) / kFewRows), kFewThreads, 0, st,
                    packed, rb, gamma, N, pieces, sums, scale, y, ydt, static_cast<int>(M), ns, ep);
}

template <int FMT>
cudaError_t launch_few_fmt(const uint8_t* packed, int64_t rb, const float* gamma, int64_t N, int64_t K, const void* x,
                           int xdt, float* scale, int64_t M, void* y, int ydt, const Epilogue& ep, void* scratch,
                           cudaStream_t st) {
  const int mb = 8 * few_groups(M);
  uint4* pieces = static_cast<uint4*>(scratch);
  int* sums = reinterpret_cast<int*>(pieces + few_chunks(rb) * few_pieces(FMT) * mb * 4);
  auto kern = xdt == BL_F32 ? act_pieces_kernel<BL_F32, FMT>
                            : xdt == BL_BF16 ? act_pieces_kernel<BL_BF16, FMT> : act_pieces_kernel<BL_I8, FMT>;
  const cudaError_t e = launch_pdl(kern, static_cast<unsigned>(M), kPieceThreads, 0, st, x, K, scale, pieces, sums,
                                   few_chunks(rb), mb);
  if (e != cudaSuccess) return e;
  switch (mb / 8) {
    case 1: return launch_few<FMT, 1>(packed, rb, gamma, N, pieces, sums, scale, y, ydt, M, ep, st);
    case 2: return launch_few<FMT, 2>(packed, rb, gamma, N, pieces, sums, scale, y, ydt, M, ep, st);
    case 4: return launch_few<FMT, 4>(packed, rb, gamma, N, pieces, sums, scale, y, ydt, M, ep, st);
    default: return launch_few<FMT, 8>(packed, rb, gamma, N, pieces, sums, scale, y, ydt, M, ep, st);
  }
}

}  // namespace

size_t gemm_few_bytes(int64_t M, int64_t rowbytes, int fmt) {
  const size_t mb = 8 * static_cast<size_t>(few_groups(M));
  return static_cast<size_t>(few_chunks(rowbytes)) * few_pieces(fmt) * mb * 4 * sizeof(uint4) + mb * sizeof(int);
}

cudaError_t launch_gemm_few(const uint8_t* packed, int fmt, int64_t rowbytes, const float* gamma, int64_t N, int64_t K,
                            const void* x, int xdt, float* scale, int64_t M, void* y, int ydt, const Epilogue& ep,
                            void* scratch, cudaStream_t st) {
  const cudaError_t e =
      fmt == BL_PACK_I2
          ? launch_few_fmt<BL_PACK_I2>(packed, rowbytes, gamma, N, K, x, xdt, scale, M, y, ydt, ep, scratch, st)
      : fmt == BL_PACK_T5
          ? launch_few_fmt<BL_PACK_T5>(packed, rowbytes, gamma, N, K, x, xdt, scale, M, y, ydt, ep, scratch, st)
          : launch_few_fmt<BL_PACK_B1>(packed, rowbytes, gamma, N, K, x, xdt, scale, M, y, ydt, ep, scratch, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
