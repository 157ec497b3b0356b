// bl_gemm_grad.cu -- the two gradient products of many tokens on the
// 5th-generation tensor cores:
//
//   dx[m, k] = gamma sum_n dz[m, n] W_q[n, k]        dz bf16, codes exact in bf16
//   dW[n, k] = gamma sum_m dz[m, n] (s_m / 127) x_q[m, k]
//
// Both contract over the rows of a second operand stored [R, J] with the output
// column contiguous (W_q by rows n; x_q by rows m), so it is an MN-major operand
// of the MMA; the first operand is K-major for dx (a token's gradient is
// contiguous along n) and MN-major for dW.
//
// For dW the token's factor varies along the contraction and cannot move to
// the epilogue: v = fl(dz s_m) is scaled by a power of two per output row n
// (the row's largest |v| near 2^13) and split into two fp16 parts, hi = fp16(v)
// and lo = fp16(v - hi): 22 bits of v, against x_q exact in fp16.  Two bf16
// parts would keep 16 bits and cost the same.  The epilogue undoes the scale.
//
// A cluster of two CTAs computes a tile of 256 x 256 outputs with
// tcgen05.mma.cta_group::2 (each CTA stages 128 rows of A and 128 columns of B,
// 64 contracted elements a stage, by TMA), accumulating in tensor memory.  The
// tensor core's fp32 additions truncate, so runs are kept to 32 MMAs: eight
// epilogue warps add each finished run to fp32 registers (round to nearest)
// while the MMAs fill the other half of tensor memory.  (dW over 4096 tokens is
// 1.1e-6 off in the 2-norm with runs of 64.)  Few tiles (few tokens in dx) are spread over the SMs by cutting the
// contraction; the parts are added in order by a second kernel.
// Every wait is bounded: on expiry the kernel sets the workspace timeout flag,
// drains what it issued, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cstring>

#include "bl_common.cuh"
#include "bl_kernels.h"
#include "bl_sm100.cuh"
#include "bl_tensormap.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kTile = 128;   // rows of A, and columns of B, staged per CTA
constexpr int kBR = 64;      // contracted elements per stage: 128 bytes, four MMAs of 16
constexpr uint32_t kPlane = kTile * kBR * 2;  // 16384 bytes: one staged operand plane
constexpr int kGradThreads = 320;             // warp 0 TMA, 1 MMA, 2-9 epilogue
constexpr uint32_t kGradTmemCols = 512;       // two accumulators of 256 columns
constexpr long long kGradTimeout = 1ll << 32;  // ~2 s at 1.9 GHz

template <bool DW>
struct GradCfg {
  static constexpr int kPlanesA = DW ? 2 : 1;  // hi and lo of dW's first operand
  static constexpr uint32_t kStage = (kPlanesA + 1) * kPlane;
  static constexpr int kStages = DW ? 4 : 6;
  static constexpr int kRun = DW ? 4 : 8;  // stages (32 MMAs) added up in tensor memory before the registers take over
  static constexpr size_t kSmem = 1024 + kStages * kStage + 8 * (2 * kStages + 5) + 16;
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ void mma_f16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 128-byte-swizzled operand descriptors.  K-major: rows of 128 bytes (64
// contracted elements), 8-row groups 1024 bytes apart.  MN-major: chunks of 64
// outer elements (128 bytes) x 64 contracted rows, 8-row groups 1024 bytes apart
// (stride offset), chunks 8192 bytes apart (leading offset).
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr, bool mn_major) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3fffu);
  d |= static_cast<uint64_t>(mn_major ? (8192 >> 4) : 1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Instruction descriptor of kind::f16: fp32 accumulator; A and B both bf16 (1)
// or both fp16 (0); bit 15 / 16: A / B MN-major; shape 256 x 256.
__host__ __device__ constexpr uint32_t f16_idesc(bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(256 >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
}

// 16 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_load16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// D[i, j] = alpha(i) sum over R: a unit is a 256 x 256 tile over a range of
// stages.  I x J outputs with row stride J.  alpha = gamma for dx and (gamma /
// 127) 2^-e_i for dW (rowinv[i] = 2^-e_i).  With ks > 1 the unit writes its
// plain sums to part[kz][i][j].
template <bool DW>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    gemm_grad_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a2,
                     const __grid_constant__ CUtensorMap tm_b, const float* __restrict__ gamma,
                     const float* __restrict__ rowinv, void* __restrict__ out, int odt, int I, int J, int R, int ks,
                     float* __restrict__ part, WsHeader* __restrict__ hdr, long long limit) {
  pdl_enter(gamma, rowinv, out, part, hdr);
  using Cfg = GradCfg<DW>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;  // S x [A planes, B plane], each 16 KB, swizzled
  uint64_t* full = reinterpret_cast<uint64_t*>(stages + S * Cfg::kStage);  // leader: the loads of both CTAs
  uint64_t* empty = full + S;                                              // local: the MMAs have read the stage
  uint64_t* accf = empty + S;                                              // local: a run is in tensor memory (2)
  uint64_t* acce = accf + 2;                                               // leader: both CTAs have taken it (2)
  uint64_t* drain = acce + 2;                                              // leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int steps = (R + kBR - 1) / kBR;
  const int j_tiles = (J + 2 * kTile - 1) / (2 * kTile);
  const int i_tiles = (I + 2 * kTile - 1) / (2 * kTile);
  const int units = i_tiles * j_tiles * ks;  // ks <= steps (host): no unit is empty
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  struct Unit {
    int it, jt, kz, s0, s1;
  };
  auto unit_of = [&](int u) {
    Unit w;
    w.jt = u % j_tiles;
    const int r = u / j_tiles;
    w.kz = r % ks;
    w.it = r / ks;
    w.s0 = static_cast<int>(static_cast<int64_t>(w.kz) * steps / ks);
    w.s1 = static_cast<int>(static_cast<int64_t>(w.kz + 1) * steps / ks);
    return w;
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf + a, 1);
      mbar_init(acce + a, 16);  // eight epilogue warps of each CTA
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kGradTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_before();
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrive or copy
  tc_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&](uint32_t site) {
    set_flag(hdr, kFlagTimeout, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit w = unit_of(u);
        const int i0 = w.it * 2 * kTile + static_cast<int>(rank) * kTile;
        const int j0 = w.jt * 2 * kTile + static_cast<int>(rank) * kTile;
        for (int st = w.s0; st < w.s1; ++st, ++it) {
          const int s = it % S;
          if (!wait1(empty + s, ((it / S) & 1) ^ 1, limit, abort_flag)) {
            fail(0x221);
            ok = false;
            break;
          }
          if (leader) mbar_expect_tx(full + s, 2 * Cfg::kStage);
          const uint32_t bar = mapa_shared(smem_u32(full + s), 0);
          uint8_t* a = stages + s * Cfg::kStage;
          uint8_t* b = a + Cfg::kPlanesA * kPlane;
          const int r0 = st * kBR;
          if constexpr (DW) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // chunks of 64 output rows
              tma_load_2d_pair(a + c * 8192, &tm_a, bar, i0 + 64 * c, r0);
              tma_load_2d_pair(a + kPlane + c * 8192, &tm_a2, bar, i0 + 64 * c, r0);
            }
          } else {
            tma_load_2d_pair(a, &tm_a, bar, r0, i0);
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) tma_load_2d_pair(b + c * 8192, &tm_b, bar, j0 + 64 * c, r0);
        }
      }
      // this CTA's last copies have landed before it leaves, since the MMAs
      // that read them have completed (after a failure: one limit's time)
      for (int j = (it > S ? it - S : 0); j < it; ++j)
        if (!wait_drain(empty + (j % S), (j / S) & 1, limit)) break;
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (leader) -------------------------
    if (leader && lane == 0) {
      constexpr uint32_t idesc = f16_idesc(!DW, DW, true);
      int it = 0, run = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += pairs) {
        const Unit w = unit_of(u);
        for (int st = w.s0; st < w.s1 && ok; ++run) {
          const int a = run & 1;
          if (!wait1(acce + a, ((run >> 1) & 1) ^ 1, limit, abort_flag)) {
            fail(0x321);
            ok = false;
            break;
          }
          tc_after();
          const uint32_t d = tmem + static_cast<uint32_t>(a * 2 * kTile);
          const int end = st + Cfg::kRun < w.s1 ? st + Cfg::kRun : w.s1;
          for (int first = st; st < end; ++st, ++it) {
            const int s = it % S;
            if (!wait1(full + s, (it / S) & 1, limit, abort_flag)) {
              fail(0x322);
              ok = false;
              break;
            }
            tc_after();
            const uint32_t sa = smem_u32(stages + s * Cfg::kStage), sb = sa + Cfg::kPlanesA * kPlane;
#pragma unroll
            for (int pl = 0; pl < Cfg::kPlanesA; ++pl)
#pragma unroll
              for (int k = 0; k < kBR / 16; ++k) {
                // 16 contracted elements further: 32 bytes of a K-major row, 16 rows of an MN-major chunk
                const uint32_t ao = DW ? 2048 * k : 32 * k;
                mma_f16_pair(d, op_desc(sa + pl * kPlane + ao, DW), op_desc(sb + 2048 * k, true), idesc,
                             (st != first || pl != 0 || k != 0) ? 1u : 0u);
              }
            commit_pair(empty + s, 0x3);
          }
          if (ok) commit_pair(accf + a, 0x3);
        }
      }
      commit_pair(drain, 0x1);
      (void)wait_drain(drain, 0, limit);
    }
  } else {
    // ------------------------------ epilogue (both CTAs) ------------------------
    // warp: 32 output rows (its tensor-memory lane quarter) x 128 columns
    const int q = warp & 3, half = (warp - 2) >> 2;
    const float g = __ldcg(gamma);
    int run = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += pairs) {
      const Unit w = unit_of(u);
      float sum[kTile];
#pragma unroll
      for (int j = 0; j < kTile; ++j) sum[j] = 0.0f;
      for (int st = w.s0; st < w.s1; st += Cfg::kRun, ++run) {
        const int a = run & 1;
        if (!wait_warp(accf + a, (run >> 1) & 1, limit, abort_flag)) {
          if (lane == 0) fail(0x521);
          ok = false;
          break;
        }
        tc_after();
#pragma unroll
        for (int c = 0; c < kTile / 16; ++c) {
          uint32_t v[16];
          tmem_load16(tmem + (static_cast<uint32_t>(32 * q) << 16) +
                          static_cast<uint32_t>(a * 2 * kTile + half * kTile + 16 * c),
                      v);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[16 * c + j] += __uint_as_float(v[j]);
        }
        tc_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acce + a), 0));
      }
      if (!ok) break;
      const int i = w.it * 2 * kTile + static_cast<int>(rank) * kTile + 32 * q + lane;
      const int j0 = w.jt * 2 * kTile + half * kTile;
      if (i < I) {
        float alpha = 1.0f;
        void* dst = out;
        int dt = odt;
        int64_t o = static_cast<int64_t>(i) * J + j0;
        if (ks > 1) {
          dst = part;
          dt = BL_F32;
          o += static_cast<int64_t>(w.kz) * I * J;
        } else {
          alpha = DW ? __fmul_rn(__fdiv_rn(g, 127.0f), __ldcg(rowinv + i)) : g;
        }
#pragma unroll
        for (int j = 0; j < kTile; ++j) sum[j] = __fmul_rn(sum[j], alpha);
        if (J % 8 == 0) {
#pragma unroll
          for (int j = 0; j < kTile; j += 8)
            if (j0 + j < J) store_vec_dt<8>(dst, dt, o + j, sum + j);
        } else {
#pragma unroll
          for (int j = 0; j < kTile; ++j)
            if (j0 + j < J) store_vec_dt<1>(dst, dt, o + j, sum + j);
        }
      }
    }
  }

  __syncthreads();
  tc_before();
  cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kGradTmemCols) : "memory");
  }
}

// The parts of a cut contraction, added in order; then the factor and the
// rounding to the output's type (dx).
__global__ void __launch_bounds__(256)
    grad_parts_kernel(const float* __restrict__ part, int ks, int64_t n, const float* __restrict__ gamma,
                      void* __restrict__ out, int odt) {
  pdl_enter(part, gamma, out);
  const float g = __ldcg(gamma);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += stride) {
    float s = __ldcg(part + e);
    for (int z = 1; z < ks; ++z) s += __ldcg(part + z * n + e);
    s = __fmul_rn(s, g);
    store_vec_dt<1>(out, odt, e, &s);
  }
}

// 2-bit rows as bf16 {-1, 0, 1} rows of ld elements (ld = K rounded up to 64):
// one 16-byte packed segment (64 weights, padding decodes to 0) per thread.
__global__ void __launch_bounds__(256)
    i2_to_bf16_kernel(const uint8_t* __restrict__ i2, int64_t segs, uint16_t* __restrict__ w) {
  pdl_enter(i2, w);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; s < segs; s += stride) {
    const uint4 v = __ldcg(reinterpret_cast<const uint4*>(i2) + s);
    const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
    uint4* dst = reinterpret_cast<uint4*>(w) + 8 * s;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t d = (wd[i >> 1] >> (16 * (i & 1) + 4 * j)) & 0xfu;  // two digits
        const uint32_t a = d & 3u, c = d >> 2;
        // digit 0 -> 0xBF80 (-1), 1 -> 0, 2 -> 0x3F80 (+1)
        const uint32_t ha = a == 1u ? 0u : (a == 0u ? 0xbf80u : 0x3f80u);
        const uint32_t hc = c == 1u ? 0u : (c == 0u ? 0xbf80u : 0x3f80u);
        o[j] = ha | (hc << 16);
      }
      dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// dz rows copied to a row stride of ld elements (a multiple of 8), for TMA.
__global__ void __launch_bounds__(256)
    pad_rows_kernel(const uint16_t* __restrict__ src, int64_t M, int64_t N, int64_t ld, uint16_t* __restrict__ dst) {
  pdl_enter(src, dst);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x, n = M * ld;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < n; e += stride) {
    const int64_t m = e / ld, c = e - m * ld;
    dst[e] = c < N ? __ldcg(src + m * N + c) : static_cast<uint16_t>(0);
  }
}

// The largest |dz s_m| of each output row n over a range of tokens, as bits
// (finite magnitudes order like unsigned integers): part[range][n].
__global__ void __launch_bounds__(256)
    grad_rowmax_kernel(const uint16_t* __restrict__ dz, const float* __restrict__ scale, int64_t M, int64_t N,
                       int64_t rows_per, uint32_t* __restrict__ part) {
  pdl_enter(dz, scale, part);
  const int64_t n = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (n >= N) return;
  const int64_t m0 = blockIdx.y * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  float mx = 0.0f;
#pragma unroll 8
  for (int64_t m = m0; m < m1; ++m)
    mx = fmaxf(mx, fabsf(__fmul_rn(bf16_bits_to_f32(__ldcg(dz + m * N + n)), __ldcg(scale + m))));
  part[blockIdx.y * N + n] = __float_as_uint(mx);
}

// 2^e with the largest |v| 2^e of the row in [2^13, 2^14) (|e| <= 126; a row of
// zeros keeps 1), and its inverse.
__global__ void __launch_bounds__(256)
    grad_rowscale_kernel(const uint32_t* __restrict__ part, int64_t ranges, int64_t N, float* __restrict__ rowscale,
                         float* __restrict__ rowinv) {
  pdl_enter(part, rowscale, rowinv);
  const int64_t n = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (n >= N) return;
  uint32_t mx = 0;
  for (int64_t r = 0; r < ranges; ++r) mx = max(mx, __ldcg(part + r * N + n));
  const int ex = static_cast<int>(mx >> 23);  // biased exponent (0: below 2^-126)
  int e = mx == 0 ? 0 : 13 - (ex - 127);
  e = e > 126 ? 126 : (e < -126 ? -126 : e);
  rowscale[n] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  rowinv[n] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
}

// hi and lo fp16 parts of v = fl(dz s_m) 2^e, rows of ld elements (zeros past N).
__global__ void __launch_bounds__(256)
    grad_split_kernel(const uint16_t* __restrict__ dz, const float* __restrict__ scale,
                      const float* __restrict__ rowscale, int64_t M, int64_t N, int64_t ld, __half* __restrict__ hi,
                      __half* __restrict__ lo) {
  pdl_enter(dz, scale, rowscale, hi, lo);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x, total = M * ld;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += stride) {
    const int64_t m = e / ld, n = e - m * ld;
    float v = 0.0f;
    if (n < N)
      v = __fmul_rn(__fmul_rn(bf16_bits_to_f32(__ldcg(dz + m * N + n)), __ldcg(scale + m)), __ldcg(rowscale + n));
    const __half h = __float2half_rn(v);
    hi[e] = h;
    lo[e] = __float2half_rn(__fsub_rn(v, __half2float(h)));
  }
}

// x_q as fp16 rows of ld elements (zeros past K).
__global__ void __launch_bounds__(256)
    i8_to_f16_kernel(const int8_t* __restrict__ xq, int64_t M, int64_t K, int64_t ld, __half* __restrict__ x) {
  pdl_enter(xq, x);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x, total = M * ld;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < total; e += stride) {
    const int64_t m = e / ld, k = e - m * ld;
    x[e] = __int2half_rn(k < K ? static_cast<int>(__ldcg(reinterpret_cast<const signed char*>(xq) + m * K + k)) : 0);
  }
}

unsigned flat_grid(int64_t items) {
  const int64_t cap = static_cast<int64_t>(device_sms()) * 8, g = (items + 255) / 256;
  return static_cast<unsigned>(g < 1 ? 1 : (g < cap ? g : cap));
}

template <bool DW>
cudaError_t launch_product(const void* a, const void* a2, int64_t lda, const void* b, int64_t ldb, const float* gamma,
                           const float* rowinv, void* out, int odt, int64_t I, int64_t J, int64_t R, int ks,
                           float* part, void* ws, cudaStream_t st) {
  CUtensorMap ta, ta2, tb;
  // A: [I, R] K-major (dx) or [R, I] (dW); B: [R, J]
  const bool ok =
      DW ? encode_2d_b16(&ta, a, static_cast<uint64_t>(I), static_cast<uint64_t>(R), static_cast<uint64_t>(lda) * 2, 64,
                         kBR) &&
               encode_2d_b16(&ta2, a2, static_cast<uint64_t>(I), static_cast<uint64_t>(R),
                             static_cast<uint64_t>(lda) * 2, 64, kBR)
         : encode_2d_b16(&ta, a, static_cast<uint64_t>(R), static_cast<uint64_t>(I), static_cast<uint64_t>(lda) * 2,
                         kBR, kTile);
  if (!ok || !encode_2d_b16(&tb, b, static_cast<uint64_t>(J), static_cast<uint64_t>(R), static_cast<uint64_t>(ldb) * 2,
                            64, kBR))
    return cudaErrorInvalidValue;
  if (!DW) memset(&ta2, 0, sizeof ta2);
  auto kern = gemm_grad_kernel<DW>;
  const size_t smem = GradCfg<DW>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t units = ((I + 2 * kTile - 1) / (2 * kTile)) * ((J + 2 * kTile - 1) / (2 * kTile)) * ks;
  const int64_t most = device_sms() / 2, pairs = units < most ? units : most;
  return launch_pdl(kern, static_cast<unsigned>(2 * pairs), kGradThreads, smem, st, ta, ta2, tb, gamma, rowinv, out,
                    odt, static_cast<int>(I), static_cast<int>(J), static_cast<int>(R), ks, part,
                    static_cast<WsHeader*>(ws), kGradTimeout);
}

}  // namespace

int64_t grad_ld(int64_t n) { return (n + 63) / 64 * 64; }

// Parts of dx's contraction: the number in 1..16 with the least work on the
// busiest pair of SMs, in stages, plus 4 per unit (filling the ring, the
// epilogue) and 12 for the pass over the parts.
int grad_dx_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((M + 2 * kTile - 1) / (2 * kTile)) * ((K + 2 * kTile - 1) / (2 * kTile));
  const int64_t steps = (N + kBR - 1) / kBR, pairs = device_sms() / 2 > 0 ? device_sms() / 2 : 1;
  int best = 1;
  int64_t best_cost = -1;
  for (int ks = 1; ks <= 16 && ks <= steps; ++ks) {
    const int64_t cost = (tiles * ks + pairs - 1) / pairs * ((steps + ks - 1) / ks + 4) + (ks > 1 ? 12 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = ks;
    }
  }
  return best;
}

int64_t grad_rowmax_ranges(int64_t M) {
  const int64_t r = (M + 127) / 128;
  const int64_t per = (M + 63) / 64;  // at most 64 ranges
  return r <= 64 ? (r < 1 ? 1 : r) : (M + per - 1) / per;
}

cudaError_t launch_i2_to_bf16(const uint8_t* i2, int64_t N, int64_t rowbytes, uint16_t* w, cudaStream_t st) {
  const int64_t segs = N * (rowbytes / 16);
  return launch_pdl(i2_to_bf16_kernel, flat_grid(segs), 256, 0, st, i2, segs, w);
}

cudaError_t launch_pad_rows(const uint16_t* src, int64_t M, int64_t N, int64_t ld, uint16_t* dst, cudaStream_t st) {
  return launch_pdl(pad_rows_kernel, flat_grid(M * ld), 256, 0, st, src, M, N, ld, dst);
}

cudaError_t launch_grad_dx(const uint16_t* dz, int64_t lddz, const uint16_t* w, int64_t ldw, const float* gamma,
                           int64_t M, int64_t N, int64_t K, void* dx, int dxdt, float* part, void* ws,
                           cudaStream_t st) {
  const int ks = grad_dx_parts(M, N, K);
  cudaError_t e = launch_product<false>(dz, nullptr, lddz, w, ldw, gamma, nullptr, dx, dxdt, M, K, N, ks, part, ws, st);
  if (e != cudaSuccess) return e;
  if (ks > 1)
    e = launch_pdl(grad_parts_kernel, flat_grid(M * K), 256, 0, st, static_cast<const float*>(part), ks, M * K, gamma,
                   dx, dxdt);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_grad_dw(const uint16_t* dz, const int8_t* xq, const float* scale, const float* gamma, int64_t M,
                           int64_t N, int64_t K, float* dw, const GradDwScratch& s, void* ws, cudaStream_t st) {
  const int64_t ranges = grad_rowmax_ranges(M), rows_per = (M + ranges - 1) / ranges;
  const int64_t ldn = grad_ld(N), ldk = grad_ld(K);
  const unsigned nb = static_cast<unsigned>((N + 255) / 256);
  cudaError_t e = launch_pdl(grad_rowmax_kernel, dim3(nb, static_cast<unsigned>(ranges)), 256, 0, st, dz, scale, M, N,
                             rows_per, s.maxes);
  if (e == cudaSuccess)
    e = launch_pdl(grad_rowscale_kernel, nb, 256, 0, st, static_cast<const uint32_t*>(s.maxes), ranges, N, s.rowscale,
                   s.rowinv);
  if (e == cudaSuccess)
    e = launch_pdl(grad_split_kernel, flat_grid(M * ldn), 256, 0, st, dz, scale, static_cast<const float*>(s.rowscale),
                   M, N, ldn, static_cast<__half*>(s.hi), static_cast<__half*>(s.lo));
  if (e == cudaSuccess)
    e = launch_pdl(i8_to_f16_kernel, flat_grid(M * ldk), 256, 0, st, xq, M, K, ldk, static_cast<__half*>(s.x));
  if (e == cudaSuccess)
    e = launch_product<true>(s.hi, s.lo, ldn, s.x, ldk, gamma, s.rowinv, dw, BL_F32, N, K, M, 1, nullptr, ws, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
