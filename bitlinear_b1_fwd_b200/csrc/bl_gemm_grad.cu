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
// and lo = fp16(v - hi): 22 bits of v, or 2^-25 (the subnormals' half step, 2^-38 of
// the row's largest) where that is more, against x_q exact in fp16.  Two bf16
// parts would keep 16 bits and cost the same.  The epilogue undoes the scale.
//
// A cluster of two CTAs computes a tile of 256 x 256 outputs with
// tcgen05.mma.cta_group::2 (each CTA stages 128 rows of A and 128 columns of B,
// 64 contracted elements a stage, by TMA), accumulating in tensor memory.  The
// tensor core's fp32 additions truncate, so runs are kept to 32 MMAs: eight
// epilogue warps add each finished run to fp32 registers (round to nearest)
// while the MMAs fill the other half of tensor memory.  (dW over 4096 tokens is
// 1.1e-6 off in the 2-norm with runs of 64.)  Few tiles (few tokens in dx) are
// spread over the SMs by cutting the contraction; the parts are added in order by
// a second kernel.  4096 x 3200 x 8640: dx 166 us (1360 TFLOP/s), dW 288 us (two
// parts: 1570 TFLOP/s), the conversions before them 20, 30 and 45 us.
// Every wait is bounded: on expiry the kernel sets the workspace timeout flag,
// drains what it issued, frees its tensor memory and returns.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cstring>
#include <type_traits>

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
constexpr int kGradEpiWarps = 8;
constexpr uint32_t kOutBox = 32 * 128;        // output staging of a warp: 32 rows of 128 bytes
constexpr uint32_t kGradTmemCols = 512;       // two accumulators of 256 columns
constexpr long long kGradTimeout = 1ll << 32;  // ~2 s at 1.9 GHz

// SHORT: units of few stages, where the output counts: two output boxes per warp
// and a stage less in the ring (16 stages: 1024 tokens, 3200 x 3200, both products
// 84 us against 92; 64 stages: 4096 x 3200 x 8640, 534 against 522).
constexpr int kShortSteps = 24;
template <bool DW, bool SHORT>
struct GradCfg {
  static constexpr int kPlanesA = DW ? 2 : 1;  // hi and lo of dW's first operand
  static constexpr uint32_t kStage = (kPlanesA + 1) * kPlane;
  static constexpr int kStages = (DW ? 4 : 6) - (SHORT ? 1 : 0);
  static constexpr int kBoxes = SHORT ? 2 : 1;
  static constexpr int kRun = DW ? 4 : 8;  // stages (32 MMAs) added up in tensor memory before the registers take over
  static constexpr size_t kSmem = 1024 + kStages * kStage + kBoxes * kGradEpiWarps * kOutBox + 8 * (2 * kStages + 5) + 16;
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

// D[i, j] = alpha(i) sum over R: a unit is a 256 x 256 tile over a range of
// stages.  I x J outputs with row stride J.  alpha = gamma for dx and (gamma /
// 127) 2^-e_i for dW (rowinv[i] = 2^-e_i).  With ks > 1 the unit writes its
// plain sums to part[kz][i][j].
// F32: the type of the outputs (or parts); O_TMA: they have a tensor map.
template <bool DW, bool SHORT, bool O_TMA, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGradThreads, 1)
    gemm_grad_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_a2,
                     const __grid_constant__ CUtensorMap tm_b, const __grid_constant__ CUtensorMap tm_o,
                     const float* __restrict__ gamma, const float* __restrict__ rowinv, void* __restrict__ out, int I, int J, int R, int ks,
                     float* __restrict__ part, WsHeader* __restrict__ hdr, long long limit, int skip_producer) {
  pdl_enter(gamma, rowinv, out, part, hdr);
  using Cfg = GradCfg<DW, SHORT>;
  constexpr int S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;  // S x [A planes, B plane], each 16 KB, swizzled
  uint8_t* outs = stages + S * Cfg::kStage;  // the output boxes of each epilogue warp, swizzled
  uint64_t* full = reinterpret_cast<uint64_t*>(outs + Cfg::kBoxes * kGradEpiWarps * kOutBox);  // leader: the loads of both CTAs
  uint64_t* empty = full + S;                                              // local: the MMAs have read the stage
  uint64_t* accf = empty + S;                                              // local: a run is in tensor memory (2)
  uint64_t* acce = accf + 2;                                               // leader: both CTAs have taken it (2)
  uint64_t* drain = acce + 2;                                              // leader
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int steps = (R - 1) / kBR + 1;  // I and R reach 2^31 - 1: nothing is added to them
  const int j_tiles = (J - 1) / (2 * kTile) + 1;
  const int i_tiles = (I - 1) / (2 * kTile) + 1;
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
    set_flag(hdr, kFlagTimeout | kFlagProductGrad, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------
    if (lane == 0 && !skip_producer) {
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
    const float g = DW ? __fdiv_rn(__ldcg(gamma), 127.0f) : __ldcg(gamma);
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
      const int i0 = w.it * 2 * kTile + static_cast<int>(rank) * kTile + 32 * q, i = i0 + lane;
      const int j0 = w.jt * 2 * kTile + half * kTile;
      float alpha = ks > 1 ? 1.0f : g, inv = 1.0f;
      if constexpr (DW) {
        inv = i < I ? __ldcg(rowinv + i) : 0.0f;
        // a power of two: one factor for both, unless that has no 24 bits (a row of gradients below some 2^-100)
        if (const float both = __fmul_rn(g, inv); fabsf(both) >= 1.17549435e-38f) {
          alpha = both;
          inv = 1.0f;
        }
      }
      auto scaled = [&](float v) { return DW ? __fmul_rn(__fmul_rn(v, alpha), inv) : __fmul_rn(v, alpha); };
      // 32 rows x 128 bytes at a time through this warp's boxes; the TMA unit clips
      // rows past I and columns past J.  (Two boxes of 64-byte rows: 130 tokens,
      // 3200 x 3200, 53 us for both products against 45.)  Rows of the output that
      // are no multiple of 16 bytes have no tensor map: the warp copies the box
      // itself, neighbouring lanes neighbouring columns.
      uint8_t* box = outs + Cfg::kBoxes * (warp - 2) * kOutBox;
      int ln = lane;  // opaque: the pieces' addresses are formed here, not kept in registers through the runs
      asm volatile("" : "+r"(ln));
      auto next_box = [&](int c) {
        box = outs + (Cfg::kBoxes * (warp - 2) + c % Cfg::kBoxes) * kOutBox;
        if (O_TMA && lane == 0) bulk_wait_read<Cfg::kBoxes - 1>();  // the last store issued from it has read it
        __syncwarp();
      };
      auto put = [&](int c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
        *reinterpret_cast<uint4*>(box + ln * 128 + ((c ^ (ln & 7)) << 4)) = make_uint4(a0, a1, a2, a3);
      };
      auto store = [&](int j) {
        if constexpr (O_TMA) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && i0 < I && j0 + j < J) tma_store_3d(&tm_o, box, j0 + j, i0, ks > 1 ? w.kz : 0);
          if (lane == 0) bulk_commit();
        } else {
          using Elem = typename std::conditional<F32, uint32_t, uint16_t>::type;
          constexpr int NC = 128 / static_cast<int>(sizeof(Elem));
          Elem* dst = static_cast<Elem*>(ks > 1 ? part : out) + (ks > 1 ? static_cast<int64_t>(w.kz) * I * J : 0);
          __syncwarp();
#pragma unroll
          for (int col = ln; col < NC; col += 32) {
            const int at = col * static_cast<int>(sizeof(Elem));
            if (j0 + j + col < J) {
#pragma unroll 4
              for (int r = 0; r < 32 && i0 + r < I; ++r)
                dst[static_cast<int64_t>(i0 + r) * J + j0 + j + col] =
                    *reinterpret_cast<const Elem*>(box + r * 128 + ((((at >> 4) ^ (r & 7)) << 4) | (at & 15)));
            }
          }
        }
      };
      if constexpr (F32) {
#pragma unroll
        for (int j = 0; j < kTile; j += 32) {
          next_box(j / 32);
#pragma unroll
          for (int c = 0; c < 8; ++c)
            put(c, __float_as_uint(scaled(sum[j + 4 * c])), __float_as_uint(scaled(sum[j + 4 * c + 1])),
                __float_as_uint(scaled(sum[j + 4 * c + 2])), __float_as_uint(scaled(sum[j + 4 * c + 3])));
          store(j);
        }
      } else {
#pragma unroll
        for (int j = 0; j < kTile; j += 64) {
          next_box(j / 64);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float* v = sum + j + 8 * c;
            auto two = [&](int k) { return bf16_pair(scaled(v[k]), scaled(v[k + 1])); };
            put(c, two(0), two(2), two(4), two(6));
          }
          store(j);
        }
      }
    }
    if (O_TMA && lane == 0) bulk_wait<0>();  // every output has landed before the CTA leaves
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
// rounding to the output's type (dx).  V outputs per thread (n a multiple of V).
template <int V>
__global__ void __launch_bounds__(256)
    grad_parts_kernel(const float* __restrict__ part, int ks, int64_t n, const float* __restrict__ gamma,
                      void* __restrict__ out, int odt) {
  pdl_enter(part, gamma, out);
  const float g = __ldcg(gamma);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x * V;
  for (int64_t e = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * V; e < n; e += stride) {
    float s[V], t[V];
    load_vec<BL_F32, V>(part, e, s);
#pragma unroll 4
    for (int z = 1; z < ks; ++z) {
      load_vec<BL_F32, V>(part, z * n + e, t);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += t[j];
    }
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = __fmul_rn(s[j], g);
    store_vec_dt<V>(out, odt, e, s);
  }
}

// 2-bit rows as bf16 {-1, 0, 1} rows of ld elements (ld = K rounded up to 64,
// the weights of a 16-byte packed segment; padding decodes to 0): one packed
// word (16 weights, 32 output bytes) per thread.  Digit d becomes the bytes
// (lo, hi) = (80 BF), (00 00), (80 3F), picked by a byte permute whose selector
// is d, 4 + d for each of two digits.
__global__ void __launch_bounds__(256)
    i2_to_bf16_kernel(const uint32_t* __restrict__ i2, int64_t words, uint16_t* __restrict__ w) {
  pdl_enter(i2, w);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  int64_t s = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  auto expand = [&](uint32_t v, int64_t at) {
    uint4* dst = reinterpret_cast<uint4*>(w) + 2 * at;
    const uint32_t even = v & 0x33333333u, odd = (v >> 2) & 0x33333333u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = (even >> (16 * i + 4 * j)) & 0x3u, c = (odd >> (16 * i + 4 * j)) & 0x3u;
        o[j] = __byte_perm(0x00800080u, 0x003f00bfu, a * 0x11u + c * 0x1100u + 0x4040u);
      }
      dst[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  };
  for (; s + 3 * stride < words; s += 4 * stride) {
    uint32_t v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = __ldcg(i2 + s + u * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u) expand(v[u], s + u * stride);
  }
  for (; s < words; s += stride) expand(__ldcg(i2 + s), s);
}

// dz rows copied to a row stride of ld elements (a multiple of 8, zeros past
// N), for TMA: eight elements per thread.
__global__ void __launch_bounds__(256)
    pad_rows_kernel(const uint16_t* __restrict__ src, int64_t M, int64_t N, int64_t ld, uint16_t* __restrict__ dst) {
  pdl_enter(src, dst);
  const int64_t per_row = ld / 8, items = M * per_row;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; e < items; e += stride) {
    const int64_t m = e / per_row, c = 8 * (e - m * per_row);
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < N ? __ldcg(src + m * N + c + j) : 0u;
    reinterpret_cast<uint4*>(dst)[e] = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
}

// ---- dW's operands ------------------------------------------------------------------
// Two passes over dz.  Blocks of 32 column threads (8 neighbouring columns each) x
// 8 row threads over a range of rows; the first launch also carries the conversion
// of x_q, the other operand, in blocks of its own.  4096 x 3200 x 8640: 110 MB in 30
// us and 214 MB in 45 us, 0.6 and 0.7 of the copy rate, waiting for their loads (20
// cycles of it for each instruction issued; the issue slots are 31 % busy).
constexpr int kGcCols = 256, kGcRows = 8, kGcUnroll = 4;

// dz[m, n0 .. n0 + 7] (zeros past N)
__device__ __forceinline__ void load_dz8(const uint16_t* dz, int64_t m, int64_t n0, int64_t N, bool wide, float* v) {
  if (wide) {
    if (n0 < N) {
      load_vec<BL_BF16, 8>(dz, m * N + n0, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = n0 + j < N ? bf16_bits_to_f32(__ldcg(dz + m * N + n0 + j)) : 0.0f;
  }
}

// 4 int8 -> 4 fp16: 0x6400 | (q + 128) is the fp16 1152 + q
__device__ __forceinline__ uint2 i8x4_to_f16(uint32_t q) {
  q ^= 0x80808080u;
  const uint32_t a = __byte_perm(q, 0x64646464u, 0x4140), b = __byte_perm(q, 0x64646464u, 0x4342);
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  const __half2 ha = __hsub2(*reinterpret_cast<const __half2*>(&a), bias);
  const __half2 hb = __hsub2(*reinterpret_cast<const __half2*>(&b), bias);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&ha), *reinterpret_cast<const uint32_t*>(&hb));
}

// Blocks below max_blocks: the largest |dz s_m| of each column n over a range of
// rows, as bits (finite magnitudes order like unsigned integers), to
// part[range][n].  The others: x_q as fp16 rows of ldk elements (zeros past K).
__global__ void __launch_bounds__(256)
    grad_max_kernel(const uint16_t* __restrict__ dz, const float* __restrict__ scale, int64_t M, int64_t N,
                    int64_t rows_per, uint32_t* __restrict__ part, const int8_t* __restrict__ xq, int64_t K,
                    int64_t ldk, __half* __restrict__ x, int col_blocks, int max_blocks) {
  pdl_enter(dz, scale, part, xq, x);
  if (static_cast<int>(blockIdx.x) >= max_blocks) {
    const int64_t stride = static_cast<int64_t>(gridDim.x - max_blocks) * blockDim.x;
    int64_t e = static_cast<int64_t>(blockIdx.x - max_blocks) * blockDim.x + threadIdx.x;
    uint4* dst = reinterpret_cast<uint4*>(x);
    if (K % 16 == 0) {  // 16 elements per item
      const int64_t per_row = K / 16, items = M * per_row;
#pragma unroll 2
      for (; e < items; e += stride) {
        const uint4 q = __ldcg(reinterpret_cast<const uint4*>(xq) + e);
        const uint2 a = i8x4_to_f16(q.x), b = i8x4_to_f16(q.y), c = i8x4_to_f16(q.z), d = i8x4_to_f16(q.w);
        const int64_t m = e / per_row, o = (m * ldk + 16 * (e - m * per_row)) / 8;
        dst[o] = make_uint4(a.x, a.y, b.x, b.y);
        dst[o + 1] = make_uint4(c.x, c.y, d.x, d.y);
      }
    } else {  // 8 elements per item
      const int64_t per_row = ldk / 8, items = M * per_row;
      for (; e < items; e += stride) {
        const int64_t m = e / per_row, k = 8 * (e - m * per_row);
        uint32_t q[2] = {0u, 0u};
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (k + j < K)
            q[j >> 2] |= static_cast<uint32_t>(__ldcg(reinterpret_cast<const uint8_t*>(xq) + m * K + k + j))
                         << (8 * (j & 3));
        const uint2 a = i8x4_to_f16(q[0]), b = i8x4_to_f16(q[1]);
        dst[e] = make_uint4(a.x, a.y, b.x, b.y);
      }
    }
    return;
  }
  __shared__ uint32_t mx[kGcRows][kGcCols];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t cb = blockIdx.x % col_blocks, range = blockIdx.x / col_blocks;
  const int64_t n0 = cb * kGcCols + 8 * tx;
  const int64_t m0 = range * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  const bool wide = N % 8 == 0;
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
  if (n0 < N) {
#pragma unroll kGcUnroll
    for (int64_t m = m0 + ty; m < m1; m += kGcRows) {
      float d[8];
      load_dz8(dz, m, n0, N, wide, d);
      const float s = __ldcg(scale + m);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = fmaxf(v[j], fabsf(__fmul_rn(d[j], s)));
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) mx[ty][8 * tx + j] = __float_as_uint(v[j]);
  __syncthreads();
  const int64_t n = cb * kGcCols + threadIdx.x;
  if (n < N) {
    uint32_t a = 0;
#pragma unroll
    for (int r = 0; r < kGcRows; ++r) a = max(a, mx[r][threadIdx.x]);
    part[range * N + n] = a;
  }
}

// The two fp16 parts of v = fl(dz s_m) 2^e, rows of ld elements (zeros past N).
// 2^e brings the column's largest |v| into [2^13, 2^14) (|e| <= 126; a column of
// zeros keeps 1); its inverse goes to rowinv for the product's epilogue.
__global__ void __launch_bounds__(256)
    grad_split_kernel(const uint16_t* __restrict__ dz, const float* __restrict__ scale,
                      const uint32_t* __restrict__ part, int ranges, int64_t M, int64_t N, int64_t rows_per,
                      int64_t ld, float* __restrict__ rowinv, __half* __restrict__ hi, __half* __restrict__ lo) {
  pdl_enter(dz, scale, part, rowinv, hi, lo);
  __shared__ float factor[kGcCols];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  {
    const int64_t n = static_cast<int64_t>(blockIdx.x) * kGcCols + threadIdx.x;
    uint32_t mx = 0;
    if (n < N) {
#pragma unroll 16
      for (int r = 0; r < ranges; ++r) mx = max(mx, __ldcg(part + r * N + n));
    }
    const int ex = static_cast<int>(mx >> 23);  // biased exponent (0: below 2^-126)
    int e = mx == 0 ? 0 : 13 - (ex - 127);
    e = e > 126 ? 126 : (e < -126 ? -126 : e);
    factor[threadIdx.x] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    if (blockIdx.y == 0 && n < N) rowinv[n] = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  }
  __syncthreads();
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kGcCols + 8 * tx;
  if (n0 >= ld) return;
  const int64_t m0 = blockIdx.y * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  const bool wide = N % 8 == 0;
  float f[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = factor[8 * tx + j];
#pragma unroll kGcUnroll
  for (int64_t m = m0 + ty; m < m1; m += kGcRows) {
    float d[8];
    load_dz8(dz, m, n0, N, wide, d);
    const float s = __ldcg(scale + m);
    uint32_t h[4], l[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = __fmul_rn(__fmul_rn(d[2 * j], s), f[2 * j]), b = __fmul_rn(__fmul_rn(d[2 * j + 1], s), f[2 * j + 1]);
      const __half2 hh = __floats2half2_rn(a, b);
      const float2 back = __half22float2(hh);
      const __half2 ll = __floats2half2_rn(__fsub_rn(a, back.x), __fsub_rn(b, back.y));
      h[j] = *reinterpret_cast<const uint32_t*>(&hh);
      l[j] = *reinterpret_cast<const uint32_t*>(&ll);
    }
    const int64_t o = (m * ld + n0) / 8;
    reinterpret_cast<uint4*>(hi)[o] = make_uint4(h[0], h[1], h[2], h[3]);
    reinterpret_cast<uint4*>(lo)[o] = make_uint4(l[0], l[1], l[2], l[3]);
  }
}

unsigned flat_grid(int64_t items) {
  const int64_t cap = static_cast<int64_t>(device_sms()) * 8, g = (items + 255) / 256;
  return static_cast<unsigned>(g < 1 ? 1 : (g < cap ? g : cap));
}

template <bool DW>
cudaError_t launch_product(const void* a, const void* a2, int64_t lda, const void* b, int64_t ldb, const float* gamma,
                           const float* rowinv, void* out, int odt, int64_t I, int64_t J, int64_t R, int ks,
                           float* part, void* ws, cudaStream_t st, long long limit = kGradTimeout,
                           int skip_producer = 0) {
  CUtensorMap ta, ta2, tb, to;
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
  const bool o_tma = encode_out(&to, ks > 1 ? part : out, ks > 1 || odt == BL_F32, static_cast<uint64_t>(J),
                                  static_cast<uint64_t>(I), static_cast<uint64_t>(ks), 128);
  if (!o_tma) memset(&to, 0, sizeof to);
  const bool brief = (R + kBR - 1) / kBR <= kShortSteps * ks;
  const bool f32 = DW || ks > 1 || odt == BL_F32;
  auto pick = [&](auto s, auto t) {
    if constexpr (DW)
      return gemm_grad_kernel<DW, s.value, t.value, true>;
    else
      return f32 ? gemm_grad_kernel<DW, s.value, t.value, true> : gemm_grad_kernel<DW, s.value, t.value, false>;
  };
  const std::true_type yes;
  const std::false_type no;
  auto kern = o_tma ? (brief ? pick(yes, yes) : pick(no, yes)) : (brief ? pick(yes, no) : pick(no, no));
  const size_t smem = brief ? GradCfg<DW, true>::kSmem : GradCfg<DW, false>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  const int64_t units = ((I + 2 * kTile - 1) / (2 * kTile)) * ((J + 2 * kTile - 1) / (2 * kTile)) * ks;
  const int64_t most = device_sms() / 2, pairs = units < most ? units : most;
  return launch_pdl(kern, static_cast<unsigned>(2 * pairs), kGradThreads, smem, st, ta, ta2, tb, to, gamma, rowinv, out,
                    static_cast<int>(I), static_cast<int>(J), static_cast<int>(R), ks, part,
                    static_cast<WsHeader*>(ws), limit, skip_producer);
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

// Row ranges of the passes over dz: one wave of four blocks per SM, each range of
// at least 8 rows.
int64_t grad_rowmax_ranges(int64_t M, int64_t N) {
  const int64_t cols = (N + kGcCols - 1) / kGcCols, want = 4 * static_cast<int64_t>(device_sms()) / cols;
  const int64_t most = (M + kGcRows - 1) / kGcRows;
  int64_t r = want < 1 ? 1 : (want > 32 ? 32 : want);
  if (r > most) r = most < 1 ? 1 : most;
  const int64_t per = (M + r - 1) / r;
  return per > 0 ? (M + per - 1) / per : 1;
}

cudaError_t launch_i2_to_bf16(const uint8_t* i2, int64_t N, int64_t rowbytes, uint16_t* w, cudaStream_t st) {
  const int64_t words = N * (rowbytes / 4);
  return launch_pdl(i2_to_bf16_kernel, flat_grid(words), 256, 0, st, reinterpret_cast<const uint32_t*>(i2), words, w);
}

cudaError_t launch_pad_rows(const uint16_t* src, int64_t M, int64_t N, int64_t ld, uint16_t* dst, cudaStream_t st) {
  return launch_pdl(pad_rows_kernel, flat_grid(M * ld / 8), 256, 0, st, src, M, N, ld, dst);
}

cudaError_t launch_grad_parts(const float* part, int ks, int64_t n, const float* gamma, void* out, int odt,
                              cudaStream_t st) {
  return n % 8 == 0 ? launch_pdl(grad_parts_kernel<8>, flat_grid(n / 8), 256, 0, st, part, ks, n, gamma, out, odt)
                    : launch_pdl(grad_parts_kernel<1>, flat_grid(n), 256, 0, st, part, ks, n, gamma, out, odt);
}

cudaError_t launch_grad_dx(const uint16_t* dz, int64_t lddz, const uint16_t* w, int64_t ldw, const float* gamma,
                           int64_t M, int64_t N, int64_t K, void* dx, int dxdt, float* part, void* ws,
                           cudaStream_t st) {
  const int ks = grad_dx_parts(M, N, K);
  cudaError_t e = launch_product<false>(dz, nullptr, lddz, w, ldw, gamma, nullptr, dx, dxdt, M, K, N, ks, part, ws, st);
  if (e != cudaSuccess) return e;
  if (ks > 1) e = launch_grad_parts(part, ks, M * K, gamma, dx, dxdt, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_grad_dw(const uint16_t* dz, const int8_t* xq, const float* scale, const float* gamma, int64_t M,
                           int64_t N, int64_t K, float* dw, const GradDwScratch& s, void* ws, cudaStream_t st) {
  const int64_t ranges = grad_rowmax_ranges(M, N), rows_per = (M + ranges - 1) / ranges;
  const int64_t ldn = grad_ld(N), ldk = grad_ld(K);
  const int cols = static_cast<int>((N + kGcCols - 1) / kGcCols), max_blocks = static_cast<int>(cols * ranges);
  const int64_t items = M * (K % 16 == 0 ? K / 16 : ldk / 8);
  cudaError_t e = launch_pdl(grad_max_kernel, static_cast<unsigned>(max_blocks) + flat_grid(items), 256, 0, st, dz,
                             scale, M, N, rows_per, s.maxes, xq, K, ldk, static_cast<__half*>(s.x), cols, max_blocks);
  if (e == cudaSuccess)
    e = launch_pdl(grad_split_kernel, dim3(static_cast<unsigned>(cols), static_cast<unsigned>(ranges)), 256, 0, st, dz,
                   scale, static_cast<const uint32_t*>(s.maxes), static_cast<int>(ranges), M, N, rows_per, ldn,
                   s.rowinv, static_cast<__half*>(s.hi), static_cast<__half*>(s.lo));
  if (e == cudaSuccess)
    e = launch_product<true>(s.hi, s.lo, ldn, s.x, ldk, gamma, s.rowinv, dw, BL_F32, N, K, M, 1, nullptr, ws, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_grad_selftest(void* op, void* ws, long long limit, cudaStream_t st) {
  const float* f = static_cast<const float*>(op);
  cudaError_t e = launch_product<false>(op, nullptr, 64, op, 64, f, nullptr, op, BL_F32, 16, 64, 16, 1, nullptr, ws, st,
                                        limit, 1);
  if (e == cudaSuccess)
    e = launch_product<true>(op, op, 64, op, 64, f, f, op, BL_F32, 16, 64, 16, 1, nullptr, ws, st, limit, 1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
