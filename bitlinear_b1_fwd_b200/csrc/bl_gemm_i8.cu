// bl_gemm_i8.cu -- the forward product of many tokens with its epilogue, on
// weights expanded to int8 beforehand.
//
//   acc[t, n] = sum_k x_q[t, k] W_q[n, k]     INT32, tcgen05.mma.kind::i8
//   z = fl(fl(acc c_t) + bias_n),  y = act(z) + residual,   c_t = (gamma s_t) / 127
//
// gemm_i2_2sm_kernel (bl_gemm_sm100.cu) expands the 2-bit weights of a tile
// again for every 256 tokens, in the warps' issue slots and shared memory that a
// rich epilogue needs too: 4096 x 3200 -> 8640 with SiLU and the kept
// pre-activation took 176 us there, 118 us with neither.  Here one pass writes
// the weights as int8 rows (N K bytes) beside the tokens' codes, and the product
// only moves tiles and computes.
//
// A cluster of two CTAs computes 256 tokens x 256 weight rows
// (tcgen05.mma.cta_group::2, M = tokens): each CTA stages 128 tokens and 128
// weight rows, 128 bytes of K a stage, both K-major by TMA, and accumulates its
// 128 tokens x 256 rows in one of two halves of tensor memory while sixteen
// epilogue warps empty the other.  An epilogue lane owns a token, so the values
// it takes from tensor memory are neighbours in y: it packs them into 16-byte
// pieces of a swizzled box of 32 tokens x 64 bytes, which one TMA tensor store
// writes; the residual comes in, and the kept pre-activation goes out, through
// boxes of the same kind.  4096 x 3200 -> 8640 with SiLU and the kept
// pre-activation, ternarized normal weights, inputs changing from call to call: 98
// us (the int8 rate bounds it at 68), 124 with the pass over the operands before it;
// equal weights, which draw less of the power cap, 114.  (With eight epilogue warps,
// and spills, the product took 1.2 times as long.)  Every wait is bounded: on expiry
// the kernel sets the workspace timeout flag, drains what it issued, frees its
// tensor memory and returns.
#include <cuda.h>
#include <cstring>

#include "bl_common.cuh"
#include "bl_epilogue.cuh"
#include "bl_gemv.cuh"
#include "bl_kernels.h"
#include "bl_sm100.cuh"
#include "bl_tensormap.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kTile = 128;                     // tokens, and weight rows, staged per CTA
constexpr int kBK = 128;                       // bytes of K per stage: four MMAs of 32
constexpr uint32_t kPlane = kTile * kBK;       // 16384 bytes
constexpr uint32_t kStage = 2 * kPlane;
constexpr int kStages = 5;
constexpr int kThreads = 640;                  // warp 0 TMA, 1 MMA, 4-19 epilogue
constexpr int kEpiWarps = 16;
constexpr uint32_t kBox = 32 * 64;             // a warp's 32 tokens x 64 bytes
constexpr uint32_t kTmemCols = 512;            // two accumulators of 256 columns
constexpr long long kTimeout = 1ll << 32;      // ~2 s at 1.9 GHz
constexpr size_t kSmem =
    1024 + kStages * kStage + 2 * kEpiWarps * kBox + 256 * 4 + 8 * (2 * kStages + 5 + kEpiWarps) + 16;
static_assert(kSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ void mma_i8_256(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// K-major operand rows of 128 bytes, 128-byte swizzle, 8-row groups 1024 bytes apart
__device__ __forceinline__ uint64_t k_major_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3fffu);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// s32 accumulator, signed A and B, both K-major, shape 256 x 256
constexpr uint32_t kIdesc = (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(256 >> 3) << 17) |
                            (static_cast<uint32_t>(256 >> 4) << 24);

template <int YDT>
struct OutElem;
template <>
struct OutElem<BL_F32> {
  using type = uint32_t;
};
template <>
struct OutElem<BL_I32> {
  using type = uint32_t;
};
template <>
struct OutElem<BL_BF16> {
  using type = uint16_t;
};

// YDT: the type of y, residual and kept pre-activation; BL_I32: no epilogue, the
// INT32 sums of part kz of a cut contraction go to plane kz of y ([ks][M][N]).
template <int YDT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                   const __grid_constant__ CUtensorMap tm_p, int o_tma, const float* __restrict__ gamma,
                   const float* __restrict__ scale, void* __restrict__ y, int M, int N, int K, int ks,
                   WsHeader* __restrict__ hdr, long long limit, int skip_producer, const Epilogue ep_arg) {
  pdl_enter(gamma, scale, y, hdr);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  uint8_t* stages = smem_raw + pad;                   // kStages x [x plane, W plane], swizzled
  uint8_t* boxes = stages + kStages * kStage;         // per epilogue warp: y (and residual), pre-activation
  float* bias_s = reinterpret_cast<float*>(boxes + 2 * kEpiWarps * kBox);  // the tile's 256 biases
  uint64_t* full = reinterpret_cast<uint64_t*>(bias_s + 256);  // leader: the loads of both CTAs
  uint64_t* empty = full + kStages;                   // local: the MMAs have read the stage
  uint64_t* accf = empty + kStages;                   // local: an accumulator is complete (2)
  uint64_t* acce = accf + 2;                          // leader: both CTAs have taken it (2)
  uint64_t* drain = acce + 2;                         // leader
  uint64_t* resf = drain + 1;                         // per epilogue warp: its residual box has landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(resf + kEpiWarps);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int kblocks = (K + kBK - 1) / kBK;
  const int j_tiles = (N - 1) / (2 * kTile) + 1;  // M and N reach 2^31 - 1: nothing is added to them
  const int tiles = j_tiles * ((M - 1) / (2 * kTile) + 1) * ks;  // ks <= kblocks: no part is empty
  // tile u: weight rows u % j_tiles, then part of the contraction, then tokens
  auto tokens_of = [&](int u) { return u / j_tiles / ks * 2 * kTile + static_cast<int>(rank) * kTile; };
  auto part_of = [&](int u) { return u / j_tiles % ks; };
  auto first_block = [&](int kz) { return static_cast<int>(static_cast<int64_t>(kz) * kblocks / ks); };
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full + s, 1);
      mbar_init(empty + s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf + a, 1);
      mbar_init(acce + a, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(resf + w, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_before();
  cluster_sync_all();  // both CTAs' barriers exist before any remote arrive or copy
  tc_after();
  const uint32_t tmem = *tmem_slot;

  auto fail = [&](uint32_t site) {
    set_flag(hdr, kFlagTimeout | kFlagProductI8, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------
    if (lane == 0 && !skip_producer) {
      int it = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += pairs) {
        const int j0 = (u % j_tiles) * 2 * kTile + static_cast<int>(rank) * kTile;
        const int i0 = tokens_of(u), kz = part_of(u), kb1 = first_block(kz + 1);
        for (int kb = first_block(kz); kb < kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (!wait1(empty + s, ((it / kStages) & 1) ^ 1, limit, abort_flag)) {
            fail(0x231);
            ok = false;
            break;
          }
          if (leader) mbar_expect_tx(full + s, 2 * kStage);
          const uint32_t bar = mapa_shared(smem_u32(full + s), 0);
          uint8_t* a = stages + s * kStage;
          tma_load_2d_pair(a, &tm_x, bar, kb * kBK, i0);
          tma_load_2d_pair(a + kPlane, &tm_w, bar, kb * kBK, j0);
        }
      }
      // this CTA's last copies have landed before it leaves, since the MMAs
      // that read them have completed (after a failure: one limit's time)
      for (int j = (it > kStages ? it - kStages : 0); j < it; ++j)
        if (!wait_drain(empty + (j % kStages), (j / kStages) & 1, limit)) break;
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (leader) -------------------------
    if (leader && lane == 0) {
      int it = 0, tc = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += pairs, ++tc) {
        const int a = tc & 1;
        if (!wait1(acce + a, ((tc >> 1) & 1) ^ 1, limit, abort_flag)) {
          fail(0x331);
          break;
        }
        tc_after();
        const uint32_t d = tmem + static_cast<uint32_t>(a * 2 * kTile);
        const int kz = part_of(u), kb0 = first_block(kz), kb1 = first_block(kz + 1);
        for (int kb = kb0; kb < kb1; ++kb, ++it) {
          const int s = it % kStages;
          if (!wait1(full + s, (it / kStages) & 1, limit, abort_flag)) {
            fail(0x332);
            ok = false;
            break;
          }
          tc_after();
          const uint32_t sa = smem_u32(stages + s * kStage);
#pragma unroll
          for (int k = 0; k < kBK / 32; ++k)
            mma_i8_256(d, k_major_desc(sa + 32 * k), k_major_desc(sa + kPlane + 32 * k), kIdesc, kb != kb0 || k != 0);
          commit_pair(empty + s, 0x3);
        }
        if (ok) commit_pair(accf + a, 0x3);
      }
      commit_pair(drain, 0x1);
      (void)wait_drain(drain, 0, limit);
    }
  } else if (warp >= 4) {
    // ------------------------------ epilogue (both CTAs) ------------------------
    // warp: 32 tokens (its tensor-memory lane quarter) x 64 weight rows, in
    // chunks of 64 bytes of y
    constexpr int NC = YDT == BL_BF16 ? 32 : 16, kCols = 64;
    const int q = warp & 3, e = warp - 4, part = e >> 2, et = threadIdx.x - 128;
    const float g = __ldcg(gamma);
    Epilogue ep = epilogue_after_wait(ep_arg);
    if constexpr (YDT == BL_I32) ep.res = ep.pre = nullptr;
    uint8_t* box = boxes + 2 * e * kBox;
    uint8_t* row = box + lane * 64;  // this lane's token, its 16-byte pieces in the 64-byte swizzle
    auto piece = [&](int c) { return reinterpret_cast<uint4*>(row + ((c ^ ((lane >> 1) & 3)) << 4)); };
    // Rows of y that are no multiple of 16 bytes have no tensor map: the warp
    // copies between its box and an array itself, neighbouring lanes neighbouring
    // columns (tokens i0 .., columns c .. of the array).
    using Elem = typename OutElem<YDT>::type;
    auto cell = [&](uint8_t* bx, int r, int c) {  // token r, column c of a box
      const int at = c * static_cast<int>(sizeof(Elem));
      return reinterpret_cast<Elem*>(bx + r * 64 + ((((at >> 4) ^ ((r >> 1) & 3)) << 4) | (at & 15)));
    };
    auto box_in = [&](uint8_t* bx, const void* src, int i0, int c0) {
#pragma unroll 4
      for (int r = lane / NC; r < 32; r += 32 / NC) {
        const int c = lane % NC;
        if (i0 + r < M && c0 + c < N)
          *cell(bx, r, c) = __ldcg(static_cast<const Elem*>(src) + static_cast<int64_t>(i0 + r) * N + c0 + c);
      }
    };
    auto box_out = [&](void* dst, uint8_t* bx, int i0, int c0) {
#pragma unroll 4
      for (int r = lane / NC; r < 32; r += 32 / NC) {
        const int c = lane % NC;
        if (i0 + r < M && c0 + c < N)
          static_cast<Elem*>(dst)[static_cast<int64_t>(i0 + r) * N + c0 + c] = *cell(bx, r, c);
      }
    };
    uint32_t res_phase = 0;
    int tc = 0;
    bool ok = true;
    for (int u = pair; u < tiles; u += pairs, ++tc) {
      // every warp is done with the previous tile's biases, or one has given up
      uint32_t go;
      asm volatile(
          "{\n\t.reg .pred pi, po;\n\t"
          "setp.ne.u32 pi, %1, 0;\n\t"
          "bar.red.and.pred po, 1, 512, pi;\n\t"
          "selp.u32 %0, 1, 0, po;\n\t}"
          : "=r"(go)
          : "r"(ok ? 1u : 0u)
          : "memory");
      if (!go) break;
      const int a = tc & 1;
      const int i0 = tokens_of(u) + 32 * q;
      const int jt = (u % j_tiles) * 2 * kTile, j0 = jt + part * kCols;
      const float cf = YDT != BL_I32 && i0 + lane < M ? dequant_factor(g, __ldcg(scale + i0 + lane)) : 0.0f;
      if (et < 256) bias_s[et] = ep.bias != nullptr && jt + et < N ? __ldcg(ep.bias + jt + et) : 0.0f;
      asm volatile("bar.sync 1, 512;" ::: "memory");
      if (!wait_warp(accf + a, (tc >> 1) & 1, limit, abort_flag)) {
        if (lane == 0) fail(0x531);
        ok = false;
      }
      tc_after();
#pragma unroll 1
      for (int c0 = 0; c0 < kCols; c0 += NC) {
        const bool live = ok && i0 < M && j0 + c0 < N;  // (uniform)
        if (lane == 0) bulk_wait_read<0>();  // the stores issued from the boxes have read them
        __syncwarp();
        if (live && ep.res != nullptr) {
          if (!o_tma) {
            box_in(box, ep.res, i0, j0 + c0);
          } else if (lane == 0) {
            mbar_expect_tx(resf + e, kBox);
            tma_load_2d(box, &tm_r, resf + e, j0 + c0, i0);
          }
        }
        uint32_t v[NC];
        if (ok) {
#pragma unroll
          for (int c = 0; c < NC; c += 16) {
            uint32_t t[16];
            tmem_load16(tmem + (static_cast<uint32_t>(32 * q) << 16) +
                            static_cast<uint32_t>(a * 2 * kTile + part * kCols + c0 + c), t);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[c + j] = t[j];
          }
        }
        if (c0 + NC == kCols) {  // the accumulator has been read
          tc_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(acce + a), 0));
        }
        if (!live) continue;
        if constexpr (YDT != BL_I32) {
          const float4* bs = reinterpret_cast<const float4*>(bias_s + part * kCols + c0);
#pragma unroll
          for (int j = 0; j < NC; j += 4) {
            const float4 b = bs[j / 4];
            const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              v[j + k] = __float_as_uint(__fadd_rn(__fmul_rn(__int2float_rn(static_cast<int>(v[j + k])), cf), bb[k]));
          }
        }
        auto put = [&](uint32_t at) {  // v as 16-byte pieces of this lane's row of a box
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 p;
            if constexpr (YDT != BL_BF16) {
              p = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            } else {
              auto two = [&](int j) { return bf16_pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1])); };
              p = make_uint4(two(8 * c), two(8 * c + 2), two(8 * c + 4), two(8 * c + 6));
            }
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(piece(c)) + at) = p;
          }
        };
        if (ep.pre != nullptr) put(kBox);
        if constexpr (YDT != BL_I32) epilogue_act<NC, YDT == BL_BF16>(ep.act, v);
        if (ep.res != nullptr) {
          if (!o_tma) {
            __syncwarp();
          } else if (!wait_warp(resf + e, res_phase, limit, abort_flag)) {
            if (lane == 0) {
              fail(0x532);
              (void)wait_drain(resf + e, res_phase, limit);
            }
            ok = false;
            continue;
          }
          res_phase ^= 1;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint4 p = *piece(c);
            const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (YDT != BL_BF16) {
                v[4 * c + k] = __float_as_uint(__fadd_rn(__uint_as_float(v[4 * c + k]), __uint_as_float(w[k])));
              } else {
                uint32_t* d = v + 8 * c + 2 * k;
                d[0] = __float_as_uint(__fadd_rn(__uint_as_float(d[0]), __uint_as_float(w[k] << 16)));
                d[1] = __float_as_uint(__fadd_rn(__uint_as_float(d[1]), __uint_as_float(w[k] & 0xffff0000u)));
              }
            }
          }
        }
        put(0);
        if (!o_tma) {
          __syncwarp();
          box_out(YDT == BL_I32 ? static_cast<int32_t*>(y) + static_cast<int64_t>(part_of(u)) * M * N : y, box, i0,
                  j0 + c0);
          if (ep.pre != nullptr) box_out(ep.pre, box + kBox, i0, j0 + c0);
          continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if constexpr (YDT == BL_I32)
            tma_store_3d(&tm_y, box, j0 + c0, i0, part_of(u));
          else
            tma_store_2d(&tm_y, box, j0 + c0, i0);
          if (ep.pre != nullptr) tma_store_2d(&tm_p, box + kBox, j0 + c0, i0);
          bulk_commit();
        }
      }
    }
    if (lane == 0) bulk_wait<0>();  // every output has landed before the CTA leaves
  }

  __syncthreads();
  tc_before();
  cluster_sync_all();  // no CTA leaves while its peer may still signal its barriers
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// ---- the operands -------------------------------------------------------------------
// One launch for both (they are independent, and each alone leaves SMs idle at
// its end): the first blocks expand weights, the others quantize a token each.
constexpr int kPrepThreads = 128;
constexpr int kPrepChunk = 16 * kPrepThreads;  // columns a block turns around in shared memory at a time

// 16-weight word w of a segment of any format as int8.
template <int FMT>
__device__ __forceinline__ void expand_segments(const uint8_t* packed, int64_t N, int64_t rowbytes, int64_t ldw,
                                                uint4* w, int64_t item, int64_t stride) {
  if constexpr (FMT == BL_PACK_I2) {  // a word per item: rows stay aligned with each other (ldw = 4 rowbytes)
    const uint32_t* src = reinterpret_cast<const uint32_t*>(packed);
    const int64_t words = N * (rowbytes / 4);
    for (; item + 3 * stride < words; item += 4 * stride) {
      uint32_t v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = __ldcg(src + item + u * stride);
#pragma unroll
      for (int u = 0; u < 4; ++u) w[item + u * stride] = expand16(v[u]);
    }
    for (; item < words; item += stride) w[item] = expand16(__ldcg(src + item));
  } else {  // a segment per item: 80 or 128 weights, cut at the row's end
    constexpr int W = FMT == BL_PACK_T5 ? 5 : 8;
    const uint32_t segs = static_cast<uint32_t>(rowbytes >> 4);
    const int64_t items = N * segs, row_words = ldw / 16;
    for (; item < items; item += stride) {
      const int64_t n = item / segs, sg = item - n * segs;
      const uint4 v = __ldcg(reinterpret_cast<const uint4*>(packed) + item);
      uint4* dst = w + n * row_words;
      if constexpr (FMT == BL_PACK_T5) {
        uint32_t c[5];
        t5_segment(v, c);
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (sg * W + i < row_words) dst[sg * W + i] = expand16(c[i]);
      } else {
        const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (sg * W + i < row_words) dst[sg * W + i] = expand16_bits((i & 1) ? c[i >> 1] >> 16 : c[i >> 1]);
      }
    }
  }
}

// Codes of token m in rows of ldx bytes (zeros past K) and its scale (XDT = I8:
// the codes are given and only take the new row length).  A row's first 4096
// values are read once and kept in registers.
template <int XDT>
__device__ __forceinline__ void quantize_token(const void* x, int64_t m, int64_t K, int64_t ldx, int8_t* xq,
                                               float* scale, uint8_t* turn, BlockSum& sum) {
  int8_t* out = xq + m * ldx;
  if constexpr (XDT != BL_I8) {
    if (K % 8 == 0) {
      constexpr int kKeep = 4;
      Raw<XDT, 8> r[kKeep];
      float amax = 0.0f;
      auto take = [&](const Raw<XDT, 8>& q) {
        float v[8];
        q.get(v);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
      };
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int64_t k = 8 * (static_cast<int64_t>(i) * kPrepThreads + threadIdx.x);
        if (k < K) r[i].load(x, m * K + k);
        else r[i].zero();
      }
#pragma unroll
      for (int i = 0; i < kKeep; ++i) take(r[i]);
      for (int64_t k = 8 * (static_cast<int64_t>(kKeep) * kPrepThreads + threadIdx.x); k < K; k += 8 * kPrepThreads) {
        Raw<XDT, 8> q;
        q.load(x, m * K + k);
        take(q);
      }
      const float s = fmaxf(sum.max(amax), 1e-6f), c127 = __fdiv_rn(127.0f, s);
      if (threadIdx.x == 0) scale[m] = s;
      auto give = [&](const Raw<XDT, 8>& q, int64_t k) {
        float v[8];
        int c[8];
        q.get(v);
        quant_act_fast_n<8>(v, s, c127, c);
        *reinterpret_cast<uint2*>(out + k) = make_uint2(pack4(c), pack4(c + 4));
      };
#pragma unroll
      for (int i = 0; i < kKeep; ++i) {
        const int64_t k = 8 * (static_cast<int64_t>(i) * kPrepThreads + threadIdx.x);
        if (k < K) give(r[i], k);
      }
      for (int64_t k = 8 * (static_cast<int64_t>(kKeep) * kPrepThreads + threadIdx.x); k < K; k += 8 * kPrepThreads) {
        Raw<XDT, 8> q;
        q.load(x, m * K + k);
        give(q, k);
      }
      if (threadIdx.x == 0 && K < ldx) *reinterpret_cast<uint2*>(out + K) = make_uint2(0u, 0u);
      return;
    }
  }
  // rows that start anywhere: neighbouring threads load neighbouring values, and
  // the codes turn around in shared memory into 16-byte stores
  float s = 1.0f, c127 = 0.0f;
  if constexpr (XDT != BL_I8) {
    float amax = 0.0f;
#pragma unroll 8
    for (int64_t k = threadIdx.x; k < K; k += kPrepThreads) amax = fmaxf(amax, fabsf(load_elem<XDT>(x, m * K + k)));
    s = fmaxf(sum.max(amax), 1e-6f);
    c127 = __fdiv_rn(127.0f, s);
    if (threadIdx.x == 0) scale[m] = s;
  }
  for (int64_t k0 = 0; k0 < ldx; k0 += kPrepChunk) {
#pragma unroll 8
    for (int i = 0; i < kPrepChunk / kPrepThreads; ++i) {
      const int at = i * kPrepThreads + threadIdx.x;
      const int64_t k = k0 + at;
      int c = 0;
      if (k < K) {
        if constexpr (XDT == BL_I8)
          c = __ldcg(static_cast<const signed char*>(x) + m * K + k);
        else
          c = quant_act_fast(load_elem<XDT>(x, m * K + k), s, c127);
      }
      turn[at] = static_cast<uint8_t>(c);
    }
    __syncthreads();
    const int64_t k = k0 + 16 * threadIdx.x;
    if (k < ldx) *reinterpret_cast<uint4*>(out + k) = *reinterpret_cast<const uint4*>(turn + 16 * threadIdx.x);
    __syncthreads();
  }
}

template <int FMT, int XDT>
__global__ void __launch_bounds__(kPrepThreads)
    gemm_operands_kernel(const uint8_t* __restrict__ packed, int64_t N, int64_t K, int64_t rowbytes, int64_t ldw,
                         uint4* __restrict__ w, int wblocks, const void* __restrict__ x, int64_t M, int64_t ldx,
                         int8_t* __restrict__ xq, float* __restrict__ scale) {
  pdl_enter(packed, w, x, xq, scale);
  if (static_cast<int>(blockIdx.x) < wblocks) {
    expand_segments<FMT>(packed, N, rowbytes, ldw, w, static_cast<int64_t>(blockIdx.x) * kPrepThreads + threadIdx.x,
                         static_cast<int64_t>(wblocks) * kPrepThreads);
    return;
  }
  __shared__ __align__(16) uint8_t turn[kPrepChunk];
  __shared__ __align__(16) float sum_mem[2][4][32];
  BlockSum sum(sum_mem);
  for (int64_t m = blockIdx.x - wblocks; m < M; m += gridDim.x - wblocks)
    quantize_token<XDT>(x, m, K, ldx, xq, scale, turn, sum);
}

// The parts of a cut contraction (exact INT32 sums, V = 4 or 1 neighbouring
// outputs per thread), then the epilogue.
template <int V>
__global__ void __launch_bounds__(128)
    gemm_parts_kernel(const int32_t* __restrict__ part, int ks, int64_t M, int64_t N, const float* __restrict__ gamma,
                      const float* __restrict__ scale, void* __restrict__ y, int ydt, const Epilogue ep_arg) {
  pdl_enter(part, gamma, scale, y);
  const Epilogue ep = epilogue_after_wait(ep_arg);
  const float g = __ldcg(gamma);
  const int64_t plane = M * N, stride = static_cast<int64_t>(gridDim.x) * blockDim.x * V;
  for (int64_t o = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) * V; o < plane; o += stride) {
    int s[V];
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] = 0;
#pragma unroll 8
    for (int kz = 0; kz < ks; ++kz) {
      if constexpr (V == 4) {
        const int4 p = __ldcg(reinterpret_cast<const int4*>(part + kz * plane + o));
        s[0] += p.x;
        s[1] += p.y;
        s[2] += p.z;
        s[3] += p.w;
      } else {
        s[0] += __ldcg(part + kz * plane + o);
      }
    }
    const int64_t m = o / N, n = o - m * N;
    const float cf = dequant_factor(g, __ldcg(scale + m));
#pragma unroll
    for (int j = 0; j < V; ++j) epilogue_store(ep, y, ydt, o + j, n + j, s[j], cf);
  }
}

}  // namespace

// Parts of the contraction: few tiles leave most SMs without work (128 tokens,
// 8640 -> 3200: 13 tiles, 36 us whole and 25 us in parts).  The number in 1..16
// with the least work on the busiest pair of SMs, in k-blocks, plus 3 per tile
// (filling the ring, the epilogue) and for the pass over the parts 8 and their
// bytes' worth.
int gemm_i8_parts(int64_t M, int64_t N, int64_t K) {
  const int64_t tiles = ((N + 2 * kTile - 1) / (2 * kTile)) * ((M + 2 * kTile - 1) / (2 * kTile));
  const int64_t kblocks = (K + kBK - 1) / kBK, pairs = device_sms() / 2 > 0 ? device_sms() / 2 : 1;
  int best = 1;
  int64_t best_cost = -1;
  for (int ks = 1; ks <= 16 && ks <= kblocks; ++ks) {
    const int64_t cost = (tiles * ks + pairs - 1) / pairs * ((kblocks + ks - 1) / ks + 3) +
                         (ks > 1 ? 8 + ks * M * N / 500000 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best_cost = cost;
      best = ks;
    }
  }
  return best;
}

int64_t gemm_i8_row(int64_t K, int fmt) {
  return fmt == BL_PACK_I2 ? (K + 63) / 64 * 64 : (K + 15) / 16 * 16;
}

cudaError_t launch_gemm_operands(const uint8_t* packed, int fmt, int64_t rowbytes, int64_t N, int64_t K, int8_t* w,
                                 const void* x, int xdt, int64_t M, int64_t ldx, int8_t* xq, float* scale,
                                 cudaStream_t st) {
  const int64_t items = fmt == BL_PACK_I2 ? N * (rowbytes / 4) / 4 : N * (rowbytes / 16);
  const int64_t cap = static_cast<int64_t>(device_sms()) * 8, g = (items + kPrepThreads - 1) / kPrepThreads;
  const int wblocks = static_cast<int>(g < cap ? (g < 1 ? 1 : g) : cap);
  const int64_t grid = wblocks + (xq == nullptr ? 0 : (M < (1 << 20) ? M : 1 << 20));
  auto run = [&](auto kern) {
    return launch_pdl(kern, static_cast<unsigned>(grid), kPrepThreads, 0, st, packed, N, K, rowbytes,
                      gemm_i8_row(K, fmt), reinterpret_cast<uint4*>(w), wblocks, x, M, ldx, xq, scale);
  };
#define BL_GO(FMT)                                                        \
  return xdt == BL_F32    ? run(gemm_operands_kernel<FMT, BL_F32>)        \
         : xdt == BL_BF16 ? run(gemm_operands_kernel<FMT, BL_BF16>)       \
                          : run(gemm_operands_kernel<FMT, BL_I8>)
  if (fmt == BL_PACK_I2) BL_GO(BL_PACK_I2);
  if (fmt == BL_PACK_T5) BL_GO(BL_PACK_T5);
  BL_GO(BL_PACK_B1);
#undef BL_GO
}

cudaError_t launch_gemm_i8(const int8_t* xq, int64_t ldx, const int8_t* w, int64_t ldw, const float* gamma,
                           const float* scale, void* y, int ydt, int64_t M, int64_t N, int64_t K, const Epilogue& ep,
                           int32_t* part, void* ws, long long limit, int skip_producer, cudaStream_t st) {
  CUtensorMap tx, tw, ty, tr, tp;
  if (!encode_2d_u8(&tx, xq, static_cast<uint64_t>(K), static_cast<uint64_t>(M), static_cast<uint64_t>(ldx), kBK, kTile,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d_u8(&tw, w, static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(ldw), kBK, kTile,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const int ks = skip_producer ? 1 : gemm_i8_parts(M, N, K);
  const int odt = ks > 1 ? static_cast<int>(BL_I32) : ydt;
  void* out = ks > 1 ? part : y;
  auto box_map = [&](CUtensorMap* m, const void* p) {
    return encode_out(m, const_cast<void*>(p), odt != BL_BF16, static_cast<uint64_t>(N), static_cast<uint64_t>(M),
                         ks > 1 ? static_cast<uint64_t>(ks) : 0, 64);
  };
  const int o_tma = N * (odt == BL_BF16 ? 2 : 4) % 16 == 0 ? 1 : 0;
  memset(&ty, 0, sizeof ty);
  if (o_tma && !box_map(&ty, out)) return cudaErrorInvalidValue;
  tr = tp = ty;
  if (o_tma && ks == 1 && ep.res != nullptr && !box_map(&tr, ep.res)) return cudaErrorInvalidValue;
  if (o_tma && ks == 1 && ep.pre != nullptr && !box_map(&tp, ep.pre)) return cudaErrorInvalidValue;
  auto kern = odt == BL_I32 ? gemm_i8_kernel<BL_I32> : odt == BL_F32 ? gemm_i8_kernel<BL_F32> : gemm_i8_kernel<BL_BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((N + 2 * kTile - 1) / (2 * kTile)) * ((M + 2 * kTile - 1) / (2 * kTile)) * ks;
  const int64_t most = device_sms() / 2, pairs = tiles < most ? tiles : most;
  e = launch_pdl(kern, static_cast<unsigned>(2 * pairs), kThreads, kSmem, st, tx, tw, ty, tr, tp, o_tma, gamma, scale,
                 out, static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), ks, static_cast<WsHeader*>(ws),
                 limit > 0 ? limit : kTimeout, skip_producer, ep);
  if (e == cudaSuccess && ks > 1) {
    const int64_t v = N % 4 == 0 ? 4 : 1, cap = static_cast<int64_t>(device_sms()) * 16, g = (M * N / v + 127) / 128;
    e = launch_pdl(v == 4 ? gemm_parts_kernel<4> : gemm_parts_kernel<1>, static_cast<unsigned>(g < cap ? g : cap), 128,
                   0, st, static_cast<const int32_t*>(part), ks, M, N, gamma, scale, y, ydt, ep);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
