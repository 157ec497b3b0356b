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
// the weights as int8 rows (N K bytes, 7 us for that layer) and the product only
// moves tiles and computes.
//
// A cluster of two CTAs computes 256 tokens x 256 weight rows
// (tcgen05.mma.cta_group::2, M = tokens): each CTA stages 128 tokens and 128
// weight rows, 128 bytes of K a stage, both K-major by TMA, and accumulates its
// 128 tokens x 256 rows in one of two halves of tensor memory while sixteen
// epilogue warps empty the other.  An epilogue lane owns a token, so the values
// it takes from tensor memory are neighbours in y: it packs them into 16-byte
// pieces of a swizzled box of 32 tokens x 64 bytes, which one TMA tensor store
// writes; the residual comes in, and the kept pre-activation goes out, through
// boxes of the same kind.  Every wait is bounded: on expiry the kernel sets the
// workspace timeout flag, drains what it issued, frees its tensor memory and
// returns.
#include <cuda.h>
#include <cstring>

#include "bl_common.cuh"
#include "bl_epilogue.cuh"
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
struct OutElem<BL_BF16> {
  using type = uint16_t;
};

// YDT: the type of y, residual and kept pre-activation
template <int YDT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    gemm_i8_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                   const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r,
                   const __grid_constant__ CUtensorMap tm_p, int o_tma, const float* __restrict__ gamma,
                   const float* __restrict__ scale, void* __restrict__ y, int M, int N, int K,
                   WsHeader* __restrict__ hdr, long long limit, const Epilogue ep_arg) {
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
  const int j_tiles = (N + 2 * kTile - 1) / (2 * kTile);
  const int tiles = j_tiles * ((M + 2 * kTile - 1) / (2 * kTile));
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
    set_flag(hdr, kFlagTimeout, site);
    *abort_flag = 1;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int u = pair; u < tiles && ok; u += pairs) {
        const int j0 = (u % j_tiles) * 2 * kTile + static_cast<int>(rank) * kTile;
        const int i0 = (u / j_tiles) * 2 * kTile + static_cast<int>(rank) * kTile;
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
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
        for (int kb = 0; kb < kblocks; ++kb, ++it) {
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
            mma_i8_256(d, k_major_desc(sa + 32 * k), k_major_desc(sa + kPlane + 32 * k), kIdesc, (kb | k) != 0);
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
    constexpr int NC = YDT == BL_F32 ? 16 : 32, kCols = 64;
    const int q = warp & 3, e = warp - 4, part = e >> 2, et = threadIdx.x - 128;
    const float g = __ldcg(gamma);
    const Epilogue ep = epilogue_after_wait(ep_arg);
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
      const int i0 = (u / j_tiles) * 2 * kTile + static_cast<int>(rank) * kTile + 32 * q;
      const int jt = (u % j_tiles) * 2 * kTile, j0 = jt + part * kCols;
      const float cf = i0 + lane < M ? dequant_factor(g, __ldcg(scale + i0 + lane)) : 0.0f;
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
        const float4* bs = reinterpret_cast<const float4*>(bias_s + part * kCols + c0);
#pragma unroll
        for (int j = 0; j < NC; j += 4) {
          const float4 b = bs[j / 4];
          const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            v[j + k] = __float_as_uint(__fadd_rn(__fmul_rn(__int2float_rn(static_cast<int>(v[j + k])), cf), bb[k]));
        }
        auto put = [&](uint32_t at) {  // v as 16-byte pieces of this lane's row of a box
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4 p;
            if constexpr (YDT == BL_F32) {
              p = make_uint4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
            } else {
              auto two = [&](int j) { return bf16_pair(__uint_as_float(v[j]), __uint_as_float(v[j + 1])); };
              p = make_uint4(two(8 * c), two(8 * c + 2), two(8 * c + 4), two(8 * c + 6));
            }
            *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(piece(c)) + at) = p;
          }
        };
        if (ep.pre != nullptr) put(kBox);
        epilogue_act<NC, YDT == BL_BF16>(ep.act, v);
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
              if constexpr (YDT == BL_F32) {
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
          box_out(y, box, i0, j0 + c0);
          if (ep.pre != nullptr) box_out(ep.pre, box + kBox, i0, j0 + c0);
          continue;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
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

// 2-bit rows as int8 rows of 4 rowbytes codes (padding decodes to 0): one packed
// word (16 weights, 16 output bytes) per item, four in flight.
__global__ void __launch_bounds__(256)
    i2_to_i8_kernel(const uint32_t* __restrict__ i2, int64_t words, uint4* __restrict__ w) {
  pdl_enter(i2, w);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  int64_t s = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  for (; s + 3 * stride < words; s += 4 * stride) {
    uint32_t v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = __ldcg(i2 + s + u * stride);
#pragma unroll
    for (int u = 0; u < 4; ++u) w[s + u * stride] = expand16(v[u]);
  }
  for (; s < words; s += stride) w[s] = expand16(__ldcg(i2 + s));
}

}  // namespace

cudaError_t launch_i2_to_i8(const uint8_t* i2, int64_t N, int64_t rowbytes, int8_t* w, cudaStream_t st) {
  const int64_t words = N * (rowbytes / 4), cap = static_cast<int64_t>(device_sms()) * 8, g = (words + 255) / 256;
  return launch_pdl(i2_to_i8_kernel, static_cast<unsigned>(g < cap ? g : cap), 256, 0, st,
                    reinterpret_cast<const uint32_t*>(i2), words, reinterpret_cast<uint4*>(w));
}

cudaError_t launch_gemm_i8(const int8_t* xq, int64_t ldx, const int8_t* w, int64_t ldw, const float* gamma,
                           const float* scale, void* y, int ydt, int64_t M, int64_t N, int64_t K, const Epilogue& ep,
                           void* ws, cudaStream_t st) {
  CUtensorMap tx, tw, ty, tr, tp;
  if (!encode_2d_u8(&tx, xq, static_cast<uint64_t>(K), static_cast<uint64_t>(M), static_cast<uint64_t>(ldx), kBK, kTile,
                    CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d_u8(&tw, w, static_cast<uint64_t>(K), static_cast<uint64_t>(N), static_cast<uint64_t>(ldw), kBK, kTile,
                    CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto box_map = [&](CUtensorMap* m, const void* p) {
    return encode_out_2d(m, const_cast<void*>(p), ydt == BL_F32, static_cast<uint64_t>(N), static_cast<uint64_t>(M));
  };
  const int o_tma = N * (ydt == BL_F32 ? 4 : 2) % 16 == 0 ? 1 : 0;
  memset(&ty, 0, sizeof ty);
  if (o_tma && !box_map(&ty, y)) return cudaErrorInvalidValue;
  tr = tp = ty;
  if (o_tma && ep.res != nullptr && !box_map(&tr, ep.res)) return cudaErrorInvalidValue;
  if (o_tma && ep.pre != nullptr && !box_map(&tp, ep.pre)) return cudaErrorInvalidValue;
  auto kern = ydt == BL_F32 ? gemm_i8_kernel<BL_F32> : gemm_i8_kernel<BL_BF16>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem));
  if (e != cudaSuccess) return e;
  const int64_t tiles = ((N + 2 * kTile - 1) / (2 * kTile)) * ((M + 2 * kTile - 1) / (2 * kTile));
  const int64_t most = device_sms() / 2, pairs = tiles < most ? tiles : most;
  e = launch_pdl(kern, static_cast<unsigned>(2 * pairs), kThreads, kSmem, st, tx, tw, ty, tr, tp, o_tma, gamma, scale, y,
                 static_cast<int>(M), static_cast<int>(N), static_cast<int>(K), static_cast<WsHeader*>(ws), kTimeout,
                 ep);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
