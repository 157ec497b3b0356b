// bl_norm.cu -- the norms around a block's end with its gate and residual
// scale, forward and backward.
//
//   u = norm_post(b) w1 + b1;  h = rs r + bs gate u;  y = norm_pre(h) w2 + b2
//   xq, s = per-token absmax INT8 of y
// and, with n1, n2 the normalised rows, r1, r2 = 1 / deviation:
//   dn2 = dy w2;  dh = dh_in + r2 (dn2 - [mean dn2] - n2 mean(dn2 n2))
//   dr = rs dh;   du = bs gate dh;  dn1 = du w1
//   db = r1 (dn1 - [mean dn1] - n1 mean(dn1 n1))
//   dw2 = sum dy n2;  db2 = sum dy;  dgate = sum bs dh u;  dw1 = sum du n1;  db1 = sum du
// ([mean ...] for LayerNorm only.)
//
// Both are bound by HBM in principle (forward: b and r read, h and y or the
// codes written; backward: four arrays read, two written), so a block keeps a
// token's row in registers from the load to the store: one read and one write
// of each array.  What is left to hide is latency: the next row is loaded while
// this one is worked on, the per-column vectors (gate, weights, biases) are
// folded once per block into slots of shared memory that belong to their
// thread, and a row takes one barrier per dependent sum (RMS + RMS: two, and one
// for the codes' maximum; backward two).  The column sums of the backward stay
// in registers over a block's rows and meet in a second kernel in a fixed order.
// Statistics are two-pass (the mean, then the squares about it) in fp32.
#include "bl_common.cuh"
#include "bl_gemv.cuh"
#include "bl_kernels.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

// Threads of a block, by chunks and values per thread: what its registers allow.
constexpr int norm_max_threads(int vec, int ni) { return vec == 8 && ni == 2 ? 576 : 512; }
constexpr int grad_max_threads(int vec, int ni) { return vec == 8 && ni == 1 || ni == 4 ? 512 : 384; }
constexpr int kNormLongThreads = 512;
constexpr int kGradBlocks = 1;  // backward: blocks per SM
constexpr size_t kGradSmemBudget = 225 * 1024;  // slots of the backward

__device__ __forceinline__ NormParams params_after_wait(NormParams p) {
  pdl_after(p.post_w);
  pdl_after(p.post_b);
  pdl_after(p.gate);
  pdl_after(p.pre_w);
  pdl_after(p.pre_b);
  return p;
}

// VEC values of a per-column vector (NULL: the constant c).
template <int VEC>
__device__ __forceinline__ void load_col(const float* p, int64_t k, float c, float* v) {
  if (p == nullptr) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = c;
  } else if ((reinterpret_cast<uintptr_t>(p + k) & 15) == 0 && VEC == 8) {
    load_vec<BL_F32, VEC>(p, k, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __ldcg(p + k + j);
  }
}

// 1 / sqrt of the mean square plus eps
__device__ __forceinline__ float inv_dev(float sumsq, int64_t K, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(sumsq / static_cast<float>(K) + eps));
}

// Column of value j of a thread's chunk i (VEC = 8: chunks of 8 neighbouring
// columns; VEC = 1: neighbouring threads hold neighbouring columns).
template <int VEC>
__device__ __forceinline__ int64_t col0(int i) {
  return (static_cast<int64_t>(i) * blockDim.x + threadIdx.x) * VEC;
}

// Per-column vectors folded once per block: vector v of chunk i of this thread,
// in shared slots that no other thread touches (16-byte accesses of
// neighbouring threads are neighbours).
template <int VEC, int NI>
struct Slots {
  float* s;
  __device__ __forceinline__ void put(int v, int i, const float* x) {
    if constexpr (VEC == 8) {
      float4* q = reinterpret_cast<float4*>(s) + (v * NI + i) * 2 * blockDim.x + threadIdx.x;
      q[0] = make_float4(x[0], x[1], x[2], x[3]);
      q[blockDim.x] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
      s[(v * NI + i) * blockDim.x + threadIdx.x] = x[0];
    }
  }
  __device__ __forceinline__ void get(int v, int i, float* x) const {
    if constexpr (VEC == 8) {
      const float4* q = reinterpret_cast<const float4*>(s) + (v * NI + i) * 2 * blockDim.x + threadIdx.x;
      const float4 a = q[0], b = q[blockDim.x];
      x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
      x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
      x[0] = s[(v * NI + i) * blockDim.x + threadIdx.x];
    }
  }
};

// bs gate w1 and bs gate b1: the branch's factor and offset, h = rs r + gw n1 + gb
template <int VEC>
__device__ __forceinline__ void branch_factor(const NormParams& p, const float* gate, int64_t k, float* gw) {
  float g[VEC];
  load_col<VEC>(gate, k, 1.0f, g);
  load_col<VEC>(p.post_w, k, 1.0f, gw);
#pragma unroll
  for (int j = 0; j < VEC; ++j) gw[j] = __fmul_rn(__fmul_rn(p.branch_scale, g[j]), gw[j]);
}
template <int VEC>
__device__ __forceinline__ void branch_offset(const NormParams& p, const float* gate, int64_t k, float* gb) {
  float g[VEC];
  load_col<VEC>(gate, k, 1.0f, g);
  load_col<VEC>(p.post_b, k, 0.0f, gb);
#pragma unroll
  for (int j = 0; j < VEC; ++j) gb[j] = __fmul_rn(__fmul_rn(p.branch_scale, g[j]), gb[j]);
}

// Normalises the row held in v (zeros past K) in place; returns 1 / deviation.
template <int VEC, int NI>
__device__ __forceinline__ float normalise(float (&v)[NI][VEC], int kind, float eps, int64_t K, BlockSum& sum) {
  if (kind == BL_NORM_NONE) return 1.0f;
  if (kind == BL_NORM_LAYER) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s += v[i][j];
    const float mean = sum.one(s) / static_cast<float>(K);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = col0<VEC>(i) < K ? v[i][j] - mean : 0.0f;
  }
  float q = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) q += v[i][j] * v[i][j];
  const float r = inv_dev(sum.one(q), K, eps);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] *= r;
  return r;
}

// ---- forward, the row in registers --------------------------------------------
// Up to 16 values per thread: the next row is in flight during this one, and the
// column vectors sit in shared slots (0: gw, 1: w2, 2: gb, 3: b2); 32 values:
// neither fits, the vectors are read again for each row.
constexpr bool norm_hold(int values) { return values <= 16; }

template <int BDT, int RDT, int VEC, int NI, bool BIAS>
__global__ void __launch_bounds__(norm_max_threads(VEC, NI))
    residual_norm_kernel(const NormParams p_arg, const void* __restrict__ b, const void* __restrict__ r, int64_t M,
                         int64_t K, void* __restrict__ h, void* __restrict__ y, int ydt, int8_t* __restrict__ xq,
                         float* __restrict__ scale) {
  pdl_enter(b, r, h, y, xq, scale);
  const NormParams p = params_after_wait(p_arg);
  constexpr bool kHold = norm_hold(VEC * NI);
  extern __shared__ __align__(16) float slot_mem[];
  Slots<VEC, NI> slots{slot_mem};
  __shared__ float4 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  Raw<BDT, VEC> nb[NI];
  Raw<RDT, VEC> nr[NI];
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (m < M && k < K) {
        nb[i].load(b, m * K + k);
        nr[i].load(r, m * K + k);
      } else {
        nb[i].zero();
        nr[i].zero();
      }
    }
  };
  auto gate_row = [&](int64_t m) { return p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K; };
  auto hold_branch = [&](int64_t m) {
    const float* gate = gate_row(m);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float t[VEC];
        branch_factor<VEC>(p, gate, k, t);
        slots.put(0, i, t);
        if constexpr (BIAS) {
          branch_offset<VEC>(p, gate, k, t);
          slots.put(2, i, t);
        }
      }
    }
  };
  fetch(blockIdx.x);
  int64_t g_next = M;  // first token past the gate row held in the slots
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float t[VEC];
        load_col<VEC>(p.pre_w, k, 1.0f, t);
        slots.put(1, i, t);
        if constexpr (BIAS) {
          load_col<VEC>(p.pre_b, k, 0.0f, t);
          slots.put(3, i, t);
        }
      }
    }
    hold_branch(blockIdx.x);
    if (p.gate != nullptr) g_next = (blockIdx.x / p.gate_rows + 1) * p.gate_rows;
  }
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    float v[NI][VEC], rr[NI][VEC];
    if constexpr (!kHold) {
      if (m != blockIdx.x) fetch(m);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      nb[i].get(v[i]);
      nr[i].get(rr[i]);
    }
    if constexpr (kHold) {
      fetch(m + gridDim.x);
      if (m >= g_next) {
        hold_branch(m);
        g_next = (m / p.gate_rows + 1) * p.gate_rows;
      }
    }
    normalise<VEC, NI>(v, p.post, p.post_eps, K, sum);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float gw[VEC], gb[VEC];
        if constexpr (kHold) {
          slots.get(0, i, gw);
          if constexpr (BIAS) slots.get(2, i, gb);
        } else {
          branch_factor<VEC>(p, gate_row(m), k, gw);
          if constexpr (BIAS) branch_offset<VEC>(p, gate_row(m), k, gb);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float t = p.res_scale * rr[i][j];
          if constexpr (BIAS) t += gb[j];
          v[i][j] = fmaf(gw[j], v[i][j], t);
        }
        if (h != nullptr) store_vec<RDT, VEC>(h, m * K + k, v[i]);
      }
    }
    if (y == nullptr && xq == nullptr) continue;
    normalise<VEC, NI>(v, p.pre, p.pre_eps, K, sum);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float w[VEC], c[VEC];
        if constexpr (kHold) {
          slots.get(1, i, w);
          if constexpr (BIAS) slots.get(3, i, c);
        } else {
          load_col<VEC>(p.pre_w, k, 1.0f, w);
          if constexpr (BIAS) load_col<VEC>(p.pre_b, k, 0.0f, c);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = BIAS ? fmaf(v[i][j], w[j], c[j]) : __fmul_rn(v[i][j], w[j]);
          amax = fmaxf(amax, fabsf(v[i][j]));
        }
        if (y != nullptr) store_vec_dt<VEC>(y, ydt, m * K + k, v[i]);
      }
    }
    if (xq == nullptr) continue;
    const float s = fmaxf(sum.max(amax), 1e-6f);
    const float c127 = __fdiv_rn(127.0f, s);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        int q[VEC];
        quant_act_fast_n<VEC>(v[i], s, c127, q);
        if constexpr (VEC == 8)
          *reinterpret_cast<uint2*>(xq + m * K + k) = make_uint2(pack4(q), pack4(q + 4));
        else
          xq[m * K + k] = static_cast<int8_t>(q[0]);
      }
    }
    if (threadIdx.x == 0) scale[m] = s;
  }
}

// ---- forward, rows too long for registers ----------------------------------------
// Each sum is a pass over the row (L2 holds it between passes); h is formed
// again in every pass, so it needs no storage.
template <int BDT, int RDT>
__global__ void __launch_bounds__(kNormLongThreads)
    residual_norm_long_kernel(const NormParams p_arg, const void* __restrict__ b, const void* __restrict__ r, int64_t M,
                              int64_t K, void* __restrict__ h, void* __restrict__ y, int ydt, int8_t* __restrict__ xq,
                              float* __restrict__ scale) {
  pdl_enter(b, r, h, y, xq, scale);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float4 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  const float fk = static_cast<float>(K);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
    float mean1 = 0.0f, r1 = 1.0f, mean2 = 0.0f, r2 = 1.0f;
    auto bv = [&](int64_t k) { return load_elem<BDT>(b, m * K + k); };
    auto hv = [&](int64_t k) {
      float w, c, g;
      load_col<1>(p.post_w, k, 1.0f, &w);
      load_col<1>(p.post_b, k, 0.0f, &c);
      load_col<1>(gate, k, 1.0f, &g);
      return p.res_scale * load_elem<RDT>(r, m * K + k) + p.branch_scale * g * ((bv(k) - mean1) * r1 * w + c);
    };
    auto yv = [&](float hk, int64_t k) {
      float w, c;
      load_col<1>(p.pre_w, k, 1.0f, &w);
      load_col<1>(p.pre_b, k, 0.0f, &c);
      return (hk - mean2) * r2 * w + c;
    };
    // sum over the row of f(k); two runs of neighbouring partial sums per thread
    auto total = [&](auto f) {
      float s0 = 0.0f, s1 = 0.0f;
      for (int64_t k = threadIdx.x; k < K; k += 2 * blockDim.x) {
        s0 += f(k);
        if (k + blockDim.x < K) s1 += f(k + blockDim.x);
      }
      return sum.one(s0 + s1);
    };
    if (p.post == BL_NORM_LAYER) mean1 = total(bv) / fk;
    if (p.post != BL_NORM_NONE)
      r1 = inv_dev(total([&](int64_t k) { const float d = bv(k) - mean1; return d * d; }), K, p.post_eps);
    if (y != nullptr || xq != nullptr) {
      if (p.pre == BL_NORM_LAYER) mean2 = total(hv) / fk;
      if (p.pre != BL_NORM_NONE)
        r2 = inv_dev(total([&](int64_t k) { const float d = hv(k) - mean2; return d * d; }), K, p.pre_eps);
    }
    float s = 1.0f, c127 = 127.0f;
    if (xq != nullptr) {
      float amax = 0.0f;
      for (int64_t k = threadIdx.x; k < K; k += blockDim.x) amax = fmaxf(amax, fabsf(yv(hv(k), k)));
      s = fmaxf(sum.max(amax), 1e-6f);
      c127 = __fdiv_rn(127.0f, s);
      if (threadIdx.x == 0) scale[m] = s;
    }
    for (int64_t k = threadIdx.x; k < K; k += blockDim.x) {  // h may replace r: the last pass writes it
      const float hk = hv(k);
      const float yk = yv(hk, k);
      if (h != nullptr) store_vec<RDT, 1>(h, m * K + k, &hk);
      if (y != nullptr) store_vec_dt<1>(y, ydt, m * K + k, &yk);
      if (xq != nullptr) xq[m * K + k] = static_cast<int8_t>(quant_act_fast(yk, s, c127));
    }
  }
}

// ---- backward, the row in registers -----------------------------------------------
// Block c takes rows [c rows_per, (c + 1) rows_per).  part: [4][gridDim.x][K]
// (dw2, db2, dw1, db1).  A run of a block's rows with one gate row g keeps
//   A = sum dh n1,  B = sum dh,
// from which dgate = bs (w1 A + b1 B), dw1 += bs g A, db1 += bs g B.  dgate of a
// run that is all of its gate row goes out at once, else to gpart row (block +
// gate row) for the sums in order.  Slots: 0 gw = bs gate w1, 1 w2.  Up to 8
// values per thread the next row is in flight during this one, the running sums
// stay in registers and dw1, db1 in slots 2, 3; with 24 values slots 2 .. 5 hold
// the running sums (dw2, A, db2, B) and dw1, db1 go to part as they grow.
__host__ __device__ __forceinline__ bool gate_row_whole(int64_t g, int64_t gate_rows, int64_t M, int64_t m0,
                                                        int64_t m1) {
  const int64_t end = (g + 1) * gate_rows < M ? (g + 1) * gate_rows : M;
  return g * gate_rows >= m0 && end <= m1;
}

constexpr int grad_slots(int values, bool bias) { return values <= 8 ? (bias ? 4 : 3) : (bias ? 6 : 4); }

template <int BDT, int RDT, int VEC, int NI, bool BIAS>
__global__ void __launch_bounds__(grad_max_threads(VEC, NI))
    residual_norm_grad_kernel(const NormParams p_arg, const void* __restrict__ dy, int dydt,
                              const void* __restrict__ dh, const void* __restrict__ b, const void* __restrict__ h,
                              int64_t M, int64_t K, int64_t rows_per, void* __restrict__ dr, void* __restrict__ db,
                              float* __restrict__ part, float* __restrict__ gpart, float* __restrict__ dgate) {
  pdl_enter(dy, dh, b, h, dr, db, part, gpart, dgate);
  const NormParams p = params_after_wait(p_arg);
  extern __shared__ __align__(16) float slot_mem[];
  Slots<VEC, NI> slots{slot_mem};
  __shared__ float4 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  const float fk = static_cast<float>(K);
  const int64_t m0 = blockIdx.x * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  constexpr bool kInReg = VEC * NI <= 8;
  constexpr int kRegs = kInReg ? NI : 1;
  constexpr int kAcc = 2;  // first slot of the running sums
  const int64_t plane = static_cast<int64_t>(gridDim.x) * K;
  bool grown = false;  // part holds dw1, db1 of earlier runs
  float aw2[kRegs][VEC], aA[kRegs][VEC];
  float ab2[BIAS ? kRegs : 1][VEC], aB[BIAS ? kRegs : 1][VEC];
  Raw<BDT, VEC> rb[NI];
  Raw<RDT, VEC> rh[NI], rg[NI];
  float gy[NI][VEC];
  auto fetch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      rg[i].zero();
      if (m < m1 && k < K) {
        rb[i].load(b, m * K + k);
        rh[i].load(h, m * K + k);
        load_vec_dt<VEC>(dy, dydt, m * K + k, gy[i]);
        if (dh != nullptr) rg[i].load(dh, m * K + k);
      } else {
        rb[i].zero();
        rh[i].zero();
#pragma unroll
        for (int j = 0; j < VEC; ++j) gy[i][j] = 0.0f;
      }
    }
  };
  auto gate_row = [&](int64_t m) { return p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K; };
  auto hold_branch = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float t[VEC];
        branch_factor<VEC>(p, gate_row(m), k, t);
        slots.put(0, i, t);
      }
    }
  };
  // the sums of a run that ends with token m: into dw1, db1 (slots) and its gate row
  auto flush = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float g[VEC], w[VEC], c[VEC], t[VEC];
        float sA[VEC], sB[VEC];
        const float zero[VEC] = {};
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          sA[j] = aA[kInReg ? i : 0][j];
          sB[j] = BIAS ? aB[BIAS && kInReg ? i : 0][j] : 0.0f;
        }
        if constexpr (!kInReg) {
          slots.get(kAcc + 1, i, sA);
          slots.put(kAcc + 1, i, zero);
          if constexpr (BIAS) {
            slots.get(kAcc + 3, i, sB);
            slots.put(kAcc + 3, i, zero);
          }
        }
        load_col<VEC>(gate_row(m), k, 1.0f, g);
        auto grow = [&](int slot, int vec, const float* a) {
          float* at = kInReg || part == nullptr ? nullptr : part + vec * plane + blockIdx.x * K + k;
          if constexpr (kInReg) {
            slots.get(slot, i, t);
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) t[j] = 0.0f;
            if (grown && at != nullptr) load_vec<BL_F32, VEC>(at, 0, t);
          }
#pragma unroll
          for (int j = 0; j < VEC; ++j) t[j] = fmaf(__fmul_rn(p.branch_scale, g[j]), a[j], t[j]);
          if constexpr (kInReg)
            slots.put(slot, i, t);
          else if (at != nullptr)
            store_vec<BL_F32, VEC>(at, 0, t);
        };
        grow(2, 2, sA);
        if constexpr (BIAS) grow(3, 3, sB);
        if (dgate != nullptr) {
          load_col<VEC>(p.post_w, k, 1.0f, w);
          if constexpr (BIAS) load_col<VEC>(p.post_b, k, 0.0f, c);
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            t[j] = __fmul_rn(w[j], sA[j]);
            if constexpr (BIAS) t[j] = fmaf(c[j], sB[j], t[j]);
            t[j] = __fmul_rn(p.branch_scale, t[j]);
          }
          const int64_t row = m / p.gate_rows;
          const bool whole = gate_row_whole(row, p.gate_rows, M, m0, m1);
          float* dst = whole ? dgate + row * K + k : gpart + (blockIdx.x + row) * K + k;
          if (VEC == 8 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
            store_vec<BL_F32, VEC>(dst, 0, t);
          } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) dst[j] = t[j];
          }
        }
      }
      if constexpr (kInReg) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          aA[i][j] = 0.0f;
          if constexpr (BIAS) aB[i][j] = 0.0f;
        }
      }
    }
    grown = true;
  };
  fetch(m0);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t k = col0<VEC>(i);
    const float zero[VEC] = {};
#pragma unroll
    for (int v = 2; v < grad_slots(VEC * NI, BIAS); ++v) slots.put(v, i, zero);
    if constexpr (kInReg) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        aw2[i][j] = aA[i][j] = 0.0f;
        if constexpr (BIAS) ab2[i][j] = aB[i][j] = 0.0f;
      }
    }
    if (k < K) {
      float t[VEC];
      load_col<VEC>(p.pre_w, k, 1.0f, t);
      slots.put(1, i, t);
    }
  }
  hold_branch(m0);
  int64_t g_next = p.gate == nullptr ? M : (m0 / p.gate_rows + 1) * p.gate_rows;
  for (int64_t m = m0; m < m1; ++m) {
    float n1[NI][VEC], n2[NI][VEC], d2[NI][VEC], d[NI][VEC], dyv[NI][VEC];
    if constexpr (!kInReg) {
      if (m != m0) fetch(m);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      rb[i].get(n1[i]);
      rh[i].get(n2[i]);
      rg[i].get(d[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) dyv[i][j] = gy[i][j];
    }
    if constexpr (kInReg) fetch(m + 1);
    if (m >= g_next) {
      flush(m - 1);
      hold_branch(m);
      g_next += p.gate_rows;
    }
    if (p.post == BL_NORM_LAYER || p.pre == BL_NORM_LAYER) {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          s1 += n1[i][j];
          s2 += n2[i][j];
        }
      const float2 t = sum.two(s1, s2);
      const float mean1 = p.post == BL_NORM_LAYER ? t.x / fk : 0.0f;
      const float mean2 = p.pre == BL_NORM_LAYER ? t.y / fk : 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          n1[i][j] = col0<VEC>(i) < K ? n1[i][j] - mean1 : 0.0f;
          n2[i][j] = col0<VEC>(i) < K ? n2[i][j] - mean2 : 0.0f;
        }
    }
    // both deviations, and the sums through the norm before the next block
    float q1 = 0.0f, q2 = 0.0f, sd = 0.0f, sq = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      float w[VEC];
      if (k < K) slots.get(1, i, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        d2[i][j] = k < K ? __fmul_rn(dyv[i][j], w[j]) : 0.0f;
        q1 = fmaf(n1[i][j], n1[i][j], q1);
        q2 = fmaf(n2[i][j], n2[i][j], q2);
        sd += d2[i][j];
        sq = fmaf(d2[i][j], n2[i][j], sq);
      }
    }
    const float4 t = sum.four(q1, q2, sd, sq);
    const float r1 = p.post == BL_NORM_NONE ? 1.0f : inv_dev(t.x, K, p.post_eps);
    const float r2 = p.pre == BL_NORM_NONE ? 1.0f : inv_dev(t.y, K, p.pre_eps);
    const float s = p.pre == BL_NORM_LAYER ? t.z / fk : 0.0f;
    const float q = p.pre == BL_NORM_NONE ? 0.0f : __fmul_rn(r2, t.w) / fk;
    float s1 = 0.0f, p1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float gw[VEC], out[VEC];
        slots.get(0, i, gw);
        float sw2[VEC], sA[VEC], sb2[VEC], sB[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          sw2[j] = aw2[kInReg ? i : 0][j];
          sA[j] = aA[kInReg ? i : 0][j];
          sb2[j] = ab2[BIAS && kInReg ? i : 0][j];
          sB[j] = aB[BIAS && kInReg ? i : 0][j];
        }
        if constexpr (!kInReg) {
          slots.get(kAcc, i, sw2);
          slots.get(kAcc + 1, i, sA);
          if constexpr (BIAS) {
            slots.get(kAcc + 2, i, sb2);
            slots.get(kAcc + 3, i, sB);
          }
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float u2 = __fmul_rn(n2[i][j], r2);
          n1[i][j] = __fmul_rn(n1[i][j], r1);
          d[i][j] = fmaf(r2, fmaf(-u2, q, __fsub_rn(d2[i][j], s)), d[i][j]);
          out[j] = __fmul_rn(p.res_scale, d[i][j]);
          sw2[j] = fmaf(dyv[i][j], u2, sw2[j]);
          sA[j] = fmaf(d[i][j], n1[i][j], sA[j]);
          if constexpr (BIAS) {
            sb2[j] += dyv[i][j];
            sB[j] += d[i][j];
          }
          d2[i][j] = __fmul_rn(gw[j], d[i][j]);  // dn1
          s1 += d2[i][j];
          p1 = fmaf(d2[i][j], n1[i][j], p1);
        }
        if constexpr (kInReg) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            aw2[i][j] = sw2[j];
            aA[i][j] = sA[j];
            if constexpr (BIAS) {
              ab2[i][j] = sb2[j];
              aB[i][j] = sB[j];
            }
          }
        } else {
          slots.put(kAcc, i, sw2);
          slots.put(kAcc + 1, i, sA);
          if constexpr (BIAS) {
            slots.put(kAcc + 2, i, sb2);
            slots.put(kAcc + 3, i, sB);
          }
        }
        if (dr != nullptr) store_vec<RDT, VEC>(dr, m * K + k, out);
      }
    }
    if (db != nullptr) {
      if (p.post == BL_NORM_NONE) {
        s1 = p1 = 0.0f;
      } else {
        const float2 t1 = sum.two(s1, p1);
        s1 = p.post == BL_NORM_LAYER ? t1.x / fk : 0.0f;
        p1 = t1.y / fk;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int64_t k = col0<VEC>(i);
        if (k < K) {
          float out[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            out[j] = __fmul_rn(r1, fmaf(-n1[i][j], p1, __fsub_rn(d2[i][j], s1)));
          store_vec<BDT, VEC>(db, m * K + k, out);
        }
      }
    }
  }
  flush(m1 - 1);
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t k = col0<VEC>(i), o = static_cast<int64_t>(blockIdx.x) * K + k;
    if (k < K) {
      float t[VEC];
      auto sums = [&](const float* in_reg, int slot) {
        if constexpr (kInReg) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) t[j] = in_reg[j];
        } else {
          slots.get(slot, i, t);
        }
      };
      sums(aw2[kInReg ? i : 0], kAcc);
      store_vec<BL_F32, VEC>(part, o, t);
      if constexpr (BIAS) {
        sums(ab2[BIAS && kInReg ? i : 0], kAcc + 2);
        store_vec<BL_F32, VEC>(part, o + plane, t);
      }
      if constexpr (kInReg) {
        slots.get(2, i, t);
        store_vec<BL_F32, VEC>(part, o + 2 * plane, t);
        if constexpr (BIAS) {
          slots.get(3, i, t);
          store_vec<BL_F32, VEC>(part, o + 3 * plane, t);
        }
      }
    }
  }
}

// ---- backward, rows too long for registers -------------------------------------------
// The row statistics first: stats[m] = mean1, r1, mean2, r2, mean dn2,
// mean(dn2 n2), mean dn1, mean(dn1 n1); then one pass by columns.
struct GradRow {
  float mean1, r1, mean2, r2, s, q, s1, q1;
};

template <int BDT, int RDT>
struct GradElem {
  float n1, n2, gy, dhk, bd, w1, u;  // gy = dy (before w2)
  __device__ __forceinline__ void at(const NormParams& p, const GradRow& t, const void* dy, int dydt, const void* dh,
                                     const void* b, const void* h, int64_t e, int64_t k) {
    float w2, c1;
    load_col<1>(p.pre_w, k, 1.0f, &w2);
    load_col<1>(p.post_w, k, 1.0f, &w1);
    load_col<1>(p.post_b, k, 0.0f, &c1);
    n1 = (load_elem<BDT>(b, e) - t.mean1) * t.r1;
    n2 = (load_elem<RDT>(h, e) - t.mean2) * t.r2;
    load_vec_dt<1>(dy, dydt, e, &gy);
    dhk = (dh != nullptr ? load_elem<RDT>(dh, e) : 0.0f) + t.r2 * (gy * w2 - t.s - n2 * t.q);
    bd = p.branch_scale * dhk;
    u = n1 * w1 + c1;
  }
};

template <int BDT, int RDT>
__global__ void __launch_bounds__(kNormLongThreads)
    residual_norm_grad_stats_kernel(const NormParams p_arg, const void* __restrict__ dy, int dydt,
                                    const void* __restrict__ dh, const void* __restrict__ b,
                                    const void* __restrict__ h, int64_t M, int64_t K, GradRow* __restrict__ stats) {
  pdl_enter(dy, dh, b, h, stats);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float4 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  const float fk = static_cast<float>(K);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
    GradRow t{0.0f, 1.0f, 0.0f, 1.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    auto total = [&](auto f) {
      float a = 0.0f, c = 0.0f;
      for (int64_t k = threadIdx.x; k < K; k += blockDim.x) f(k, a, c);
      return sum.two(a, c);
    };
    auto bv = [&](int64_t k) { return load_elem<BDT>(b, m * K + k); };
    auto hv = [&](int64_t k) { return load_elem<RDT>(h, m * K + k); };
    const float2 mean = total([&](int64_t k, float& a, float& c) {
      a += bv(k);
      c += hv(k);
    });
    if (p.post == BL_NORM_LAYER) t.mean1 = mean.x / fk;
    if (p.pre == BL_NORM_LAYER) t.mean2 = mean.y / fk;
    const float2 sq = total([&](int64_t k, float& a, float& c) {
      const float d1 = bv(k) - t.mean1, d2 = hv(k) - t.mean2;
      a += d1 * d1;
      c += d2 * d2;
    });
    if (p.post != BL_NORM_NONE) t.r1 = inv_dev(sq.x, K, p.post_eps);
    if (p.pre != BL_NORM_NONE) {
      t.r2 = inv_dev(sq.y, K, p.pre_eps);
      const float2 v = total([&](int64_t k, float& a, float& c) {
        float g, w2;
        load_vec_dt<1>(dy, dydt, m * K + k, &g);
        load_col<1>(p.pre_w, k, 1.0f, &w2);
        a += g * w2;
        c += g * w2 * (hv(k) - t.mean2) * t.r2;
      });
      t.s = p.pre == BL_NORM_LAYER ? v.x / fk : 0.0f;
      t.q = v.y / fk;
    }
    if (p.post != BL_NORM_NONE) {
      const float2 v = total([&](int64_t k, float& a, float& c) {
        GradElem<BDT, RDT> e;
        float g;
        e.at(p, t, dy, dydt, dh, b, h, m * K + k, k);
        load_col<1>(gate, k, 1.0f, &g);
        const float dn1 = e.bd * g * e.w1;
        a += dn1;
        c += dn1 * e.n1;
      });
      t.s1 = p.post == BL_NORM_LAYER ? v.x / fk : 0.0f;
      t.q1 = v.y / fk;
    }
    if (threadIdx.x == 0) stats[m] = t;
  }
}

constexpr int kGradColThreads = 256;

template <int BDT, int RDT>
__global__ void __launch_bounds__(kGradColThreads)
    residual_norm_grad_cols_kernel(const NormParams p_arg, const void* __restrict__ dy, int dydt,
                                   const void* __restrict__ dh, const void* __restrict__ b,
                                   const void* __restrict__ h, int64_t M, int64_t K, int64_t rows_per,
                                   const GradRow* __restrict__ stats, void* __restrict__ dr, void* __restrict__ db,
                                   float* __restrict__ part, float* __restrict__ gpart, float* __restrict__ dgate) {
  pdl_enter(dy, dh, b, h, stats, dr, db, part, gpart, dgate);
  const NormParams p = params_after_wait(p_arg);
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kGradColThreads + threadIdx.x, c = blockIdx.y;
  if (k >= K) return;
  const int64_t m0 = c * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  float aw2 = 0.0f, ab2 = 0.0f, aw1 = 0.0f, ab1 = 0.0f, ag = 0.0f;
  for (int64_t m = m0; m < m1; ++m) {
    const float4* sp = reinterpret_cast<const float4*>(stats + m);
    const float4 t0 = __ldcg(sp), t1 = __ldcg(sp + 1);
    const GradRow t{t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
    GradElem<BDT, RDT> e;
    float g;
    e.at(p, t, dy, dydt, dh, b, h, m * K + k, k);
    load_col<1>(p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K, k, 1.0f, &g);
    const float du = e.bd * g, dn1 = du * e.w1;
    aw2 += e.gy * e.n2;
    ab2 += e.gy;
    aw1 += du * e.n1;
    ab1 += du;
    ag += e.bd * e.u;
    const float o1 = p.res_scale * e.dhk, o2 = t.r1 * (dn1 - t.s1 - e.n1 * t.q1);
    if (dr != nullptr) store_vec<RDT, 1>(dr, m * K + k, &o1);
    if (db != nullptr) store_vec<BDT, 1>(db, m * K + k, &o2);
    if (dgate != nullptr && (m + 1 == m1 || (m + 1) % p.gate_rows == 0)) {
      const int64_t row = m / p.gate_rows;
      if (gate_row_whole(row, p.gate_rows, M, m0, m1))
        dgate[row * K + k] = ag;
      else
        gpart[(c + row) * K + k] = ag;
      ag = 0.0f;
    }
  }
  if (part == nullptr) return;
  const int64_t plane = static_cast<int64_t>(gridDim.y) * K;
  float* o = part + c * K + k;
  o[0] = aw2;
  o[plane] = ab2;
  o[2 * plane] = aw1;
  o[3 * plane] = ab1;
}

// The column sums: vector v < 4 of the blocks' partials, or (v >= 4) gate row
// v - 4 from the runs of its rows (a gate row within one block is done already).
// 16 threads share a column, each adding every 16th row in order; their sums
// meet in a fixed order.
constexpr int kSumCols = 32, kSumRows = 16;
__global__ void __launch_bounds__(kSumCols* kSumRows)
    residual_norm_grad_sum_kernel(const float* __restrict__ part, const float* __restrict__ gpart, int64_t blocks,
                                  int64_t rows_per, int64_t M, int64_t K, int64_t gate_rows, float* __restrict__ dw2,
                                  float* __restrict__ db2, float* __restrict__ dw1, float* __restrict__ db1,
                                  float* __restrict__ dgate) {
  pdl_enter(part, gpart, dw2, db2, dw1, db1, dgate);
  __shared__ float sums[kSumRows][kSumCols + 1];
  const int tx = threadIdx.x % kSumCols, ty = threadIdx.x / kSumCols;
  const int64_t k = static_cast<int64_t>(blockIdx.x) * kSumCols + tx;
  const int64_t gates = dgate == nullptr ? 0 : (M + gate_rows - 1) / gate_rows;
  for (int64_t v = blockIdx.y; v < 4 + gates; v += gridDim.y) {
    float* out;
    const float* src;
    int64_t c0 = 0, c1 = blocks;
    if (v < 4) {
      out = v == 0 ? dw2 : v == 1 ? db2 : v == 2 ? dw1 : db1;
      src = part + v * blocks * K;
      if (out == nullptr) continue;
    } else {
      const int64_t g = v - 4, last = (g + 1) * gate_rows < M ? (g + 1) * gate_rows - 1 : M - 1;
      c0 = g * gate_rows / rows_per;
      c1 = last / rows_per + 1;
      if (c1 == c0 + 1) continue;
      out = dgate + g * K;
      src = gpart + g * K;
    }
    float s = 0.0f;
    if (k < K) {
#pragma unroll 8
      for (int64_t c = c0 + ty; c < c1; c += kSumRows) s += __ldcg(src + c * K + k);
    }
    sums[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && k < K) {
      s = 0.0f;
#pragma unroll
      for (int r = 0; r < kSumRows; ++r) s += sums[r][tx];
      out[k] = s;
    }
    __syncthreads();
  }
}

// Threads of a block for a row of K columns in NI chunks of VEC per thread.
int row_threads(int64_t K, int vec, int ni) {
  const int64_t per = static_cast<int64_t>(vec) * ni;
  return static_cast<int>(((K + per - 1) / per + 31) / 32 * 32);
}

// Blocks that stay on an SM: some 1280 threads (the register form's 48 or so
// registers per thread; more blocks only add turns of the column vectors).
unsigned resident_grid(int threads, int64_t rows) {
  const int64_t per = 1280 / threads, cap = device_sms() * (per < 1 ? 1 : (per > 16 ? 16 : per));
  return static_cast<unsigned>(rows < cap ? rows : cap);
}

// Dynamic shared memory above the 48 KB that need no opt-in.
template <typename Kern>
cudaError_t allow_smem(Kern kern, size_t bytes) {
  return bytes <= 48 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(bytes));
}

template <int BDT, int RDT, int VEC, int NI>
cudaError_t launch_fwd_row(const NormParams& p, const void* b, const void* r, int64_t M, int64_t K, void* h, void* y,
                           int ydt, int8_t* xq, float* scale, cudaStream_t st) {
  const bool bias = p.post_b != nullptr || p.pre_b != nullptr;
  auto kern = bias ? residual_norm_kernel<BDT, RDT, VEC, NI, true> : residual_norm_kernel<BDT, RDT, VEC, NI, false>;
  const int t = row_threads(K, VEC, NI);
  const size_t smem = norm_hold(VEC * NI) ? static_cast<size_t>(bias ? 4 : 2) * t * VEC * NI * sizeof(float) : 0;
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, resident_grid(t, M), t, smem, st, p, b, r, M, K, h, y, ydt, xq, scale);
}

template <int BDT, int RDT>
cudaError_t launch_fwd(const NormParams& p, const void* b, const void* r, int64_t M, int64_t K, void* h, void* y,
                       int ydt, int8_t* xq, float* scale, cudaStream_t st) {
  const bool wide = K % 8 == 0 && (reinterpret_cast<uintptr_t>(xq) & 7) == 0;
#define BL_NF(VEC, NI)                                               \
  if (K <= static_cast<int64_t>(norm_max_threads(VEC, NI)) * (VEC) * (NI)) \
  return launch_fwd_row<BDT, RDT, VEC, NI>(p, b, r, M, K, h, y, ydt, xq, scale, st)
  if (wide) {
    BL_NF(8, 1);
    BL_NF(8, 2);
    BL_NF(8, 4);
  } else {
    BL_NF(1, 4);
    BL_NF(1, 16);
  }
#undef BL_NF
  auto kern = residual_norm_long_kernel<BDT, RDT>;
  return launch_pdl(kern, resident_grid(kNormLongThreads, M), kNormLongThreads, 0, st, p, b, r, M, K, h, y, ydt, xq,
                    scale);
}

template <int VEC, int NI>
size_t grad_smem(int64_t K, bool bias) {
  return static_cast<size_t>(grad_slots(VEC * NI, bias)) * row_threads(K, VEC, NI) * VEC * NI * sizeof(float);
}

template <int BDT, int RDT, int VEC, int NI>
cudaError_t launch_bwd_row(const NormParams& p, const void* dy, int dydt, const void* dh, const void* b, const void* h,
                           int64_t M, int64_t K, void* dr, void* db, bool bias, int64_t blocks, int64_t rows_per,
                           float* part, float* gpart, float* dgate, cudaStream_t st) {
  auto kern = bias ? residual_norm_grad_kernel<BDT, RDT, VEC, NI, true>
                   : residual_norm_grad_kernel<BDT, RDT, VEC, NI, false>;
  const int t = row_threads(K, VEC, NI);
  const size_t smem = grad_smem<VEC, NI>(K, bias);
  const cudaError_t e = allow_smem(kern, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, static_cast<unsigned>(blocks), t, smem, st, p, dy, dydt, dh, b, h, M, K, rows_per, dr, db,
                    part, gpart, dgate);
}

template <int BDT, int RDT>
cudaError_t launch_bwd(const NormParams& p, const void* dy, int dydt, const void* dh, const void* b, const void* h,
                       int64_t M, int64_t K, void* dr, void* db, bool bias, int64_t blocks, int64_t rows_per,
                       float* part, float* gpart, float* dgate, void* stats, cudaStream_t st) {
#define BL_NB(VEC, NI)                                                                                              \
  if (K <= static_cast<int64_t>(grad_max_threads(VEC, NI)) * (VEC) * (NI) &&                                   \
      grad_smem<VEC, NI>(K, true) <= kGradSmemBudget)                                                               \
  return launch_bwd_row<BDT, RDT, VEC, NI>(p, dy, dydt, dh, b, h, M, K, dr, db, bias, blocks, rows_per, part, gpart, \
                                           dgate, st)
  if (K % 8 == 0) {
    BL_NB(8, 1);
    BL_NB(8, 3);
  } else {
    BL_NB(1, 4);
    BL_NB(1, 8);
  }
#undef BL_NB
  GradRow* rows = static_cast<GradRow*>(stats);
  auto ks = residual_norm_grad_stats_kernel<BDT, RDT>;
  cudaError_t e = launch_pdl(ks, resident_grid(kNormLongThreads, M), kNormLongThreads, 0, st, p, dy, dydt, dh, b, h, M,
                             K, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(residual_norm_grad_cols_kernel<BDT, RDT>,
                    dim3(static_cast<unsigned>((K + kGradColThreads - 1) / kGradColThreads),
                         static_cast<unsigned>(blocks)),
                    kGradColThreads, 0, st, p, dy, dydt, dh, b, h, M, K, rows_per,
                    static_cast<const GradRow*>(rows), dr, db, part, gpart, dgate);
}

}  // namespace

// Row blocks of the backward (partial sums): kGradBlocks per SM.
int64_t norm_grad_blocks(int64_t M) {
  const int64_t most = kGradBlocks * device_sms();
  const int64_t rows_per = (M + most - 1) / most;
  return rows_per > 0 ? (M + rows_per - 1) / rows_per : 1;
}

cudaError_t launch_residual_norm(const NormParams& p, const void* b, int bdt, const void* r, int rdt, int64_t M,
                                 int64_t K, void* h, void* y, int ydt, int8_t* xq, float* scale, cudaStream_t st) {
  cudaError_t e;
  if (bdt == BL_F32)
    e = rdt == BL_F32 ? launch_fwd<BL_F32, BL_F32>(p, b, r, M, K, h, y, ydt, xq, scale, st)
                      : launch_fwd<BL_F32, BL_BF16>(p, b, r, M, K, h, y, ydt, xq, scale, st);
  else
    e = rdt == BL_F32 ? launch_fwd<BL_BF16, BL_F32>(p, b, r, M, K, h, y, ydt, xq, scale, st)
                      : launch_fwd<BL_BF16, BL_BF16>(p, b, r, M, K, h, y, ydt, xq, scale, st);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_residual_norm_grad(const NormParams& p, const void* dy, int dydt, const void* dh, const void* b,
                                      int bdt, const void* h, int rdt, int64_t M, int64_t K, void* dr, void* db,
                                      float* dw1, float* db1, float* dgate, float* dw2, float* db2, float* part,
                                      float* gpart, void* stats, cudaStream_t st) {
  const int64_t blocks = norm_grad_blocks(M);
  const int64_t rows_per = (M + blocks - 1) / blocks;
  const bool sums = db1 != nullptr || db2 != nullptr;
  const bool bias = sums || (dgate != nullptr && p.post_b != nullptr);  // dgate takes sum dh with a bias
  float* ps = sums || dw1 != nullptr || dw2 != nullptr ? part : nullptr;
  cudaError_t e;
#define BL_NB(BDT, RDT) \
  e = launch_bwd<BDT, RDT>(p, dy, dydt, dh, b, h, M, K, dr, db, bias, blocks, rows_per, ps, gpart, dgate, stats, st)
  if (bdt == BL_F32) {
    if (rdt == BL_F32)
      BL_NB(BL_F32, BL_F32);
    else
      BL_NB(BL_F32, BL_BF16);
  } else {
    if (rdt == BL_F32)
      BL_NB(BL_BF16, BL_F32);
    else
      BL_NB(BL_BF16, BL_BF16);
  }
#undef BL_NB
  if (e != cudaSuccess) return e;
  // gate rows that lie in one block each need no further sum
  const bool runs = dgate != nullptr && !(rows_per % p.gate_rows == 0);
  if (ps != nullptr || runs) {
    const int64_t rows = 4 + (runs ? (M + p.gate_rows - 1) / p.gate_rows : 0);
    e = launch_pdl(residual_norm_grad_sum_kernel,
                   dim3(static_cast<unsigned>((K + kSumCols - 1) / kSumCols),
                        static_cast<unsigned>(rows < 1024 ? rows : 1024)),
                   kSumCols * kSumRows, 0, st, static_cast<const float*>(part), static_cast<const float*>(gpart),
                   blocks, rows_per, M, K, p.gate_rows > 0 ? p.gate_rows : 1, dw2, db2, dw1, db1,
                   runs ? dgate : nullptr);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
