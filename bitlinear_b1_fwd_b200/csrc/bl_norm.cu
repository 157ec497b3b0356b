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
// 4096 x 3200 bf16, RMS + RMS: forward 23 us with bf16 y (floor 16), gradient 49 us
// (floor 24: 13 warps an SM, latency-bound); 12000 x 1001, one column per lane, 46
// and 74 us (floors 15 and 22: instructions).
#include <atomic>
#include <type_traits>

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
  } else if (VEC > 1 && (reinterpret_cast<uintptr_t>(p + k) & 15) == 0) {
    load_vec<BL_F32, VEC>(p, k, v);
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = __ldcg(p + k + j);
  }
}

// 1 / sqrt of the mean square plus eps.  Means are products with rk = 1 / K and
// the root is rsqrtf (within 2 ulp): the IEEE divides and roots, in every thread
// of a block for each row, were a quarter of the instructions.
__device__ __forceinline__ float inv_dev(float sumsq, float rk, float eps) { return rsqrtf(fmaf(sumsq, rk, eps)); }

// Column of value j of a thread's chunk i (VEC = 8: chunks of 8 neighbouring
// columns; VEC = 1: neighbouring threads hold neighbouring columns).
template <int VEC>
__device__ __forceinline__ int col0(int i) {  // (K <= 2^20)
  return static_cast<int>((i * blockDim.x + threadIdx.x) * VEC);
}

// Row m of an array [.][K]: 64-bit arithmetic once per row and array, 32-bit
// columns within (per access it was a third of the instructions of narrow rows).
template <typename P>
__device__ __forceinline__ P* row_of(P* p, int dt, int64_t m, int64_t K) {
  using Byte = typename std::conditional<std::is_const<P>::value, const uint8_t, uint8_t>::type;
  return reinterpret_cast<Byte*>(p) + m * K * (dt == BL_F32 ? 4 : 2);
}

// Per-column vectors folded once per block: vector v of chunk i of this thread,
// in shared slots that no other thread touches (16-byte accesses of
// neighbouring threads are neighbours).
template <int VEC, int NI>
struct Slots {
  float* s;
  __device__ __forceinline__ void put(int v, int i, const float* x) {
    if constexpr (VEC == 1) {
      s[(v * NI + i) * blockDim.x + threadIdx.x] = x[0];
    } else {
      float4* q = reinterpret_cast<float4*>(s) + (v * NI + i) * (VEC / 4) * blockDim.x + threadIdx.x;
#pragma unroll
      for (int c = 0; c < VEC / 4; ++c) q[c * blockDim.x] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    }
  }
  __device__ __forceinline__ void put(int v, int i, const Vals<VEC>& x) {
    float f[VEC];
    x.get(f);
    put(v, i, f);
  }
  __device__ __forceinline__ Vals<VEC> get(int v, int i) const {
    float f[VEC];
    if constexpr (VEC == 1) {
      f[0] = s[(v * NI + i) * blockDim.x + threadIdx.x];
    } else {
      const float4* q = reinterpret_cast<const float4*>(s) + (v * NI + i) * (VEC / 4) * blockDim.x + threadIdx.x;
#pragma unroll
      for (int c = 0; c < VEC / 4; ++c) {
        const float4 a = q[c * blockDim.x];
        f[4 * c] = a.x; f[4 * c + 1] = a.y; f[4 * c + 2] = a.z; f[4 * c + 3] = a.w;
      }
    }
    Vals<VEC> r;
    r.set(f);
    return r;
  }
};
template <int VEC>
__device__ __forceinline__ Vals<VEC> col_vals(const float* p, int64_t k, float c) {
  float f[VEC];
  load_col<VEC>(p, k, c, f);
  Vals<VEC> r;
  r.set(f);
  return r;
}

// bs gate w1 and bs gate b1: the branch's factor and offset, h = rs r + gw n1 + gb
template <int VEC>
__device__ __forceinline__ Vals<VEC> branch_factor(const NormParams& p, const float* gate, int64_t k) {
  return mul(mul(splat<VEC>(p.branch_scale), col_vals<VEC>(gate, k, 1.0f)), col_vals<VEC>(p.post_w, k, 1.0f));
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> branch_offset(const NormParams& p, const float* gate, int64_t k) {
  return mul(mul(splat<VEC>(p.branch_scale), col_vals<VEC>(gate, k, 1.0f)), col_vals<VEC>(p.post_b, k, 0.0f));
}

template <int VEC, int NI>
__device__ __forceinline__ float sum_of(const Vals<VEC> (&v)[NI]) {
  Vals<VEC> s = v[0];
#pragma unroll
  for (int i = 1; i < NI; ++i) s = add(s, v[i]);
  return s.sum();
}
template <int VEC, int NI>
__device__ __forceinline__ float dot_of(const Vals<VEC> (&v)[NI], const Vals<VEC> (&w)[NI]) {
  Vals<VEC> s = mul(v[0], w[0]);
#pragma unroll
  for (int i = 1; i < NI; ++i) s = fma(v[i], w[i], s);
  return s.sum();
}

// v - mean, zeros past K
template <int VEC, int NI>
__device__ __forceinline__ void centre(Vals<VEC> (&v)[NI], float mean, int W) {
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    v[i] = add(v[i], splat<VEC>(col0<VEC>(i) < W ? -mean : 0.0f));
  }
}

// Normalises the row held in v (zeros past K) in place.
template <int VEC, int NI>
__device__ __forceinline__ void normalise(Vals<VEC> (&v)[NI], int kind, float eps, int W, float rk, BlockSum& sum) {
  if (kind == BL_NORM_NONE) return;
  if (kind == BL_NORM_LAYER) centre<VEC, NI>(v, __fmul_rn(sum.one(sum_of<VEC, NI>(v)), rk), W);
  const Vals<VEC> r = splat<VEC>(inv_dev(sum.one(dot_of<VEC, NI>(v, v)), rk, eps));
#pragma unroll
  for (int i = 0; i < NI; ++i) v[i] = mul(v[i], r);
}

// The codes of eight values against s (c127 = fl(127 / s), |v| <= s) as bytes:
// quant_act_fast_n with the codes taken from the low byte of t + 1.5 * 2^23 and
// one test for all eight.
__device__ __forceinline__ uint2 quant8(const Vals<8>& v, float s, float c127) {
  const F2 c(c127, c127), magic(12582912.0f, 12582912.0f), back(-12582912.0f, -12582912.0f), minus(-1.0f, -1.0f);
  uint32_t b[8];
  float far = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const F2 t = mul(v.p[i], c), r = add(t, magic), d = fma(add(r, back), minus, t);
    float r0, r1, d0, d1;
    r.get(r0, r1);
    d.get(d0, d1);
    b[2 * i] = __float_as_uint(r0);
    b[2 * i + 1] = __float_as_uint(r1);
    // NaN stays, and takes the branch below
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(far) : "f"(fabsf(d0)));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(far) : "f"(fabsf(d1)));
  }
  if (!(far < 0.49993896484375f)) {
    float f[8];
    v.get(f);
    int q[8];
    quant_act_fast_n<8>(f, s, c127, q);
    return make_uint2(pack4(q), pack4(q + 4));
  }
  auto four = [](const uint32_t* w) {
    return __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
  };
  return make_uint2(four(b), four(b + 4));
}

// ---- forward, the row in registers --------------------------------------------
// Up to 16 values per thread: the next row is in flight during this one, and the
// column vectors sit in shared slots (0: gw, 1: w2, 2: gb, 3: b2; zeros past K, so
// that only loads and stores ask whether a column exists); 32 values: neither
// fits, the vectors are read again for each row.
constexpr bool norm_hold(int values) { return values <= 16; }

template <int BDT, int RDT, int VEC, int NI, bool BIAS>
__global__ void __launch_bounds__(norm_max_threads(VEC, NI), VEC * NI <= 8 ? 2 : 1)
    residual_norm_kernel(const NormParams p_arg, const void* __restrict__ b, const void* __restrict__ r, int64_t M,
                         int64_t K, void* __restrict__ h, void* __restrict__ y, int ydt, int8_t* __restrict__ xq,
                         float* __restrict__ scale) {
  pdl_enter(b, r, h, y, xq, scale);
  const NormParams p = params_after_wait(p_arg);
  constexpr bool kHold = norm_hold(VEC * NI);
  extern __shared__ __align__(16) float slot_mem[];
  Slots<VEC, NI> slots{slot_mem};
  __shared__ __align__(16) float sum_mem[2][4][32];
  const float rk = __fdiv_rn(1.0f, static_cast<float>(K));
  const int W = static_cast<int>(K);
  Raw<BDT, VEC> nb[NI];
  Raw<RDT, VEC> nr[NI];
  auto fetch = [&](int64_t m) {
    const void *pb = row_of(b, BDT, m, K), *pr = row_of(r, RDT, m, K);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      nb[i].zero();
      nr[i].zero();
      if (m < M && k < W) {
        nb[i].load(pb, k);
        nr[i].load(pr, k);
      }
    }
  };
  fetch(blockIdx.x);
  // gate row of the block's current token, and the first token past it
  int64_t g_row = p.gate == nullptr ? 0 : blockIdx.x / p.gate_rows, g_next = (g_row + 1) * p.gate_rows;
  const float* gate = p.gate == nullptr ? nullptr : p.gate + g_row * K;
  auto hold_branch = [&]() {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      const bool live = k < W;
      slots.put(0, i, live ? branch_factor<VEC>(p, gate, k) : splat<VEC>(0.0f));
      if constexpr (BIAS) slots.put(2, i, live ? branch_offset<VEC>(p, gate, k) : splat<VEC>(0.0f));
    }
  };
  if constexpr (kHold) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      const bool live = k < W;
      slots.put(1, i, live ? col_vals<VEC>(p.pre_w, k, 1.0f) : splat<VEC>(0.0f));
      if constexpr (BIAS) slots.put(3, i, live ? col_vals<VEC>(p.pre_b, k, 0.0f) : splat<VEC>(0.0f));
    }
    hold_branch();
  }
  BlockSum sum(sum_mem);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    Vals<VEC> v[NI], rr[NI];
    if constexpr (!kHold) {
      if (m != blockIdx.x) fetch(m);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      v[i] = vals(nb[i]);
      rr[i] = vals(nr[i]);
    }
    if constexpr (kHold) fetch(m + gridDim.x);
    if (p.gate != nullptr && m >= g_next) {
      g_row = m / p.gate_rows;
      g_next = (g_row + 1) * p.gate_rows;
      gate = p.gate + g_row * K;
      if constexpr (kHold) hold_branch();
    }
    void* ph = row_of(h, RDT, m, K);
    normalise<VEC, NI>(v, p.post, p.post_eps, W, rk, sum);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      if (kHold || k < W) {
        // both products rounded before their sum: it is 0 where they cancel, and the same
        // with b and r exchanged (one fused product would leave its rounding behind)
        const Vals<VEC> gw = kHold ? slots.get(0, i) : branch_factor<VEC>(p, gate, k);
        Vals<VEC> t;
        if constexpr (BIAS)
          t = fma(gw, v[i], kHold ? slots.get(2, i) : branch_offset<VEC>(p, gate, k));
        else
          t = mul(gw, v[i]);
        v[i] = add_apart(mul(rr[i], splat<VEC>(p.res_scale)), t);
        if (h != nullptr && k < W) store_vals<RDT, VEC>(ph, k, v[i]);
      }
    }
    if (y == nullptr && xq == nullptr) continue;
    normalise<VEC, NI>(v, p.pre, p.pre_eps, W, rk, sum);
    void* py = row_of(y, ydt, m, K);
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      if (kHold || k < W) {
        const Vals<VEC> w = kHold ? slots.get(1, i) : col_vals<VEC>(p.pre_w, k, 1.0f);
        if constexpr (BIAS)
          v[i] = fma(v[i], w, kHold ? slots.get(3, i) : col_vals<VEC>(p.pre_b, k, 0.0f));
        else
          v[i] = mul(v[i], w);
        float f[VEC];
        v[i].get(f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) amax = fmaxf(amax, fabsf(f[j]));
        if (y != nullptr && k < W) store_vec_dt<VEC>(py, ydt, k, f);
      }
    }
    if (xq == nullptr) continue;
    const float s = fmaxf(sum.max(amax), 1e-6f);
    const float c127 = __fdiv_rn(127.0f, s);
    int8_t* pq = xq + m * K;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      if (k < W) {
        if constexpr (VEC == 8) {
          *reinterpret_cast<uint2*>(pq + k) = quant8(v[i], s, c127);
        } else {
          float f[VEC];
          int q[VEC];
          v[i].get(f);
          quant_act_fast_n<VEC>(f, s, c127, q);
          pq[k] = static_cast<int8_t>(q[0]);
        }
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
  __shared__ __align__(16) float sum_mem[2][4][32];
  BlockSum sum(sum_mem);
  const float rk = __fdiv_rn(1.0f, static_cast<float>(K));
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
    float mean1 = 0.0f, r1 = 1.0f, mean2 = 0.0f, r2 = 1.0f;
    auto bv = [&](int64_t k) { return load_elem<BDT>(b, m * K + k); };
    auto hv = [&](int64_t k) {
      float w, c, g;
      load_col<1>(p.post_w, k, 1.0f, &w);
      load_col<1>(p.post_b, k, 0.0f, &c);
      load_col<1>(gate, k, 1.0f, &g);
      const float u = (bv(k) - mean1) * r1 * w + c;  // (two rounded products, as in the other kernel)
      return __fadd_rn(__fmul_rn(p.res_scale, load_elem<RDT>(r, m * K + k)), __fmul_rn(p.branch_scale * g, u));
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
    if (p.post == BL_NORM_LAYER) mean1 = __fmul_rn(total(bv), rk);
    if (p.post != BL_NORM_NONE)
      r1 = inv_dev(total([&](int64_t k) { const float d = bv(k) - mean1; return d * d; }), rk, p.post_eps);
    if (y != nullptr || xq != nullptr) {
      if (p.pre == BL_NORM_LAYER) mean2 = __fmul_rn(total(hv), rk);
      if (p.pre != BL_NORM_NONE)
        r2 = inv_dev(total([&](int64_t k) { const float d = hv(k) - mean2; return d * d; }), rk, p.pre_eps);
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
  using V = Vals<VEC>;
  extern __shared__ __align__(16) float slot_mem[];
  Slots<VEC, NI> slots{slot_mem};
  __shared__ __align__(16) float sum_mem[2][4][32];
  const float rk = __fdiv_rn(1.0f, static_cast<float>(K));
  const int64_t m0 = blockIdx.x * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  constexpr bool kInReg = VEC * NI <= 8;
  constexpr int kRegs = kInReg ? NI : 1;
  constexpr int kAcc = 2;  // first slot of the running sums
  const int64_t plane = static_cast<int64_t>(gridDim.x) * K;
  bool grown = false;  // part holds dw1, db1 of earlier runs
  V aw2[kRegs], aA[kRegs], ab2[BIAS ? kRegs : 1], aB[BIAS ? kRegs : 1];
  const int W = static_cast<int>(K);
  Raw<BDT, VEC> rb[NI];
  Raw<RDT, VEC> rh[NI], rg[NI];
  RawAny<VEC> gy[NI];
  auto fetch = [&](int64_t m) {
    const void *pb = row_of(b, BDT, m, K), *ph = row_of(h, RDT, m, K), *pd = row_of(dh, RDT, m, K);
    const void* py = row_of(dy, dydt, m, K);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      rg[i].zero();
      rb[i].zero();
      rh[i].zero();
      gy[i].zero(dydt);
      if (m < m1 && k < W) {
        rb[i].load(pb, k);
        rh[i].load(ph, k);
        gy[i].load(py, dydt, k);
        if (dh != nullptr) rg[i].load(pd, k);
      }
    }
  };
  fetch(m0);
  // gate row of the current run, and the first token past it
  int64_t g_row = p.gate == nullptr ? 0 : m0 / p.gate_rows;
  int64_t g_next = p.gate == nullptr ? M : (g_row + 1) * p.gate_rows;
  auto gate = [&]() { return p.gate == nullptr ? nullptr : p.gate + g_row * K; };
  auto hold_branch = [&]() {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      slots.put(0, i, k < W ? branch_factor<VEC>(p, gate(), k) : splat<VEC>(0.0f));
    }
  };
  // the sums of a finished run: into dw1, db1 and its gate row
  auto flush = [&]() {
    const bool whole = gate_row_whole(g_row, p.gate_rows, M, m0, m1);
    float* dst = dgate == nullptr ? nullptr : whole ? dgate + g_row * K : gpart + (blockIdx.x + g_row) * K;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      if (k < W) {
        V sA, sB;
        if constexpr (kInReg) {
          sA = aA[i];
          aA[i].fill(0.0f);
          if constexpr (BIAS) {
            sB = aB[i];
            aB[i].fill(0.0f);
          }
        } else {
          sA = slots.get(kAcc + 1, i);
          slots.put(kAcc + 1, i, splat<VEC>(0.0f));
          if constexpr (BIAS) {
            sB = slots.get(kAcc + 3, i);
            slots.put(kAcc + 3, i, splat<VEC>(0.0f));
          }
        }
        const V bg = mul(splat<VEC>(p.branch_scale), col_vals<VEC>(gate(), k, 1.0f));
        auto grow = [&](int slot, int vec, const V& a) {
          if constexpr (kInReg) {
            slots.put(slot, i, fma(bg, a, slots.get(slot, i)));
          } else if (part != nullptr) {
            float* at = part + vec * plane + blockIdx.x * K;
            store_vals<BL_F32, VEC>(at, k, fma(bg, a, grown ? col_vals<VEC>(at, k, 0.0f) : splat<VEC>(0.0f)));
          }
        };
        grow(2, 2, sA);
        if constexpr (BIAS) grow(3, 3, sB);
        if (dst != nullptr) {
          V t = mul(col_vals<VEC>(p.post_w, k, 1.0f), sA);
          if constexpr (BIAS) t = fma(col_vals<VEC>(p.post_b, k, 0.0f), sB, t);
          t = mul(splat<VEC>(p.branch_scale), t);
          if (VEC > 1 && (reinterpret_cast<uintptr_t>(dst + k) & 15) == 0) {
            store_vals<BL_F32, VEC>(dst, k, t);
          } else {
            float f[VEC];
            t.get(f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) dst[k + j] = f[j];
          }
        }
      }
    }
    grown = true;
  };
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = col0<VEC>(i);
#pragma unroll
    for (int v = 2; v < grad_slots(VEC * NI, BIAS); ++v) slots.put(v, i, splat<VEC>(0.0f));
    if constexpr (kInReg) {
      aw2[i].fill(0.0f);
      aA[i].fill(0.0f);
      if constexpr (BIAS) {
        ab2[i].fill(0.0f);
        aB[i].fill(0.0f);
      }
    }
    slots.put(1, i, k < W ? col_vals<VEC>(p.pre_w, k, 1.0f) : splat<VEC>(0.0f));
  }
  hold_branch();
  BlockSum sum(sum_mem);
  for (int64_t m = m0; m < m1; ++m) {
    V n1[NI], n2[NI], d2[NI], d[NI], dyv[NI];
    if constexpr (!kInReg) {
      if (m != m0) fetch(m);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      n1[i] = vals(rb[i]);
      n2[i] = vals(rh[i]);
      d[i] = vals(rg[i]);
      float f[VEC];
      gy[i].get(dydt, f);
      dyv[i].set(f);
    }
    if constexpr (kInReg) fetch(m + 1);
    if (m >= g_next) {
      flush();
      ++g_row;
      g_next += p.gate_rows;
      hold_branch();
    }
    if (p.post == BL_NORM_LAYER || p.pre == BL_NORM_LAYER) {
      const float2 t = sum.two(sum_of<VEC, NI>(n1), sum_of<VEC, NI>(n2));
      if (p.post == BL_NORM_LAYER) centre<VEC, NI>(n1, __fmul_rn(t.x, rk), W);
      if (p.pre == BL_NORM_LAYER) centre<VEC, NI>(n2, __fmul_rn(t.y, rk), W);
    }
    // both deviations, and the sums through the norm before the next block
#pragma unroll
    for (int i = 0; i < NI; ++i) d2[i] = mul(dyv[i], slots.get(1, i));
    const float4 t = sum.four(dot_of<VEC, NI>(n1, n1), dot_of<VEC, NI>(n2, n2), sum_of<VEC, NI>(d2),
                              dot_of<VEC, NI>(d2, n2));
    const float r1 = p.post == BL_NORM_NONE ? 1.0f : inv_dev(t.x, rk, p.post_eps);
    const float r2 = p.pre == BL_NORM_NONE ? 1.0f : inv_dev(t.y, rk, p.pre_eps);
    const float s = p.pre == BL_NORM_LAYER ? __fmul_rn(t.z, rk) : 0.0f;
    const float q = p.pre == BL_NORM_NONE ? 0.0f : __fmul_rn(__fmul_rn(r2, t.w), rk);
    void *pr = row_of(dr, RDT, m, K), *po = row_of(db, BDT, m, K);
    const V r1v = splat<VEC>(r1), r2v = splat<VEC>(r2), mq = splat<VEC>(-q), ms = splat<VEC>(-s);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int k = col0<VEC>(i);
      n1[i] = mul(n1[i], r1v);
      const V u2 = mul(n2[i], r2v);
      d[i] = fma(r2v, fma(u2, mq, add(d2[i], ms)), d[i]);
      if (dr != nullptr && k < W) store_vals<RDT, VEC>(pr, k, mul(splat<VEC>(p.res_scale), d[i]));
      if constexpr (kInReg) {
        aw2[i] = fma(dyv[i], u2, aw2[i]);
        aA[i] = fma(d[i], n1[i], aA[i]);
        if constexpr (BIAS) {
          ab2[i] = add(ab2[i], dyv[i]);
          aB[i] = add(aB[i], d[i]);
        }
      } else {
        slots.put(kAcc, i, fma(dyv[i], u2, slots.get(kAcc, i)));
        slots.put(kAcc + 1, i, fma(d[i], n1[i], slots.get(kAcc + 1, i)));
        if constexpr (BIAS) {
          slots.put(kAcc + 2, i, add(slots.get(kAcc + 2, i), dyv[i]));
          slots.put(kAcc + 3, i, add(slots.get(kAcc + 3, i), d[i]));
        }
      }
      d2[i] = mul(slots.get(0, i), d[i]);  // dn1
    }
    if (db != nullptr) {
      float s1 = 0.0f, p1 = 0.0f;
      if (p.post != BL_NORM_NONE) {
        const float2 t1 = sum.two(sum_of<VEC, NI>(d2), dot_of<VEC, NI>(d2, n1));
        s1 = p.post == BL_NORM_LAYER ? __fmul_rn(t1.x, rk) : 0.0f;
        p1 = __fmul_rn(t1.y, rk);
      }
      const V mp = splat<VEC>(-p1), m1v = splat<VEC>(-s1);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int k = col0<VEC>(i);
        if (k < W) store_vals<BDT, VEC>(po, k, mul(r1v, fma(n1[i], mp, add(d2[i], m1v))));
      }
    }
  }
  flush();
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int k = col0<VEC>(i);
    const int64_t o = static_cast<int64_t>(blockIdx.x) * K + k;
    if (k < W) {
      store_vals<BL_F32, VEC>(part, o, kInReg ? aw2[kInReg ? i : 0] : slots.get(kAcc, i));
      if constexpr (BIAS) store_vals<BL_F32, VEC>(part, o + plane, kInReg ? ab2[kInReg ? i : 0] : slots.get(kAcc + 2, i));
      if constexpr (kInReg) {
        store_vals<BL_F32, VEC>(part, o + 2 * plane, slots.get(2, i));
        if constexpr (BIAS) store_vals<BL_F32, VEC>(part, o + 3 * plane, slots.get(3, i));
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
  __shared__ __align__(16) float sum_mem[2][4][32];
  BlockSum sum(sum_mem);
  const float rk = __fdiv_rn(1.0f, static_cast<float>(K));
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
    if (p.post == BL_NORM_LAYER) t.mean1 = __fmul_rn(mean.x, rk);
    if (p.pre == BL_NORM_LAYER) t.mean2 = __fmul_rn(mean.y, rk);
    const float2 sq = total([&](int64_t k, float& a, float& c) {
      const float d1 = bv(k) - t.mean1, d2 = hv(k) - t.mean2;
      a += d1 * d1;
      c += d2 * d2;
    });
    if (p.post != BL_NORM_NONE) t.r1 = inv_dev(sq.x, rk, p.post_eps);
    if (p.pre != BL_NORM_NONE) {
      t.r2 = inv_dev(sq.y, rk, p.pre_eps);
      const float2 v = total([&](int64_t k, float& a, float& c) {
        float g, w2;
        load_vec_dt<1>(dy, dydt, m * K + k, &g);
        load_col<1>(p.pre_w, k, 1.0f, &w2);
        a += g * w2;
        c += g * w2 * (hv(k) - t.mean2) * t.r2;
      });
      t.s = p.pre == BL_NORM_LAYER ? __fmul_rn(v.x, rk) : 0.0f;
      t.q = __fmul_rn(v.y, rk);
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
      t.s1 = p.post == BL_NORM_LAYER ? __fmul_rn(v.x, rk) : 0.0f;
      t.q1 = __fmul_rn(v.y, rk);
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

// The opt-in for more than 48 KB of shared memory (the kernels' own 1 KB of sums
// counts too).
template <typename Kern>
cudaError_t allow_smem(Kern kern, size_t bytes) {
  return bytes <= 44 * 1024 ? cudaSuccess
                            : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(bytes));
}

// The grid of a persistent kernel for `rows` work items: one wave.  `memo` keeps
// the blocks per SM of each block size (they depend on nothing else).
template <typename Kern>
unsigned one_wave(Kern kern, std::atomic<int>* memo, int threads, size_t smem, int64_t rows) {
  int per_sm = memo[threads / 32].load(std::memory_order_relaxed);
  if (per_sm == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess || per_sm < 1)
      per_sm = 1;
    memo[threads / 32].store(per_sm, std::memory_order_relaxed);
  }
  const int64_t cap = static_cast<int64_t>(device_sms()) * per_sm;
  return static_cast<unsigned>(rows < cap ? rows : cap);
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
  static std::atomic<int> memo[2][33];
  return launch_pdl(kern, one_wave(kern, memo[bias], t, smem, M), t, smem, st, p, b, r, M, K, h, y, ydt, xq, scale);
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
  static std::atomic<int> memo[33];
  return launch_pdl(kern, one_wave(kern, memo, kNormLongThreads, 0, M), kNormLongThreads, 0, st, p, b, r, M, K, h, y, ydt, xq,
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
  static std::atomic<int> memo[33];
  cudaError_t e = launch_pdl(ks, one_wave(ks, memo, kNormLongThreads, 0, M), kNormLongThreads, 0, st, p, dy, dydt, dh, b, h, M,
                             K, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(residual_norm_grad_cols_kernel<BDT, RDT>,
                    dim3(static_cast<unsigned>((K + kGradColThreads - 1) / kGradColThreads),
                         static_cast<unsigned>(blocks)),
                    kGradColThreads, 0, st, p, dy, dydt, dh, b, h, M, K, rows_per,
                    static_cast<const GradRow*>(rows), dr, db, part, gpart, dgate);
}

}  // namespace

// Row blocks of the backward (partial sums): one wave of what the SMs hold at 112
// registers a thread, eight blocks per SM at most (12000 x 1001: three blocks per
// SM, of which two fit, took 126 us, two take 98).
int64_t norm_grad_blocks(int64_t M, int64_t K) {
  const int threads = K % 8 == 0 ? row_threads(K, 8, K <= 8 * 512 ? 1 : 3) : row_threads(K, 1, K <= 4 * 512 ? 4 : 8);
  int64_t per_sm = 576 / threads;
  per_sm = per_sm < 1 ? 1 : (per_sm > 8 ? 8 : per_sm);
  const int64_t most = per_sm * device_sms();
  int64_t rows_per = (M + most - 1) / most;
  return M > 0 ? (M + rows_per - 1) / rows_per : 1;
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
  const int64_t blocks = norm_grad_blocks(M, K);
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
