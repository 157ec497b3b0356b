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
// of each array.  The chain of row sums (two for RMS + RMS, each a barrier)
// is the latency to hide: several blocks per SM and the next row's loads in
// flight during the sums of this one.  The column sums of the backward stay in
// registers over a block's rows and meet in a second kernel in a fixed order.
// Statistics are two-pass (the mean, then the squares about it) in fp32.
#include "bl_common.cuh"
#include "bl_gemv.cuh"
#include "bl_kernels.h"
#include "bl_vec.cuh"

namespace bl {
namespace {

constexpr int kNormMaxThreads = 512;

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
    const float mean = sum(s, 0.0f).x / static_cast<float>(K);
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
  const float r = inv_dev(sum(q, 0.0f).x, K, eps);
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[i][j] *= r;
  return r;
}

// ---- forward, the row in registers --------------------------------------------
template <int BDT, int RDT, int VEC, int NI>
__global__ void __launch_bounds__(kNormMaxThreads)
    residual_norm_kernel(const NormParams p_arg, const void* __restrict__ b, const void* __restrict__ r, int64_t M,
                         int64_t K, void* __restrict__ h, void* __restrict__ y, int ydt, int8_t* __restrict__ xq,
                         float* __restrict__ scale) {
  pdl_enter(b, r, h, y, xq, scale);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float2 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  auto fetch = [&](int64_t m, float (&vb)[NI][VEC], float (&vr)[NI][VEC]) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) vb[i][j] = vr[i][j] = 0.0f;
      if (m < M && k < K) {
        load_vec<BDT, VEC>(b, m * K + k, vb[i]);
        load_vec<RDT, VEC>(r, m * K + k, vr[i]);
      }
    }
  };
  // the next row is in flight while this one is worked on, where 16 values
  // per thread or fewer leave the registers for it
  constexpr bool kAhead = VEC * NI <= 16;
  float nb[kAhead ? NI : 1][VEC], nr[kAhead ? NI : 1][VEC];
  if constexpr (kAhead) fetch(blockIdx.x, nb, nr);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    float v[NI][VEC], rr[NI][VEC];
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = nb[i][j];
          rr[i][j] = nr[i][j];
        }
      fetch(m + gridDim.x, nb, nr);
    } else {
      fetch(m, v, rr);
    }
    normalise<VEC, NI>(v, p.post, p.post_eps, K, sum);
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float w[VEC], c[VEC], g[VEC];
        load_col<VEC>(p.post_w, k, 1.0f, w);
        load_col<VEC>(p.post_b, k, 0.0f, c);
        load_col<VEC>(gate, k, 1.0f, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[i][j] = p.res_scale * rr[i][j] + p.branch_scale * g[j] * (v[i][j] * w[j] + c[j]);
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
        load_col<VEC>(p.pre_w, k, 1.0f, w);
        load_col<VEC>(p.pre_b, k, 0.0f, c);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i][j] = v[i][j] * w[j] + c[j];
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
__global__ void __launch_bounds__(kNormMaxThreads)
    residual_norm_long_kernel(const NormParams p_arg, const void* __restrict__ b, const void* __restrict__ r, int64_t M,
                              int64_t K, void* __restrict__ h, void* __restrict__ y, int ydt, int8_t* __restrict__ xq,
                              float* __restrict__ scale) {
  pdl_enter(b, r, h, y, xq, scale);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float2 buf[2][32];
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
      return sum(s0 + s1, 0.0f).x;
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
// Block c takes rows [c rows_per, (c + 1) rows_per).  part: [gridDim.x][4][K]
// (dw2, db2, dw1, db1); gpart: a row for each run of a block's rows with one
// gate row, at index (block + gate row).
template <int BDT, int RDT, int VEC, int NI, bool BIAS>
__global__ void __launch_bounds__(kNormMaxThreads)
    residual_norm_grad_kernel(const NormParams p_arg, const void* __restrict__ dy, int dydt,
                              const void* __restrict__ dh, const void* __restrict__ b, const void* __restrict__ h,
                              int64_t M, int64_t K, int64_t rows_per, void* __restrict__ dr, void* __restrict__ db,
                              float* __restrict__ part, float* __restrict__ gpart) {
  pdl_enter(dy, dh, b, h, dr, db, part, gpart);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float2 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  const float fk = static_cast<float>(K);
  const int64_t m0 = blockIdx.x * rows_per, m1 = m0 + rows_per < M ? m0 + rows_per : M;
  float aw2[NI][VEC], aw1[NI][VEC], ag[NI][VEC];
  float ab2[BIAS ? NI : 1][VEC], ab1[BIAS ? NI : 1][VEC];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      aw2[i][j] = aw1[i][j] = ag[i][j] = 0.0f;
      if constexpr (BIAS) ab2[i][j] = ab1[i][j] = 0.0f;
    }
  auto flush_gate = [&](int64_t g) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) store_vec<BL_F32, VEC>(gpart, (blockIdx.x + g) * K + k, ag[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) ag[i][j] = 0.0f;
    }
  };
  for (int64_t m = m0; m < m1; ++m) {
    float n1[NI][VEC], n2[NI][VEC], gy[NI][VEC], gh[NI][VEC];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
#pragma unroll
      for (int j = 0; j < VEC; ++j) n1[i][j] = n2[i][j] = gy[i][j] = gh[i][j] = 0.0f;
      if (k < K) {
        load_vec<BDT, VEC>(b, m * K + k, n1[i]);
        load_vec<RDT, VEC>(h, m * K + k, n2[i]);
        load_vec_dt<VEC>(dy, dydt, m * K + k, gy[i]);
        if (dh != nullptr) load_vec<RDT, VEC>(dh, m * K + k, gh[i]);
      }
    }
    const float r1 = normalise<VEC, NI>(n1, p.post, p.post_eps, K, sum);
    const float r2 = normalise<VEC, NI>(n2, p.pre, p.pre_eps, K, sum);
    // through the norm before the next block
    float s = 0.0f, q = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float w[VEC];
        load_col<VEC>(p.pre_w, k, 1.0f, w);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          aw2[i][j] += gy[i][j] * n2[i][j];
          if constexpr (BIAS) ab2[i][j] += gy[i][j];
          gy[i][j] *= w[j];
          s += gy[i][j];
          q += gy[i][j] * n2[i][j];
        }
      }
    }
    if (p.pre == BL_NORM_NONE) {
      s = q = 0.0f;
    } else {
      const float2 t = sum(s, q);
      s = p.pre == BL_NORM_LAYER ? t.x / fk : 0.0f;
      q = t.y / fk;
    }
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
    float s1 = 0.0f, q1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t k = col0<VEC>(i);
      if (k < K) {
        float w[VEC], c[VEC], g[VEC], out[VEC];
        load_col<VEC>(p.post_w, k, 1.0f, w);
        load_col<VEC>(p.post_b, k, 0.0f, c);
        load_col<VEC>(gate, k, 1.0f, g);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float d = gh[i][j] + r2 * (gy[i][j] - s - n2[i][j] * q);
          out[j] = p.res_scale * d;
          const float bd = p.branch_scale * d;
          ag[i][j] += bd * (n1[i][j] * w[j] + c[j]);
          const float du = bd * g[j];
          aw1[i][j] += du * n1[i][j];
          if constexpr (BIAS) ab1[i][j] += du;
          gy[i][j] = du * w[j];  // dn1
          s1 += gy[i][j];
          q1 += gy[i][j] * n1[i][j];
        }
        if (dr != nullptr) store_vec<RDT, VEC>(dr, m * K + k, out);
      }
    }
    if (db != nullptr) {
      if (p.post == BL_NORM_NONE) {
        s1 = q1 = 0.0f;
      } else {
        const float2 t = sum(s1, q1);
        s1 = p.post == BL_NORM_LAYER ? t.x / fk : 0.0f;
        q1 = t.y / fk;
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int64_t k = col0<VEC>(i);
        if (k < K) {
          float out[VEC];
#pragma unroll
          for (int j = 0; j < VEC; ++j) out[j] = r1 * (gy[i][j] - s1 - n1[i][j] * q1);
          store_vec<BDT, VEC>(db, m * K + k, out);
        }
      }
    }
    if (gpart != nullptr && (m + 1 == m1 || (m + 1) % p.gate_rows == 0)) flush_gate(m / p.gate_rows);
  }
  if (part == nullptr) return;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t k = col0<VEC>(i), o = static_cast<int64_t>(blockIdx.x) * 4 * K + k;
    if (k < K) {
      store_vec<BL_F32, VEC>(part, o, aw2[i]);
      store_vec<BL_F32, VEC>(part, o + 2 * K, aw1[i]);
      if constexpr (BIAS) {
        store_vec<BL_F32, VEC>(part, o + K, ab2[i]);
        store_vec<BL_F32, VEC>(part, o + 3 * K, ab1[i]);
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
__global__ void __launch_bounds__(kNormMaxThreads)
    residual_norm_grad_stats_kernel(const NormParams p_arg, const void* __restrict__ dy, int dydt,
                                    const void* __restrict__ dh, const void* __restrict__ b,
                                    const void* __restrict__ h, int64_t M, int64_t K, GradRow* __restrict__ stats) {
  pdl_enter(dy, dh, b, h, stats);
  const NormParams p = params_after_wait(p_arg);
  __shared__ float2 buf[2][32];
  BlockSum sum{buf, static_cast<int>(blockDim.x >> 5), 0};
  const float fk = static_cast<float>(K);
  for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
    const float* gate = p.gate == nullptr ? nullptr : p.gate + (m / p.gate_rows) * K;
    GradRow t{0.0f, 1.0f, 0.0f, 1.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    auto total = [&](auto f) {
      float a = 0.0f, c = 0.0f;
      for (int64_t k = threadIdx.x; k < K; k += blockDim.x) f(k, a, c);
      return sum(a, c);
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
                                   float* __restrict__ part, float* __restrict__ gpart) {
  pdl_enter(dy, dh, b, h, stats, dr, db, part, gpart);
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
    if (gpart != nullptr && (m + 1 == m1 || (m + 1) % p.gate_rows == 0)) {
      gpart[(c + m / p.gate_rows) * K + k] = ag;
      ag = 0.0f;
    }
  }
  if (part == nullptr) return;
  float* o = part + c * 4 * K + k;
  o[0] = aw2;
  o[K] = ab2;
  o[2 * K] = aw1;
  o[3 * K] = ab1;
}

// The column sums: vector v < 4 of the blocks' partials in block order, or (v
// >= 4) gate row v - 4 from the runs of its rows, in order.
__global__ void __launch_bounds__(128)
    residual_norm_grad_sum_kernel(const float* __restrict__ part, const float* __restrict__ gpart, int64_t blocks,
                                  int64_t rows_per, int64_t M, int64_t K, int64_t gate_rows, float* __restrict__ dw2,
                                  float* __restrict__ db2, float* __restrict__ dw1, float* __restrict__ db1,
                                  float* __restrict__ dgate) {
  pdl_enter(part, gpart, dw2, db2, dw1, db1, dgate);
  const int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (k >= K) return;
  for (int64_t v = blockIdx.y; ; v += gridDim.y) {
    float s = 0.0f;
    if (v < 4) {
      float* out = v == 0 ? dw2 : v == 1 ? db2 : v == 2 ? dw1 : db1;
      if (out == nullptr) continue;
#pragma unroll 8
      for (int64_t c = 0; c < blocks; ++c) s += __ldcg(part + (c * 4 + v) * K + k);
      out[k] = s;
    } else {
      const int64_t g = v - 4;
      if (dgate == nullptr || g * gate_rows >= M) return;
      const int64_t last = (g + 1) * gate_rows < M ? (g + 1) * gate_rows - 1 : M - 1;
      const int64_t c0 = g * gate_rows / rows_per, c1 = last / rows_per;
#pragma unroll 8
      for (int64_t c = c0; c <= c1; ++c) s += __ldcg(gpart + (c + g) * K + k);
      dgate[g * K + k] = s;
    }
  }
}

// Threads of a block for a row of K columns in NI chunks of VEC per thread.
int row_threads(int64_t K, int vec, int ni) {
  const int64_t per = static_cast<int64_t>(vec) * ni;
  return static_cast<int>(((K + per - 1) / per + 31) / 32 * 32);
}

template <typename Kern>
unsigned persistent_grid(Kern kern, int threads, int64_t rows) {
  int per_sm = 1;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess || per_sm < 1) per_sm = 1;
  const int64_t cap = static_cast<int64_t>(device_sms()) * per_sm;
  return static_cast<unsigned>(rows < cap ? rows : cap);
}

template <int BDT, int RDT>
cudaError_t launch_fwd(const NormParams& p, const void* b, const void* r, int64_t M, int64_t K, void* h, void* y,
                       int ydt, int8_t* xq, float* scale, cudaStream_t st) {
  const bool wide = K % 8 == 0 && (reinterpret_cast<uintptr_t>(xq) & 7) == 0;
#define BL_NF(VEC, NI)                                                                                           \
  if (K <= static_cast<int64_t>(kNormMaxThreads) * (VEC) * (NI)) {                                               \
    auto kern = residual_norm_kernel<BDT, RDT, VEC, NI>;                                                         \
    const int t = row_threads(K, VEC, NI);                                                                       \
    return launch_pdl(kern, persistent_grid(kern, t, M), t, 0, st, p, b, r, M, K, h, y, ydt, xq, scale);         \
  }
  if (wide) {
    BL_NF(8, 1)
    BL_NF(8, 2)
    BL_NF(8, 4)
  } else {
    BL_NF(1, 4)
    BL_NF(1, 16)
  }
#undef BL_NF
  auto kern = residual_norm_long_kernel<BDT, RDT>;
  return launch_pdl(kern, persistent_grid(kern, kNormMaxThreads, M), kNormMaxThreads, 0, st, p, b, r, M, K, h, y, ydt,
                    xq, scale);
}

template <int BDT, int RDT>
cudaError_t launch_bwd(const NormParams& p, const void* dy, int dydt, const void* dh, const void* b, const void* h,
                       int64_t M, int64_t K, void* dr, void* db, bool bias, int64_t blocks, int64_t rows_per,
                       float* part, float* gpart, void* stats, cudaStream_t st) {
  const bool wide = K % 8 == 0;
#define BL_NB(VEC, NI)                                                                                            \
  if (K <= static_cast<int64_t>(kNormMaxThreads) * (VEC) * (NI)) {                                                \
    auto kern = bias ? residual_norm_grad_kernel<BDT, RDT, VEC, NI, true>                                         \
                     : residual_norm_grad_kernel<BDT, RDT, VEC, NI, false>;                                       \
    return launch_pdl(kern, static_cast<unsigned>(blocks), row_threads(K, VEC, NI), 0, st, p, dy, dydt, dh, b, h, \
                      M, K, rows_per, dr, db, part, gpart);                                                       \
  }
  if (wide) {
    BL_NB(8, 1)
  } else {
    BL_NB(1, 4)
  }
#undef BL_NB
  GradRow* rows = static_cast<GradRow*>(stats);
  auto ks = residual_norm_grad_stats_kernel<BDT, RDT>;
  cudaError_t e = launch_pdl(ks, persistent_grid(ks, kNormMaxThreads, M), kNormMaxThreads, 0, st, p, dy, dydt, dh, b,
                             h, M, K, rows);
  if (e != cudaSuccess) return e;
  return launch_pdl(residual_norm_grad_cols_kernel<BDT, RDT>,
                    dim3(static_cast<unsigned>((K + kGradColThreads - 1) / kGradColThreads),
                         static_cast<unsigned>(blocks)),
                    kGradColThreads, 0, st, p, dy, dydt, dh, b, h, M, K, rows_per,
                    static_cast<const GradRow*>(rows), dr, db, part, gpart);
}

}  // namespace

// Row blocks of the backward (partial sums): one per SM.
int64_t norm_grad_blocks(int64_t M) {
  const int64_t sms = device_sms();
  const int64_t rows_per = (M + sms - 1) / sms;
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
  const bool bias = db1 != nullptr || db2 != nullptr;
  float* ps = bias || dw1 != nullptr || dw2 != nullptr ? part : nullptr;
  float* gs = dgate != nullptr ? gpart : nullptr;
  cudaError_t e;
#define BL_NB(BDT, RDT) \
  e = launch_bwd<BDT, RDT>(p, dy, dydt, dh, b, h, M, K, dr, db, bias, blocks, rows_per, ps, gs, stats, st)
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
  if (ps != nullptr || gs != nullptr) {
    const int64_t rows = 4 + (gs != nullptr ? (M + p.gate_rows - 1) / p.gate_rows : 0);
    e = launch_pdl(residual_norm_grad_sum_kernel,
                   dim3(static_cast<unsigned>((K + 127) / 128), static_cast<unsigned>(rows < 4096 ? rows : 4096)), 128,
                   0, st, static_cast<const float*>(part), static_cast<const float*>(gs), blocks, rows_per, M, K,
                   p.gate_rows > 0 ? p.gate_rows : 1, dw2, db2, dw1, db1, dgate);
  }
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace bl
