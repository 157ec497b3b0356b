// bl_vec.cuh -- typed vector loads and stores of activations, block sums.
#pragma once

#include "bl_common.cuh"

namespace bl {

// VEC consecutive elements as loaded, widened when they are used.
template <int DT, int VEC>
struct Raw;
template <>
struct Raw<BL_BF16, 8> {
  uint4 q;
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    q = __ldcg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e));
  }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <>
struct Raw<BL_F32, 8> {
  float4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void load(const void* p, int64_t e) {
    const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
    a = __ldcg(q);
    b = __ldcg(q + 1);
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Raw<BL_F32, 1> {
  float f;
  __device__ __forceinline__ void zero() { f = 0.0f; }
  __device__ __forceinline__ void load(const void* p, int64_t e) { f = __ldcg(static_cast<const float*>(p) + e); }
  __device__ __forceinline__ void get(float* v) const { v[0] = f; }
};
template <>
struct Raw<BL_BF16, 1> {
  uint16_t q;
  __device__ __forceinline__ void zero() { q = 0; }
  __device__ __forceinline__ void load(const void* p, int64_t e) { q = __ldcg(static_cast<const uint16_t*>(p) + e); }
  __device__ __forceinline__ void get(float* v) const { v[0] = bf16_bits_to_f32(q); }
};

// The same of a type known at run time.
template <int VEC>
struct RawAny {
  Raw<BL_BF16, VEC> h;
  Raw<BL_F32, VEC> f;
  __device__ __forceinline__ void zero(int dt) { dt == BL_F32 ? f.zero() : h.zero(); }
  __device__ __forceinline__ void load(const void* p, int dt, int64_t e) { dt == BL_F32 ? f.load(p, e) : h.load(p, e); }
  __device__ __forceinline__ void get(int dt, float* v) const { dt == BL_F32 ? f.get(v) : h.get(v); }
};

// VEC consecutive elements from element e (VEC = 8: e a multiple of 8 and the
// array 16-byte aligned; VEC = 1: any), widened to fp32.
template <int DT, int VEC>
__device__ __forceinline__ void load_vec(const void* p, int64_t e, float* v) {
  if constexpr (VEC == 8) {
    float t[8];
    load8_aligned<DT>(p, e, t);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = t[j];
  } else {
    v[0] = load_elem<DT>(p, e);
  }
}
template <int VEC>
__device__ __forceinline__ void load_vec_dt(const void* p, int dt, int64_t e, float* v) {
  if (dt == BL_F32)
    load_vec<BL_F32, VEC>(p, e, v);
  else
    load_vec<BL_BF16, VEC>(p, e, v);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <int DT, int VEC>
__device__ __forceinline__ void store_vec(void* p, int64_t e, const float* v) {
  if constexpr (DT == BL_F32) {
    float* q = static_cast<float*>(p) + e;
    if constexpr (VEC == 8) {
      reinterpret_cast<float4*>(q)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(q)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      q[0] = v[0];
    }
  } else {
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) =
          make_uint4(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]), bf16_pair(v[6], v[7]));
    } else {
      static_cast<__nv_bfloat16*>(p)[e] = __float2bfloat16_rn(v[0]);
    }
  }
}
template <int VEC>
__device__ __forceinline__ void store_vec_dt(void* p, int dt, int64_t e, const float* v) {
  if (dt == BL_F32)
    store_vec<BL_F32, VEC>(p, e, v);
  else
    store_vec<BL_BF16, VEC>(p, e, v);
}

// ---- packed fp32 pairs ----------------------------------------------------------
// add, mul and fma on two fp32 values in one instruction.  The assembler makes one
// fma of a mul and an add that takes its result, which it does not do to the scalar
// __fmul_rn and __fadd_rn: where a product has to be rounded before a sum, add_apart.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float lo, float hi) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(lo), "f"(hi)); }
  __device__ __forceinline__ void get(float& lo, float& hi) const {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  }
};
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

// VEC neighbouring values as pairs (VEC = 1: one value).
template <int VEC>
struct Vals {
  static constexpr int P = VEC / 2;
  F2 p[P];
  __device__ __forceinline__ void fill(float c) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = F2(c, c);
  }
  __device__ __forceinline__ void set(const float* f) {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = F2(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ void get(float* f) const {
#pragma unroll
    for (int i = 0; i < P; ++i) p[i].get(f[2 * i], f[2 * i + 1]);
  }
  __device__ __forceinline__ float sum() const {
    F2 s = p[0];
#pragma unroll
    for (int i = 1; i < P; ++i) s = add(s, p[i]);
    float a, b;
    s.get(a, b);
    return a + b;
  }
};
template <>
struct Vals<1> {
  float f0;
  __device__ __forceinline__ void fill(float c) { f0 = c; }
  __device__ __forceinline__ void set(const float* f) { f0 = f[0]; }
  __device__ __forceinline__ void get(float* f) const { f[0] = f0; }
  __device__ __forceinline__ float sum() const { return f0; }
};
template <int VEC>
__device__ __forceinline__ Vals<VEC> splat(float c) {
  Vals<VEC> r;
  r.fill(c);
  return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> add(const Vals<VEC>& a, const Vals<VEC>& b) {
  Vals<VEC> r;
  if constexpr (VEC == 1) {
    r.f0 = __fadd_rn(a.f0, b.f0);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.p[i] = add(a.p[i], b.p[i]);
  }
  return r;
}
// a + b of values as they were rounded (scalar adds)
template <int VEC>
__device__ __forceinline__ Vals<VEC> add_apart(const Vals<VEC>& a, const Vals<VEC>& b) {
  float x[VEC], y[VEC];
  a.get(x);
  b.get(y);
#pragma unroll
  for (int j = 0; j < VEC; ++j) x[j] = __fadd_rn(x[j], y[j]);
  Vals<VEC> r;
  r.set(x);
  return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> mul(const Vals<VEC>& a, const Vals<VEC>& b) {
  Vals<VEC> r;
  if constexpr (VEC == 1) {
    r.f0 = __fmul_rn(a.f0, b.f0);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.p[i] = mul(a.p[i], b.p[i]);
  }
  return r;
}
template <int VEC>
__device__ __forceinline__ Vals<VEC> fma(const Vals<VEC>& a, const Vals<VEC>& b, const Vals<VEC>& c) {
  Vals<VEC> r;
  if constexpr (VEC == 1) {
    r.f0 = __fmaf_rn(a.f0, b.f0, c.f0);
  } else {
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) r.p[i] = fma(a.p[i], b.p[i], c.p[i]);
  }
  return r;
}
template <int DT, int VEC>
__device__ __forceinline__ Vals<VEC> vals(const Raw<DT, VEC>& r) {
  float f[VEC];
  r.get(f);
  Vals<VEC> v;
  v.set(f);
  return v;
}
template <int DT, int VEC>
__device__ __forceinline__ void store_vals(void* p, int64_t e, const Vals<VEC>& v) {
  float f[VEC];
  v.get(f);
  store_vec<DT, VEC>(p, e, f);
}

// Sums of one, two or four values over the block in a fixed order, the same in
// every thread; one barrier.  Within a warp two and four values share the
// exchanges: each step halves the values a lane carries, then the lanes (six
// shuffles for four values).  After the barrier one load per lane takes in every
// warp's sums (16 or 8 bytes: neighbouring warps), and the same exchanges over
// the lanes of a value finish.  Two buffers alternate: a buffer is written again
// only after the barrier of the next sum, which every thread reaches after its
// reads.
struct BlockSum {
  float (*buf)[4][32];  // shared [2][4][32]: phase, value, warp; zero past the last warp
  int nw, phase;
  __device__ __forceinline__ BlockSum(float (*b)[4][32]) : buf(b), nw(static_cast<int>(blockDim.x >> 5)), phase(0) {
    if (nw > 1) {
      for (int i = threadIdx.x; i < 2 * 4 * 32; i += blockDim.x) (&buf[0][0][0])[i] = 0.0f;
      __syncthreads();
    }
  }
  template <int FROM>
  static __device__ __forceinline__ float lanes(float a) {  // over groups of 2 FROM lanes
#pragma unroll
    for (int o = FROM; o >= 1; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  }
  static __device__ __forceinline__ float sum4(const float* w) {
    const float4 q = *reinterpret_cast<const float4*>(w);
    return (q.x + q.y) + (q.z + q.w);
  }
  __device__ __forceinline__ float one(float a) {
    a = lanes<16>(a);
    if (nw == 1) return a;
    float (*w)[32] = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) w[0][threadIdx.x >> 5] = a;
    __syncthreads();
    return lanes<4>(sum4(w[0] + 4 * (lane & 7)));
  }
  __device__ __forceinline__ float2 two(float a, float b) {
    const int lane = threadIdx.x & 31;
    const bool up = (lane & 16) != 0;
    a = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);  // lanes 0-15: a, 16-31: b
    a = lanes<8>(a);
    if (nw > 1) {
      float (*w)[32] = buf[phase];
      phase ^= 1;
      if ((lane & 15) == 0) w[lane >> 4][threadIdx.x >> 5] = a;
      __syncthreads();
      const float2 q = *reinterpret_cast<const float2*>(w[lane >> 4] + 2 * (lane & 15));
      a = lanes<8>(q.x + q.y);
    }
    return make_float2(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, a, 16));
  }
  __device__ __forceinline__ float4 four(float a, float b, float c, float d) {
    const int lane = threadIdx.x & 31;
    const bool up = (lane & 16) != 0, odd = (lane & 8) != 0;
    a = (up ? c : a) + __shfl_xor_sync(0xffffffffu, up ? a : c, 16);  // lanes 0-15: a, b, 16-31: c, d
    b = (up ? d : b) + __shfl_xor_sync(0xffffffffu, up ? b : d, 16);
    a = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);  // eight lanes each
    a = lanes<4>(a);
    if (nw > 1) {
      float (*w)[32] = buf[phase];
      phase ^= 1;
      if ((lane & 7) == 0) w[lane >> 3][threadIdx.x >> 5] = a;
      __syncthreads();
      a = lanes<4>(sum4(w[lane >> 3] + 4 * (lane & 7)));
    }
    return make_float4(__shfl_sync(0xffffffffu, a, 0), __shfl_sync(0xffffffffu, a, 8),
                       __shfl_sync(0xffffffffu, a, 16), __shfl_sync(0xffffffffu, a, 24));
  }
  // the largest of non-negative values (their bits order like unsigned integers)
  __device__ __forceinline__ float max(float a) {
    uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
    if (nw == 1) return __uint_as_float(m);
    float (*w)[32] = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) w[0][threadIdx.x >> 5] = __uint_as_float(m);
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < nw ? __float_as_uint(w[0][lane]) : 0u);
    return __uint_as_float(m);
  }
};

}  // namespace bl
