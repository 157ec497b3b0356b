// bl_vec.cuh -- typed vector loads and stores of activations, block sums.
#pragma once

#include "bl_common.cuh"

namespace bl {

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
template <int DT>
struct Raw<DT, 1> {
  float f;
  __device__ __forceinline__ void zero() { f = 0.0f; }
  __device__ __forceinline__ void load(const void* p, int64_t e) { f = load_elem<DT>(p, e); }
  __device__ __forceinline__ void get(float* v) const { v[0] = f; }
};

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

// Sums of one to four values over the block in a fixed order, the same in every
// thread; one barrier.  Two buffers alternate: a buffer is written again only
// after the barrier of the next sum, which every thread reaches after its
// reads.
struct BlockSum {
  float4 (*buf)[32];  // shared [2][32]
  int nw, phase;
  template <int N>
  __device__ __forceinline__ void run(float (&a)[N]) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) a[j] += __shfl_xor_sync(0xffffffffu, a[j], o);
    if (nw == 1) return;
    float4* w = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) {
      float* d = reinterpret_cast<float*>(w + (threadIdx.x >> 5));
#pragma unroll
      for (int j = 0; j < N; ++j) d[j] = a[j];
    }
    __syncthreads();
    const float* d = reinterpret_cast<const float*>(w + lane);
#pragma unroll
    for (int j = 0; j < N; ++j) a[j] = lane < nw ? d[j] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j) a[j] += __shfl_xor_sync(0xffffffffu, a[j], o);
  }
  __device__ __forceinline__ float one(float a) {
    float v[1] = {a};
    run(v);
    return v[0];
  }
  __device__ __forceinline__ float2 two(float a, float b) {
    float v[2] = {a, b};
    run(v);
    return make_float2(v[0], v[1]);
  }
  __device__ __forceinline__ float4 four(float a, float b, float c, float d) {
    float v[4] = {a, b, c, d};
    run(v);
    return make_float4(v[0], v[1], v[2], v[3]);
  }
  __device__ __forceinline__ float max(float a) {
    a = warp_maxf(a);
    if (nw == 1) return a;
    float4* w = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) w[threadIdx.x >> 5].x = a;
    __syncthreads();
    return warp_maxf(lane < nw ? w[lane].x : 0.0f);
  }
};

}  // namespace bl
