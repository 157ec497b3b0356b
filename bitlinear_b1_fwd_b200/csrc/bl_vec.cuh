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

// Sums of two values over the block in a fixed order, the same in every
// thread; one barrier.  Two buffers alternate: a buffer is written again only
// after the barrier of the next sum, which every thread reaches after its
// reads.
struct BlockSum {
  float2 (*buf)[32];  // shared [2][32]
  int nw, phase;
  __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    float2* w = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) w[threadIdx.x >> 5] = make_float2(a, b);
    __syncthreads();
    const float2 p = lane < nw ? w[lane] : make_float2(0.0f, 0.0f);
    a = p.x;
    b = p.y;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    return make_float2(a, b);
  }
  __device__ __forceinline__ float max(float a) {
    a = warp_maxf(a);
    float2* w = buf[phase];
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) w[threadIdx.x >> 5].x = a;
    __syncthreads();
    return warp_maxf(lane < nw ? w[lane].x : 0.0f);
  }
};

}  // namespace bl
