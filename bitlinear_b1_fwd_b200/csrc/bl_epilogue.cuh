// bl_epilogue.cuh -- bias, activation and residual of the forward product,
// applied where a kernel dequantizes its INT32 sums:
//   z = fl(fl(acc c) + bias),  y = act(z) + residual,
// in fp32 and rounded once per stored value.  The multiply and the add are
// kept apart (no fma), so z has the same bits in every kernel.
#pragma once

#include "bl_common.cuh"
#include "bl_kernels.h"

namespace bl {

// z e / (1 + e) for z < 0 and z / (1 + e) otherwise, e = exp(-|z|) in (0, 1]: no
// overflow, and the lower tail keeps its relative precision.  exp(-a) = 2^t
// (1 + ln2 r) with t = fl(-a log2 e) and r what that rounding and log2 e's own
// lost; the exponent unit is within 2^-22 and the reciprocal within 2^-23, so
// the result is within 8 u |a|.  About a third of the instructions of expf and
// the IEEE divide, which held the tensor-core epilogue of 4096 x 3200 -> 8640
// back by some 100 us.
__device__ __forceinline__ float act_silu(float z) {
  const float a = fminf(fabsf(z), 120.0f);
  const float t = __fmul_rn(-1.44269502162933349609375f, a);  // log2 e to 24 bits
  const float r = __fmaf_rn(-1.92596299e-8f, a, __fmaf_rn(-1.44269502162933349609375f, a, -t));
  float e, q;
  asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = __fmaf_rn(e, __fmul_rn(0.693147182f, r), e);
  asm("rcp.approx.f32 %0, %1;" : "=f"(q) : "f"(__fadd_rn(1.0f, e)));
  return __fmul_rn(z < 0.0f ? __fmul_rn(z, e) : z, q);
}
__device__ __forceinline__ float act_gelu(float z) {
  // z Phi(z); erfc keeps the relative precision of the lower tail
  return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(-0.70710678118654752f, z)));
}
__device__ __forceinline__ float act_apply(int act, float z) {
  switch (act) {
    case BL_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays
    case BL_ACT_RELU2: {
      const float p = z < 0.0f ? 0.0f : z;
      return __fmul_rn(p, p);
    }
    case BL_ACT_SILU: return act_silu(z);
    case BL_ACT_GELU: return act_gelu(z);
    default: return z;
  }
}

// The epilogue's pointers through an opaque move (see pdl_after): used by
// kernels that started before their predecessor had finished.
__device__ __forceinline__ Epilogue epilogue_after_wait(Epilogue ep) {
  pdl_after(ep.bias);
  pdl_after(ep.res);
  pdl_after(ep.pre);
  return ep;
}

__device__ __forceinline__ float load_out(const void* p, int dt, int64_t o) {
  return dt == BL_F32 ? __ldcg(static_cast<const float*>(p) + o)
                      : bf16_bits_to_f32(__ldcg(static_cast<const uint16_t*>(p) + o));
}
__device__ __forceinline__ void store_out(void* p, int dt, int64_t o, float v) {
  if (dt == BL_F32)
    static_cast<float*>(p)[o] = v;
  else
    static_cast<__nv_bfloat16*>(p)[o] = __float2bfloat16_rn(v);
}

// One output of column n (of the whole matrix) at element o of y.
__device__ __forceinline__ void epilogue_store(const Epilogue& ep, void* y, int ydt, int64_t o, int64_t n, int acc,
                                               float cf) {
  if (ydt == BL_I32) {
    static_cast<int32_t*>(y)[o] = acc;
    return;
  }
  float v = __fmul_rn(__int2float_rn(acc), cf);
  if (ep.act >= 0) {
    v = __fadd_rn(v, ep.bias != nullptr ? __ldcg(ep.bias + n) : 0.0f);
    if (ep.pre != nullptr) store_out(ep.pre, ydt, o, v);
    v = act_apply(ep.act, v);
    if (ep.res != nullptr) v = __fadd_rn(v, load_out(ep.res, ydt, o));
  }
  store_out(y, ydt, o, v);
}

// act in place over NC values (fp32 bits): one unrolled loop per activation, the
// choice is uniform and made once
template <int NC>
__device__ __forceinline__ void epilogue_act(int act, uint32_t (&acc)[NC]) {
  switch (act) {
    case BL_ACT_RELU:
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(act_apply(BL_ACT_RELU, __uint_as_float(acc[j])));
      break;
    case BL_ACT_RELU2:
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(act_apply(BL_ACT_RELU2, __uint_as_float(acc[j])));
      break;
    case BL_ACT_SILU:
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(act_silu(__uint_as_float(acc[j])));
      break;
    case BL_ACT_GELU:
#pragma unroll
      for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(act_gelu(__uint_as_float(acc[j])));
      break;
    default: break;
  }
}

// NC outputs of one column n held as INT32 sums by a tensor-core epilogue
// thread, for consecutive tokens: acc[j] becomes the bits of the fp32 output.
// cf[j]: the tokens' dequantization factors; bias: the column's; o: the first
// token's element of y, tokens ld elements apart; live: tokens to read (0 when
// the column is past N).  keep(j, z) receives the pre-activations when they
// are kept.
template <int NC, typename Keep>
__device__ __forceinline__ void epilogue_chunk(const Epilogue& ep, uint32_t (&acc)[NC], const float* cf, float bias,
                                               int ydt, int64_t o, int64_t ld, int live, Keep keep) {
#pragma unroll
  for (int j = 0; j < NC; ++j)
    acc[j] = __float_as_uint(__fmul_rn(__int2float_rn(static_cast<int>(acc[j])), cf[j]));
  if (ep.act < 0) return;
#pragma unroll
  for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(__fadd_rn(__uint_as_float(acc[j]), bias));
  if (ep.pre != nullptr) {
#pragma unroll
    for (int j = 0; j < NC; ++j) keep(j, __uint_as_float(acc[j]));
  }
  epilogue_act<NC>(ep.act, acc);
  if (ep.res != nullptr) {
    float r[NC];  // all loads in flight together
#pragma unroll
    for (int j = 0; j < NC; ++j) r[j] = j < live ? load_out(ep.res, ydt, o + j * ld) : 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(__fadd_rn(__uint_as_float(acc[j]), r[j]));
  }
}

}  // namespace bl
