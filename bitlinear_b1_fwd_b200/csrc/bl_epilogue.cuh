// bl_epilogue.cuh -- bias, activation and residual of the forward product,
// applied where a kernel dequantizes its INT32 sums:
//   z = fl(fl(acc c) + bias),  y = act(z) + residual,
// in fp32 and rounded once per stored value.  The multiply and the add are
// kept apart (no fma), so z has the same bits in every kernel.
#pragma once

#include "bl_common.cuh"
#include "bl_kernels.h"

namespace bl {

// Each activation in two forms.  For outputs of 24 bits, within 8 u |a| (GELU: and
// a few u z^2 |a|), u = 2^-24.  For bf16 outputs (half a step is 2^-9 to 2^-8 of
// the value) the hardware's exponential and reciprocal: SiLU within 2^-17 |a| while
// |z| < 100, GELU within (4 + z^2 / 2) 2^-22 |a| (its exponent is rounded twice);
// results under 2^-118 may be 0.  Every
// kernel uses the same form for the same output type.  The difference is some 15
// and 40 instructions per output: 4096 x 3200 -> 8640 with SiLU and the kept
// pre-activation took 134 us with the first form and 127 with the second, with
// GELU and a residual 158 and 134 (inputs changing from call to call).
template <bool FAST>
__device__ __forceinline__ float act_silu(float z) {
  float e, q;
  if constexpr (FAST) {
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(-1.44269504f, z)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(__fadd_rn(1.0f, e)));
    return __fmul_rn(z, q);
  } else {
    // z e / (1 + e) for z < 0 and z / (1 + e) otherwise, e = exp(-|z|) in (0, 1]: no
    // overflow, and the lower tail keeps its relative precision.  exp(-a) = 2^t
    // (1 + ln2 r) with t = fl(-a log2 e) and r what that rounding and log2 e's own
    // lost; the exponent unit is within 2^-22 and the reciprocal within 2^-23.
    const float a = fminf(fabsf(z), 120.0f);
    const float t = __fmul_rn(-1.44269502162933349609375f, a);  // log2 e to 24 bits
    const float r = __fmaf_rn(-1.92596299e-8f, a, __fmaf_rn(-1.44269502162933349609375f, a, -t));
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(t));
    e = __fmaf_rn(e, __fmul_rn(0.693147182f, r), e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q) : "f"(__fadd_rn(1.0f, e)));
    return __fmul_rn(z < 0.0f ? __fmul_rn(z, e) : z, q);
  }
}

// Phi(-|z|) = erfc(x) / 2, x = |z| / sqrt 2, and exp(-z^2 / 2).  erfc(x) exp(x^2) is
// fitted over x in [0, 10] by t times a polynomial of degree 7 in t = 1 / (1 + 0.44
// x), least largest relative error (2^-21 as evaluated in fp32; halved
// coefficients); past x = 10 the exponential is 0 in fp32 anyway.
__device__ __forceinline__ float normal_tail(float z, float* expo) {
  float t, e;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(__fmaf_rn(0.311126984f, fabsf(z), 1.0f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(__fmul_rn(-0.721347520f, z), z)));
  float p = 0.0356116086f;
  p = __fmaf_rn(p, t, -0.1389733999f);
  p = __fmaf_rn(p, t, 0.1483426839f);
  p = __fmaf_rn(p, t, -0.0100893658f);
  p = __fmaf_rn(p, t, 0.1079056114f);
  p = __fmaf_rn(p, t, 0.1086569279f);
  p = __fmaf_rn(p, t, 0.1244355664f);
  p = __fmaf_rn(p, t, 0.1241104752f);
  *expo = e;
  return __fmul_rn(__fmul_rn(p, t), e);
}

template <bool FAST>
__device__ __forceinline__ float act_gelu(float z) {
  if constexpr (FAST) {
    float e;
    const float tail = normal_tail(z, &e);
    return __fmul_rn(z, z < 0.0f ? tail : __fsub_rn(1.0f, tail));
  } else {
    // z Phi(z); erfc keeps the relative precision of the lower tail
    return __fmul_rn(__fmul_rn(0.5f, z), erfcf(__fmul_rn(-0.70710678118654752f, z)));
  }
}
template <bool FAST>
__device__ __forceinline__ float act_apply(int act, float z) {
  switch (act) {
    case BL_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays
    case BL_ACT_RELU2: {
      const float p = z < 0.0f ? 0.0f : z;
      return __fmul_rn(p, p);
    }
    case BL_ACT_SILU: return act_silu<FAST>(z);
    case BL_ACT_GELU: return act_gelu<FAST>(z);
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

// One output of column n (of the whole matrix) at element o of y (fp32 or bf16).
__device__ __forceinline__ void epilogue_store(const Epilogue& ep, void* y, int ydt, int64_t o, int64_t n, int acc,
                                               float cf) {
  float v = __fmul_rn(__int2float_rn(acc), cf);
  v = __fadd_rn(v, ep.bias != nullptr ? __ldcg(ep.bias + n) : 0.0f);
  if (ep.pre != nullptr) store_out(ep.pre, ydt, o, v);
  v = ydt == BL_BF16 ? act_apply<true>(ep.act, v) : act_apply<false>(ep.act, v);
  if (ep.res != nullptr) v = __fadd_rn(v, load_out(ep.res, ydt, o));
  store_out(y, ydt, o, v);
}

// act in place over NC values (fp32 bits): one unrolled loop per activation, the
// choice is uniform and made once
template <int NC, bool FAST>
__device__ __forceinline__ void epilogue_act(int act, uint32_t (&acc)[NC]) {
  auto all = [&](auto f) {
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[j] = __float_as_uint(f(__uint_as_float(acc[j])));
  };
  switch (act) {
    case BL_ACT_RELU: all([](float z) { return act_apply<FAST>(BL_ACT_RELU, z); }); break;
    case BL_ACT_RELU2: all([](float z) { return act_apply<FAST>(BL_ACT_RELU2, z); }); break;
    case BL_ACT_SILU: all([](float z) { return act_silu<FAST>(z); }); break;
    case BL_ACT_GELU: all([](float z) { return act_gelu<FAST>(z); }); break;
    default: break;
  }
}

}  // namespace bl
