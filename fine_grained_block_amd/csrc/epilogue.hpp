// epilogue.hpp — what the epilogue GEMM does to a finished sum: y = act(sum + bias) + residual, in
// float32, rounded once when y is stored.
//
//   relu       max(v, 0)
//   gelu       v * Phi(v): with h = Phi(-|v|) = erfc(|v| / sqrt 2) / 2, v h for v < 0 and v - v h
//              above, which keeps the relative accuracy of the negative tail where 1 + erf cancels.
//              h = exp(-v^2 / 2) t Q(t), t = 1 / (1 + 0.42 |v| / sqrt 2): erfcx(x) / t is smooth in t; Q
//              is its degree-7 fit over 0 <= x <= 9.5 (beyond, the exponential is below float32) by
//              least squares reweighted until the largest relative error is least, 1.7e-7; rounded to
//              float32, largest relative error 2.0e-7 with the constants as they are; gelu is within 1e-6
//              relative for |v| < 4.
//              (Two transcendentals and 8 FMAs; with the library's erfc the 4096 x 28672 x 4096 tiles
//              took 511 us, 396 without an activation.)
//   gelu_tanh  v/2 * (1 + tanh u) = v * sigmoid(2u), u = sqrt(2/pi) (v + 0.044715 v^3)
//   silu       v * sigmoid(v)
// sigmoid(z) = 1 / (1 + exp(-z)): for z -> -inf the exponential is +inf and the quotient 0, so no
// finite v overflows into a NaN.  A NaN stays one in every form, +inf stays +inf, and -inf gives what the
// formulas do: 0 for relu, NaN (-inf * 0) for the others.
#pragma once
#include "gemm_common.hpp"
#include "internal.h"

namespace fgb {

__device__ __forceinline__ float sigmoidf(float z) { return __builtin_amdgcn_rcpf(1.0f + __expf(-z)); }

__device__ __forceinline__ float gelu_erf(float v) {
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.29698485f, fabsf(v), 1.0f));
  float q = 0.0351071656f;
  q = __builtin_fmaf(q, t, -0.160092995f);
  q = __builtin_fmaf(q, t, 0.220275044f);
  q = __builtin_fmaf(q, t, -0.065206036f);
  q = __builtin_fmaf(q, t, 0.134340614f);
  q = __builtin_fmaf(q, t, 0.0973725319f);
  q = __builtin_fmaf(q, t, 0.119791359f);
  q = __builtin_fmaf(q, t, 0.118412219f);
  // (min: v h is 0 long before 16 in the upper tail, and at +inf it would be inf * 0)
  const float h = fminf(v, 16.0f) * (q * t * __builtin_amdgcn_exp2f(v * v * -0.72134752f));
  return v < 0.0f ? h : v - h;
}

__device__ __forceinline__ float gelu_tanh(float v) {
  const float u = 0.79788456080286536f * __builtin_fmaf(0.044715f * v * v, v, v);
  return v * sigmoidf(2.0f * u);
}

// act is uniform over the launch: f(value function) runs once, for the launch's activation.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
  if (act == kActSilu) f([](float v) { return v * sigmoidf(v); });
  else if (act == kActGeluTanh) f([](float v) { return gelu_tanh(v); });
  else if (act == kActGelu) f([](float v) { return gelu_erf(v); });
  else if (act == kActRelu) f([](float v) { return v < 0.0f ? 0.0f : v; });  // (a maximum would turn NaN into 0)
}
template <int W>
__device__ __forceinline__ void activate(int act, float (&v)[W]) {
  with_activation(act, [&](auto fn) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = fn(v[i]);
  });
}

// 4 consecutive values of a bf16 (dtype 0) or float32 (dtype 1) array from element idx, a multiple of 4,
// as float32.
__device__ __forceinline__ void load_values(const void* p, int dtype, int64_t idx, float (&v)[4]) {
  if (dtype == 0) {
    const v2u t = gload<v2u>(reinterpret_cast<const uint16_t*>(p) + idx);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = bf16_lo(t[i]);
      v[2 * i + 1] = bf16_hi(t[i]);
    }
  } else {
    const v4f t = gload<v4f>(reinterpret_cast<const float*>(p) + idx);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t[i];
  }
}

// 4 consecutive outputs of row m from column n.
__device__ __forceinline__ void epilogue_values(const Epilogue& e, int64_t m, int64_t n, float (&v)[4]) {
  if (e.bias != nullptr) {
    float b[4];
    load_values(e.bias, e.bias_dtype, n, b);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += b[i];
  }
  activate<4>(e.act, v);
  if (e.residual != nullptr) {
    float r[4];
    load_values(e.residual, e.residual_dtype, m * e.ldr + n, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += r[i];
  }
}

// Store four consecutive outputs of one token, with the epilogue where the launch has one.
template <int OUT, typename Args>
__device__ __forceinline__ void store_out(const Args& p, int64_t m, int64_t n, v4f a) {
  if constexpr (Args::kEpilogue) {
    float v[4] = {a[0], a[1], a[2], a[3]};
    epilogue_values(p.ep, m, n, v);
    a = v4f{v[0], v[1], v[2], v[3]};
  }
  store4<OUT>(p.y, p.ldy, m, n, a);
}

}  // namespace fgb
