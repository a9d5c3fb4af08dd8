// moe_float.h — element types and fp32 functions of the operators that take fp32, bf16 or fp16 tensors.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#pragma clang fp contract(off)

namespace moe {

constexpr float kNegInf = -INFINITY;

// ------------------------------------------------------------ element types
struct bf16_t {
  uint16_t b;
};
template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ float to_f32<_Float16>(_Float16 v) {
  return (float)v;
}
template <>
__device__ __forceinline__ float to_f32<bf16_t>(bf16_t v) {
  return __uint_as_float((uint32_t)v.b << 16);
}
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ _Float16 from_f32<_Float16>(float v) {
  return (_Float16)v;
}
template <>
__device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
  const __bf16 h = (__bf16)v;
  return __builtin_bit_cast(bf16_t, h);
}
// lowest finite value of the type: with NaN and -inf it marks a masked expert
template <class T>
__device__ __forceinline__ float lowest();
template <>
__device__ __forceinline__ float lowest<float>() {
  return -3.402823466e38f;
}
template <>
__device__ __forceinline__ float lowest<_Float16>() {
  return -65504.0f;
}
template <>
__device__ __forceinline__ float lowest<bf16_t>() {
  return __uint_as_float(0xFF7F0000u);
}

// ------------------------------------------------------------ scalar functions
// e^x for x <= 0 to about 1.5 units in the last place: x log2(e) in two parts, the hardware 2^x of the first, the
// second as 1 + lo ln 2. Arguments below -150 give 0 (so do all whose result is below 2^-126).
__device__ __forceinline__ float exp_neg(float x) {
  x = fmaxf(x, -150.0f);
  const float l2e = 1.44269502f, l2e_lo = 1.92596303e-8f;
  const float hi = x * l2e;
  const float lo = fmaf(x, l2e_lo, fmaf(x, l2e, -hi));
  const float r = __builtin_amdgcn_exp2f(hi);
  return fmaf(r, lo * 0.693147182f, r);
}
// s = sigmoid(z) and 1 - s, both without cancellation
__device__ __forceinline__ void sigmoid2(float z, float& s, float& miss) {
  const float a = exp_neg(-fabsf(z));
  const float d = __builtin_amdgcn_rcpf(1.0f + a);
  const float o = a * d;
  s = z >= 0.0f ? d : o;
  miss = z >= 0.0f ? o : d;
}
// sigmoid(z) e^-ref for ref = min(largest z, 0): stays in range where every sigmoid underflows
__device__ __forceinline__ float sigmoid_rel(float z, float ref) {
  const float d = __builtin_amdgcn_rcpf(1.0f + exp_neg(-fabsf(z)));
  return z >= 0.0f ? d : exp_neg(z - ref) * d;
}
// 1 / v to 1 unit in the last place, 0 for an empty sum
__device__ __forceinline__ float safe_rcp(float v) { return v > 0.0f ? __builtin_amdgcn_rcpf(v) : 0.0f; }

}  // namespace moe
