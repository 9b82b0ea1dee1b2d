// Device helpers of the selective state space layer's kernels: tokens of a
// sequence, softplus, SiLU, lane exchanges.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rows.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

using linattn::get8;
using linattn::put8;
using linattn::Raw8;

constexpr float kLog2e = 1.44269504088896340736f;

// Tokens of sequence b that count.
__device__ __forceinline__ int64_t tokens_of(const int32_t* lengths, int64_t b, int64_t T) {
  if (!lengths) return T;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n < T ? n : T;
}

// e^x to a few units of 2^-24 at any x: the product with log2 e carries its rounding.
__device__ __forceinline__ float exp_whole(float x) {
  const float t = x * kLog2e;
  const float lo = fmaf(x, kLog2e, -t) + x * 1.925963033500011e-8f;   // log2 e = kLog2e + 1.93e-8
  const float e = __builtin_amdgcn_exp2f(t);
  return fabsf(lo) < 1.f ? fmaf(e, lo * 0.69314718f, e) : e;          // (not where t is infinite)
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|), and its derivative
// 1 / (1 + exp(-v)).  log(1 + e) = 2 atanh(s) with s = e / (2 + e) <= 1/3: the
// series to s^15 leaves 2^-27 of it, and small e lose nothing.
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_whole(-fabsf(v));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = fmaf(q, 2.f / 15.f, 2.f / 13.f);
  p = fmaf(p, q, 2.f / 11.f);
  p = fmaf(p, q, 2.f / 9.f);
  p = fmaf(p, q, 2.f / 7.f);
  p = fmaf(p, q, 2.f / 5.f);
  p = fmaf(p, q, 2.f / 3.f);
  return fmaxf(v, 0.f) + fmaf(p * q, s, 2.f * s);
}

__device__ __forceinline__ float sigmoid(float v) {
  const float e = exp_whole(-fabsf(v));
  const float r = __builtin_amdgcn_rcpf(1.f + e);
  return v >= 0.f ? r : e * r;
}

// The value of the lane N places before, or behind, in a row of 16 lanes; 0
// where there is none.
template <int N>
__device__ __forceinline__ float before(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x110 | N, 0xF, 0xF, true));
}
template <int N>
__device__ __forceinline__ float behind(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x100 | N, 0xF, 0xF, true));
}

// ... `edge` where there is none.
__device__ __forceinline__ float before_or(float x, float edge) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(edge), __float_as_int(x), 0x111, 0xF, 0xF, false));
}
__device__ __forceinline__ float behind_or(float x, float edge) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(edge), __float_as_int(x), 0x101, 0xF, 0xF, false));
}

// a of the lower and a of the upper half of the wave added up in the lower
// half, b's in the upper half.
__device__ __forceinline__ float halves_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// ... of the even and odd rows of 16 lanes, in the even and odd rows.
__device__ __forceinline__ float rows16_sum(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

}  // namespace
}  // namespace ssm
