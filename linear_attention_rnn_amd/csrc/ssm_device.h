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

// e^x for x <= 88 to a few units of 2^-24: the exponent's rounding, x - t log 2,
// is a factor of its own.  Below -150 that of -150, which is 0.
__device__ __forceinline__ float exp_whole(float x) {
  x = __builtin_elementwise_maximum(x, -150.f);   // (a NaN stays one)
  const float t = x * kLog2e;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, fmaf(t, -0.69314718055994531f, x), e);
}

// softplus(v) = max(v, 0) + log(1 + e), e = exp(-|v|).  log(1 + e) = 2 atanh(s)
// with s = e / (2 + e) <= 1/3; 2 atanh(s) / s by Chebyshev interpolation over s^2
// up to 1/9, off by 2^-28 of itself, so that small e lose nothing.
__device__ __forceinline__ float softplus(float v) {
  const float e = exp_whole(-fabsf(v));
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = fmaf(q, 0.28174657f, 0.27961419f);
  p = fmaf(p, q, 0.40024854f);
  p = fmaf(p, q, 0.66666316f);
  p = fmaf(p, q, 2.00000001f);
  return fmaf(p, s, __builtin_elementwise_maximum(v, 0.f));
}

// 1 / (1 + exp(-v)).
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.f + exp_whole(__builtin_elementwise_minimum(-v, 88.f)));   // (1 + e^88: as good as infinite)
}
// The factor of a result that is rounded to bfloat16 next (BF): the exponent is
// off by up to |v| 2^-24 of e^-v, which 2^-8 hides; 6 instructions fewer.
template <bool BF>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (BF)
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e));
  else
    return sigmoid(v);
}

// N adjacent values as loaded, 4, 8 or 16 bytes at a time.
template <bool BF, int N>
struct Raw {
  static constexpr int BYTES = N * (BF ? 2 : 4);
  uint32_t q[BYTES / 4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) q[i] = 0;
  }
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const char* at = static_cast<const char*>(p) + i * (BF ? 2 : 4);
    if constexpr (BYTES == 4) {
      q[0] = *reinterpret_cast<const uint32_t*>(at);
    } else if constexpr (BYTES == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(at);
      q[0] = u.x, q[1] = u.y;
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j) {
        const uint4 u = reinterpret_cast<const uint4*>(at)[j];
        q[4 * j] = u.x, q[4 * j + 1] = u.y, q[4 * j + 2] = u.z, q[4 * j + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    char* at = static_cast<char*>(p) + i * (BF ? 2 : 4);
    if constexpr (BYTES == 4) {
      *reinterpret_cast<uint32_t*>(at) = q[0];
    } else if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2*>(at) = make_uint2(q[0], q[1]);
    } else {
#pragma unroll
      for (int j = 0; j < BYTES / 16; ++j)
        reinterpret_cast<uint4*>(at)[j] = make_uint4(q[4 * j], q[4 * j + 1], q[4 * j + 2], q[4 * j + 3]);
    }
  }
  __device__ __forceinline__ void get(float (&x)[N]) const {
#pragma unroll
    for (int j = 0; j < N; ++j)
      x[j] = __uint_as_float(!BF ? q[BF ? 0 : j] : j % 2 ? q[j / 2] & 0xFFFF0000u : q[j / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&x)[N]) {
#pragma unroll
    for (int j = 0; j < BYTES / 4; ++j) q[j] = BF ? linattn::pair(x[BF ? 2 * j : 0], x[BF ? 2 * j + 1 : 0]) : __float_as_uint(x[BF ? 0 : j]);
  }
};

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

// x += that value * by, in one instruction for each (the compiler makes a move
// and a product of it).  A value just written is read by other lanes two wait
// states later.
template <int N, int COUNT>
__device__ __forceinline__ void add_before(float (&x)[COUNT], const float (&by)[COUNT]) {
  static_assert(COUNT % 2 == 0, "two at a time");
#define SSM_ADD(dir)                                                                                              \
  _Pragma("unroll") for (int i = 0; i < COUNT; i += 2) asm(                                                       \
      "s_nop 1\n\tv_fmac_f32_dpp %0, %0, %2 " dir " row_mask:0xf bank_mask:0xf bound_ctrl:1\n\t"                   \
      "v_fmac_f32_dpp %1, %1, %3 " dir " row_mask:0xf bank_mask:0xf bound_ctrl:1"                                 \
      : "+v"(x[i]), "+v"(x[i + 1])                                                                                \
      : "v"(by[i]), "v"(by[i + 1]))
  if constexpr (N == 1) SSM_ADD("row_shr:1");
  if constexpr (N == 2) SSM_ADD("row_shr:2");
  if constexpr (N == 4) SSM_ADD("row_shr:4");
  if constexpr (N == 8) SSM_ADD("row_shr:8");
  if constexpr (N == -1) SSM_ADD("row_shl:1");
  if constexpr (N == -2) SSM_ADD("row_shl:2");
  if constexpr (N == -4) SSM_ADD("row_shl:4");
  if constexpr (N == -8) SSM_ADD("row_shl:8");
#undef SSM_ADD
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
