// Rows of float32 or bfloat16 values in pieces of 8 adjacent columns (16-byte
// loads of bfloat16), and sums over the threads that hold a row: shared by the
// kernels of the norms and of the selective state space layer.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace linattn {
namespace {

template <bool BF>
__device__ __forceinline__ void get8(const void* p, int64_t i, float (&x)[8]) {
  if constexpr (BF) {
    const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(u[j] << 16);
      x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 q = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i + 4 * j);
      x[4 * j] = q.x;
      x[4 * j + 1] = q.y;
      x[4 * j + 2] = q.z;
      x[4 * j + 3] = q.w;
    }
  }
}

// Eight values as loaded, so that rows to come take few registers.
template <bool BF>
struct Raw8 {
  uint4 q[BF ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (BF ? 2 : 4));
    q[0] = at[0];
    if constexpr (!BF) q[1] = at[1];
  }
  __device__ __forceinline__ void clear() {
    q[0] = make_uint4(0, 0, 0, 0);
    if constexpr (!BF) q[1] = q[0];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t u[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (BF) {
        x[2 * j] = __uint_as_float(u[j] << 16);
        x[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
      } else {
        const uint32_t v[4] = {q[BF ? 0 : 1].x, q[BF ? 0 : 1].y, q[BF ? 0 : 1].z, q[BF ? 0 : 1].w};
        x[j] = __uint_as_float(u[j]);
        x[4 + j] = __uint_as_float(v[j]);
      }
    }
  }
};

__device__ __forceinline__ uint32_t pair(float a, float b) {   // bfloat16, nearest even
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

template <bool BF>
__device__ __forceinline__ void put8(void* p, int64_t i, const float (&x)[8]) {
  if constexpr (BF) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
        make_uint4(pair(x[0], x[1]), pair(x[2], x[3]), pair(x[4], x[5]), pair(x[6], x[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i + 4 * j) =
          make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
  }
}

// Sum, or largest value, over the 2^k lanes that hold a group.
template <int LANES, bool MAX>
__device__ __forceinline__ float over_lanes(float x) {
#pragma unroll
  for (int m = 1; m < LANES; m *= 2) {
    const float y = __shfl_xor(x, m, 64);
    x = MAX ? fmaxf(x, y) : x + y;
  }
  return x;
}

// ... over the TPR threads of a row; `lds`: 16 floats that no one else uses.
template <int TPR, bool MAX>
__device__ __forceinline__ float over_row(float x, float* lds) {
  x = over_lanes<(TPR < 64 ? TPR : 64), MAX>(x);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = x;
    __syncthreads();
    x = lds[0];
#pragma unroll
    for (int i = 1; i < TPR / 64; ++i) x = MAX ? fmaxf(x, lds[i]) : x + lds[i];
  }
  return x;
}

}  // namespace
}  // namespace linattn
