// Rotary positions of queries and keys: pair i of a head's first R channels
// is turned by position * freqs[i],  (x, y) -> (x cos - y sin, x sin + y cos).
//
// Bound by the bytes of q and k, read and written once.  The angles of a
// token are the same for all its heads, so a workgroup takes a few tokens,
// puts the cosines and sines of their R / 2 angles into LDS and then streams
// all heads of q and k past them, 16 bytes a load.  32768 tokens of 32 heads
// of 64 channels in bfloat16: 92 us, 5.9 TB/s; one token of 64 sequences 3.6
// us, a launch.
//
// Angles are products of whole positions and float64 frequencies, carried as
// the rounded product and its rounding error and reduced to a part of a turn
// before they are rounded to float32: the quotient by 2 pi is formed with its
// rounding errors (two products), its nearest quarter turn is taken off exactly,
// and what is left, at most 3/16 of a turn, loses 2^-24 of itself.  A position of
// 2^52 is as exact as one of 10 (without the product's error it would be off by
// 2e-4 at 2^40 and by a radian at 2^52).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linattn_internal.h"

namespace linattn {
namespace {

constexpr int NTR = 256;
constexpr int kMaxTokens = 16;     // of a workgroup
constexpr int kMaxAngles = 1024;   // those times R / 2 <= 64
constexpr int kTogether = 2;       // tokens whose loads a thread has in flight
constexpr int kRows = 128;         // rows (tensor, token, head) of a workgroup

__device__ __forceinline__ float2 turn_of(double pos, double freq, bool inverse) {
  constexpr double kInv2Pi = 0.15915494309189535;       // 1 / (2 pi), rounded
  constexpr double kInv2PiLow = -9.839338337591243e-18;  // and what the rounding left
  const double angle = pos * freq, rest = fma(pos, freq, -angle);
  const double t = angle * kInv2Pi, low = fma(angle, kInv2Pi, -t) + fma(angle, kInv2PiLow, rest * kInv2Pi);
  const double k = rint(4.0 * t);
  const float f = (float)(fma(-0.25, k, t) + low);
  float s, c;
  sincospif(2.f * f, &s, &c);
  const int q = (int)(k - 4.0 * floor(0.25 * k));
  const float cs = q & 1 ? s : c, sn = q & 1 ? c : s;
  const float co = q == 1 || q == 2 ? -cs : cs, si = q >= 2 ? -sn : sn;
  return make_float2(co, inverse ? -si : si);
}

__device__ __forceinline__ uint32_t pair(float a, float b) {   // bfloat16, nearest even
  typedef float f2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// N adjacent values as one or two loads or stores of up to 16 bytes.
template <bool BF, int N>
__device__ __forceinline__ void get(const void* p, int64_t i, float (&x)[N]) {
  constexpr int Z = BF ? 2 : 4, W = N * Z / 4 > 0 ? N * Z / 4 : 1;
  uint32_t u[W];
  const char* at = static_cast<const char*>(p) + i * Z;
  if constexpr (N * Z == 2)
    u[0] = *reinterpret_cast<const uint16_t*>(at);
  else
    __builtin_memcpy(u, __builtin_assume_aligned(at, N * Z > 16 ? 16 : N * Z), N * Z);
#pragma unroll
  for (int j = 0; j < N; ++j)
    x[j] = BF ? __uint_as_float(j % 2 ? u[j / 2] & 0xFFFF0000u : u[j / 2] << 16) : __uint_as_float(u[BF ? 0 : j]);
}

template <bool BF, int N>
__device__ __forceinline__ void put(void* p, int64_t i, const float (&x)[N]) {
  constexpr int Z = BF ? 2 : 4, W = N * Z / 4 > 0 ? N * Z / 4 : 1;
  uint32_t u[W];
#pragma unroll
  for (int j = 0; j < W; ++j) u[j] = BF ? pair(x[2 * j < N ? 2 * j : 0], x[2 * j + 1 < N ? 2 * j + 1 : 0]) : __float_as_uint(x[j]);
  char* at = static_cast<char*>(p) + i * Z;
  if constexpr (N * Z == 2)
    *reinterpret_cast<uint16_t*>(at) = (uint16_t)u[0];
  else
    __builtin_memcpy(__builtin_assume_aligned(at, N * Z > 16 ? 16 : N * Z), u, N * Z);
}

// blockIdx.x: a group of `tokens` tokens, whose rows (tensor, head) are worked
// on kTogether tokens at a time.  A piece is N adjacent channels: N / 2 pairs
// in place (interleaved), or N pairs whose halves lie R / 2 apart; N divides
// what a piece must not cross (R, or R / 2).
template <bool BF, bool INTER, int N>
__global__ __launch_bounds__(NTR) void rope_kernel(Rope a, int tokens) {
  __shared__ float2 cs[kMaxAngles];
  __shared__ int64_t base[4][kMaxTokens];   // of a token's rows in q, k, q_out, k_out
  const int half = a.R / 2, tid = threadIdx.x;
  const int64_t n = a.B * a.T, first = (int64_t)blockIdx.x * tokens;
  const int nt = (int)(n - first < tokens ? n - first : tokens);
  for (int e = tid; e < nt * half; e += NTR) {
    const uint32_t tok = (uint32_t)first + e / half;
    const int64_t pos = a.start + (a.positions ? a.positions[tok] : (int32_t)(tok % (uint32_t)a.T));
    cs[e] = turn_of((double)pos, a.freqs[e % half], a.inverse);
  }
  for (int e = tid; e < 4 * nt; e += NTR) {
    const uint32_t tok = (uint32_t)first + e / 4, T = (uint32_t)a.T, b = tok / T, t = tok % T;   // fewer than 2^27 tokens
    const Tensor& x = e % 4 == 0 ? a.q : e % 4 == 1 ? a.k : e % 4 == 2 ? a.q_out : a.k_out;
    base[e % 4][e / 4] = b * x.b + t * x.t;
  }
  __syncthreads();
  // pieces of a row: those that turn, then those that are copied
  const int turning = INTER ? a.R / N : half / N, units = turning + (a.D - a.R) / N;
  const int per = NTR / units, u = tid % units, slot = tid / units;
  if (slot >= per) return;
  const int rows = a.k.p ? 2 * (int)a.H : (int)a.H, items = rows * ((nt + kTogether - 1) / kTogether);
  const bool copy = u >= turning;
  const int c = copy ? a.R + N * (u - turning) : N * u;
  for (int item = slot; item < items; item += per) {
    const int r = item % rows, t0 = item / rows * kTogether;
    const bool isk = r >= a.H;
    const Tensor& x = isk ? a.k : a.q;
    const Tensor& y = isk ? a.k_out : a.q_out;
    const int64_t h = isk ? r - a.H : r, from = h * x.h + c, to = h * y.h + c;
    const int64_t* const fb = base[isk ? 1 : 0];
    const int64_t* const tb = base[isk ? 3 : 2];
    void* const out = const_cast<void*>(y.p);
    // all tokens' loads before the first store
    float p[kTogether][N], q[INTER ? 1 : kTogether][N];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int ti = min(t0 + i, nt - 1);
      get<BF>(x.p, fb[ti] + from, p[i]);
      if constexpr (!INTER) get<BF>(x.p, fb[ti] + from + (copy ? 0 : half), q[i]);
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int ti = t0 + i;
      if (ti >= nt) break;
      if (!copy) {
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            const float2 e = cs[ti * half + N / 2 * u + j];
            const float v = p[i][2 * j], z = p[i][2 * j + 1];
            p[i][2 * j] = v * e.x - z * e.y;
            p[i][2 * j + 1] = v * e.y + z * e.x;
          }
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float2 e = cs[ti * half + N * u + j];
            const float v = p[i][j];
            p[i][j] = v * e.x - q[i][j] * e.y;
            q[i][j] = v * e.y + q[i][j] * e.x;
          }
          put<BF>(out, tb[ti] + to + half, q[i]);
        }
      }
      put<BF>(out, tb[ti] + to, p[i]);
    }
  }
}

template <bool BF, bool INTER>
auto kernel_for(const Rope& a) {
  const int fit = INTER ? a.R : a.R / 2;   // R is even, D a multiple of 8
  return fit % 8 == 0 ? rope_kernel<BF, INTER, 8> : fit % 4 == 0 ? rope_kernel<BF, INTER, 4> : rope_kernel<BF, INTER, INTER ? 2 : 1>;
}

}  // namespace

hipError_t enqueue_rope(const Rope& a, hipStream_t s) {
  const int64_t n = a.B * a.T;
  const int64_t rows = a.k.p ? 2 * a.H : a.H;
  // Tokens of a workgroup: about kRows rows (32768 tokens, 64 rows each, us, with
  // 128 / 256 / 512 / 1024 rows: 97 / 97 / 103 / 111; 16 rows each 22.3 / 23.0 /
  // 22.9 / 23.0), two at a time (2 / 4 / 8 at a time: 92 / 95 / 99), and
  // one where the card would not be filled with 1024 workgroups (64 tokens: 3.6
  // us, 8.1 with sixteen).  From 2^24 tokens on the grid would grow too large.
  int tokens = kMaxTokens;
  while (tokens > 1 && (n / tokens < 1024 || (tokens > kTogether && tokens * rows > kRows && n < (1 << 24)))) tokens /= 2;
  const dim3 grid((unsigned)((n + tokens - 1) / tokens));
  auto* kernel = a.bf16 ? (a.interleaved ? kernel_for<true, true>(a) : kernel_for<true, false>(a))
                        : (a.interleaved ? kernel_for<false, true>(a) : kernel_for<false, false>(a));
  hipLaunchKernelGGL(kernel, grid, dim3(NTR), 0, s, a, tokens);
  return hipGetLastError();
}

}  // namespace linattn
