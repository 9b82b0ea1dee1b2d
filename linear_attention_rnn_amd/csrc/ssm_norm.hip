// Between two blocks: the norm after a block, its gate, the scaled addition to
// the residual stream and the norm before the next block, in one pass:
//
//   n = x / rms(x) post  (or x),  h = residual + scale act(gate) n  (rounded to its type),
//   y = h / rms(h) pre
//
// and the gradients, with H = dh + the pre norm's gradient of dy:
//
//   dresidual = H,  dgate = scale act'(gate) H n  (summed over the rows that share a gate),
//   dpost = sum scale act H x / rms(x),  dx = the post norm's gradient of scale act H post.
//
// Bound by the bytes of the rows, each read and written once: 32768 rows of 2048 with
// a gate for each, bfloat16, 123 us, 5.5 TB/s; gradients of 16384 x 1024 with a gate for
// each sequence 53 us, 3.8 TB/s with the launch that adds up the sums.  A row stays in registers between its sums and its outputs, laid over its threads as in the
// norms of the linear-attention layer: TPR threads, NV pieces of 8 columns each.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"

namespace ssm {
namespace {

using linattn::over_row;
using linattn::pair;

// The gate's factor and, in the gradients, its derivative.
__device__ __forceinline__ float act_of(Activation act, float g) {
  return act == kNone ? g : act == kSilu ? g * sigmoid(g) : sigmoid(g);
}
__device__ __forceinline__ void act_and_slope(Activation act, float g, float& value, float& slope) {
  const float s = sigmoid(g);
  value = act == kNone ? g : act == kSilu ? g * s : s;
  slope = act == kNone ? 1.f : act == kSilu ? s * fmaf(g, 1.f - s, 1.f) : s * (1.f - s);
}

template <int TPR, int NV, bool BF>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_kernel(BlockNorm a) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  __shared__ float lds[2][16];
  const int at = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;   // all threads of a row together
  const int64_t base = row * a.C, gbase = a.gate ? row / a.gate_rows * a.C : 0;
  Raw8<BF> rx[NV], rr[NV], rg[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
    rx[v].clear();
    rr[v].clear();
    rg[v].clear();
    if (c < a.C) {
      rx[v].load(a.x, base + c);
      if (a.residual) rr[v].load(a.residual, base + c);
      if (a.gate) rg[v].load(a.gate, gbase + c);
    }
  }
  float h[NV][8];
  float r = 1.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) rx[v].get(h[v]);
  if (a.post) {
    float sum = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[v][j], h[v][j], sum);
    r = 1.f / sqrtf(over_row<TPR, false>(sum, lds[0]) / (float)a.C + a.eps);
  }
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
    float q[8];
    if (a.post && c < a.C) {
      get8<false>(a.post, c, q);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * r * q[j];
    }
    if (a.gate) {
      rg[v].get(q);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] *= act_of(a.act, q[j]);
    }
    rr[v].get(q);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[v][j] = a.residual ? fmaf(a.scale, h[v][j], q[j]) : a.scale * h[v][j];
    if constexpr (BF) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u = pair(h[v][2 * j], h[v][2 * j + 1]);
        h[v][2 * j] = __uint_as_float(u << 16);
        h[v][2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
      }
    }
    if (c < a.C) {
      put8<BF>(a.h, base + c, h[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(h[v][j], h[v][j], sum);
    }
  }
  if (!a.pre) return;
  r = 1.f / sqrtf(over_row<TPR, false>(sum, lds[1]) / (float)a.C + a.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
    if (c >= a.C) continue;
    float q[8];
    get8<false>(a.pre, c, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * r * q[j];
    put8<BF>(a.y, base + c, h[v]);
  }
}

// Threads of a row and its pieces a thread.  A row of one wave needs no exchange
// through LDS: up to two pieces a thread (us, one wave / four: 32768 rows of 1024 columns 64 /
// 79, of 768 47 / 74; gradients of 16384 of 1024 51 / 118), not four (32768 of 2048 131 / 122,
// gradients of 16384 of 2048 158 / 132).  Wider ones by four waves up to 4096 columns (four
// / eight: 32768 of 4096 244 / 268, gradients of 8192 of 4096 112 / 165), by eight up to 8192
// (four / eight: 8192 of 8192 133 / 124, gradients of 4096 184 / 137; sixteen: 126), then by
// sixteen, the gradients, whose sums fill the registers, by eight.
struct Shape {
  int tpr, nv;
};
Shape shape_of(int64_t C, bool back) {
  const int64_t pieces = C / 8;
  const int tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 512 ? 256 : pieces <= 1024 || back ? 512 : 1024;
  const int64_t need = (pieces + tpr - 1) / tpr;
  return {tpr, need <= 1 ? 1 : need <= 2 ? 2 : 4};
}

// ---- gradients.  A workgroup walks over the rows of one unit, at most
// kUnitRows for each of the rows it holds at a time, that share a gate (or, with
// a gate for every row, any), and leaves its columns' sums, [units][sums][C]:
// float32 chains of at most kUnitRows rows, added up in 64 bits.
constexpr int kUnitRows = 32;

struct Units {
  int64_t span;      // rows whose units are counted together: those of a gate, or all
  int64_t per;       // units of a span
  int rows;          // of a unit
  int64_t units;
  int sums;          // columns' sums of a unit: of post, pre and a shared gate, as far as there are any
  int post, pre, gate;   // their places, -1: none
};

Units units_of(const BlockNorm& a) {
  Units u;
  const bool shared = a.gate && a.gate_rows > 1;
  u.span = shared ? a.gate_rows : a.rows;
  // Two workgroups for each CU where there are rows for them, one of eight waves
  // (us, one / two: 2048 rows of 8192 columns 76.5 / 88.5, 1024 of 16384 99 / 124;
  // 16384 of 1024, four waves, 75 / 51).
  const int tpr = shape_of(a.C, true).tpr, side = tpr >= 256 ? 1 : 256 / tpr;
  const int64_t all = (tpr >= 512 ? 256 : 512) * side, turns = (a.rows + all - 1) / all;
  u.rows = (int)(turns < 1 ? 1 : turns > kUnitRows ? kUnitRows : turns) * side;
  u.per = u.span ? (u.span + u.rows - 1) / u.rows : 0;
  u.units = u.span ? a.rows / u.span * u.per : 0;
  u.sums = 0;
  u.post = a.post ? u.sums++ : -1;
  u.pre = a.pre ? u.sums++ : -1;
  u.gate = shared ? u.sums++ : -1;
  return u;
}

template <int TPR, int NV, bool BF>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void block_norm_bwd_kernel(BlockNorm a, Units u, float* part) {
  constexpr int NT = TPR > 256 ? TPR : 256, RW = NT / TPR;
  __shared__ float lds[2][4][16];
  __shared__ float join[RW > 1 ? RW : 1][RW > 1 ? TPR * NV * 8 : 1];
  const int at = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int64_t first = blockIdx.x / u.per * u.span;
  const int64_t begin = first + blockIdx.x % u.per * u.rows;
  const int64_t end = begin + u.rows < first + u.span ? begin + u.rows : first + u.span;
  float dpost[NV][8], dpre[NV][8], dgate[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) dpost[v][j] = dpre[v][j] = dgate[v][j] = 0.f;
  // Both weights stay in registers up to two pieces a thread: read again for every
  // row they are two thirds of what comes through the first-level cache (16384 x
  // 1024 bfloat16 with a gate for each sequence, us, 61.0 / 51.5).  Four pieces, which only rows of
  // more than 8192 columns take, spill without them already: 14 registers of bfloat16 rows, 105 of float32 ones.
  constexpr bool HELD = NV <= 2;
  float wpost[HELD ? NV : 1][8], wpre[HELD ? NV : 1][8];
  const auto weight = [&](const float* from, int v, float(&q)[8]) {
    const int c = (v * TPR + at) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = 1.f;
    if (from && c < a.C) get8<false>(from, c, q);
  };
  if constexpr (HELD)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      weight(a.post, v, wpost[v]);
      weight(a.pre, v, wpre[v]);
    }
  // every wave of a workgroup makes the same turns where rows are shared by waves (RW == 1)
  int turn = 0;
  for (int64_t row = begin + slot; row < end; row += RW, turn ^= 1) {
    const int64_t base = row * a.C, gbase = a.gate ? row / a.gate_rows * a.C : 0;
    Raw8<BF> rx[NV], rh[NV], ry[NV], rd[NV], rg[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      rx[v].clear();
      rh[v].clear();
      ry[v].clear();
      rd[v].clear();
      rg[v].clear();
      if (c < a.C) {
        rx[v].load(a.x, base + c);
        if (a.pre) {
          rh[v].load(a.h, base + c);
          ry[v].load(a.dy, base + c);
        }
        if (a.dh) rd[v].load(a.dh, base + c);
        if (a.gate) rg[v].load(a.gate, gbase + c);
      }
    }
    float hh = 0.f, hd = 0.f, xx = 0.f, xd = 0.f;
    float H[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      rd[v].get(H[v]);
      float x[8], h[8], d[8];
      if (a.post) {
        rx[v].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) xx = fmaf(x[j], x[j], xx);
      }
      if (a.pre && c < a.C) {
        rh[v].get(h);
        ry[v].get(d);
        if constexpr (!HELD) weight(a.pre, v, wpre[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hh = fmaf(h[j], h[j], hh);
          hd = fmaf(h[j], d[j] * wpre[HELD ? v : 0][j], hd);
        }
      }
    }
    if (a.pre) {
      hh = over_row<TPR, false>(hh, lds[turn][0]);
      hd = over_row<TPR, false>(hd, lds[turn][1]);
    }
    if (a.post) xx = over_row<TPR, false>(xx, lds[turn][2]);
    const float rp = 1.f / sqrtf(hh / (float)a.C + a.eps), rq = 1.f / sqrtf(xx / (float)a.C + a.eps);
    const float f = rp * (rp * (hd / (float)a.C));   // (rp^2 may pass the range where hd is small or zero)
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      if (c >= a.C) continue;
      float x[8];
      if (a.pre) {
        float h[8], d[8];
        rh[v].get(h);
        ry[v].get(d);
        if constexpr (!HELD) weight(a.pre, v, wpre[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dpre[v][j] = fmaf(d[j], h[j] * rp, dpre[v][j]);
          H[v][j] = fmaf(rp, d[j] * wpre[HELD ? v : 0][j] - h[j] * f, H[v][j]);
        }
      }
      if (a.dresidual) put8<BF>(a.dresidual, base + c, H[v]);
#pragma unroll
      for (int j = 0; j < 8; ++j) H[v][j] *= a.scale;
      rx[v].get(x);
      if constexpr (!HELD) weight(a.post, v, wpost[0]);
      if (a.gate) {
        float g[8], dg[8];
        rg[v].get(g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float value, slope;
          act_and_slope(a.act, g[j], value, slope);
          dg[j] = H[v][j] * (a.post ? x[j] * rq * wpost[HELD ? v : 0][j] : x[j]) * slope;
          H[v][j] *= value;
        }
        if (u.gate < 0) {
          put8<BF>(a.dgate, base + c, dg);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) dgate[v][j] += dg[j];
        }
      }
      if (a.post)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          dpost[v][j] = fmaf(H[v][j], x[j] * rq, dpost[v][j]);
          H[v][j] *= wpost[HELD ? v : 0][j];
          xd = fmaf(x[j], H[v][j], xd);
        }
    }
    float e = 0.f;
    if (a.post) e = rq * (rq * (over_row<TPR, false>(xd, lds[turn][3]) / (float)a.C));
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      if (c >= a.C) continue;
      if (a.post) {
        float x[8];
        rx[v].get(x);
#pragma unroll
        for (int j = 0; j < 8; ++j) H[v][j] = rq * (H[v][j] - x[j] * e);
      }
      put8<BF>(a.dx, base + c, H[v]);
    }
  }
  const auto leave = [&](const float(&d)[NV][8], int place) {
    if (place < 0) return;
    float* to = part + ((int64_t)blockIdx.x * u.sums + place) * a.C;
    if constexpr (RW > 1) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < NV; ++v) put8<false>(join[slot], (v * TPR + at) * 8, d[v]);
      __syncthreads();
      for (int c = threadIdx.x; c < a.C; c += NT) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < RW; ++i) s += join[i][c];
        to[c] = (float)s;
      }
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * TPR + at) * 8;
        if (c < a.C) put8<false>(to, c, d[v]);
      }
    }
  };
  leave(dpost, u.post);
  leave(dpre, u.pre);
  leave(dgate, u.gate);
}

// One vector of C columns added up over `count` units from unit `first` of each
// span on, in 64 bits: 16 interleaved shares of 16 columns.
__device__ __forceinline__ double unit_sum(const float* part, const Units& u, int place, int64_t first, int64_t count,
                                           int64_t C, int64_t col, double (*lds)[17]) {
  const int share = threadIdx.x / 16;
  double s = 0.0;
  if (col < C)
#pragma unroll 8
    for (int64_t i = share; i < count; i += 16) s += part[((first + i) * u.sums + place) * C + col];
  __syncthreads();
  lds[share][threadIdx.x % 16] = s;
  __syncthreads();
  s = 0.0;
  if (threadIdx.x < 16)
#pragma unroll
    for (int i = 0; i < 16; ++i) s += lds[i][threadIdx.x];
  return s;
}

// blockIdx.y: 0 dpost, 1 dpre, from 2 on the rows of dgate.
template <bool BF>
__global__ __launch_bounds__(256) void block_norm_sum_kernel(BlockNorm a, Units u, const float* part) {
  __shared__ double lds[16][17];
  const int64_t col = (int64_t)blockIdx.x * 16 + threadIdx.x % 16;
  const bool mine = threadIdx.x < 16 && col < a.C;
  if (blockIdx.y < 2) {
    const int place = blockIdx.y == 0 ? u.post : u.pre;
    if (place < 0) return;
    const double s = unit_sum(part, u, place, 0, u.units, a.C, col, lds);
    if (mine) (blockIdx.y == 0 ? a.dpost : a.dpre)[col] = (float)s;
    return;
  }
  const int64_t gates = a.rows / a.gate_rows;
  for (int64_t g = blockIdx.y - 2; g < gates; g += gridDim.y - 2) {
    const double s = unit_sum(part, u, u.gate, g * u.per, u.per, a.C, col, lds);
    if (!mine) continue;
    if constexpr (BF)
      static_cast<uint16_t*>(a.dgate)[g * a.C + col] = (uint16_t)pair((float)s, 0.f);
    else
      static_cast<float*>(a.dgate)[g * a.C + col] = (float)s;
  }
}

template <int TPR, int NV>
void launch(const BlockNorm& a, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  const dim3 grid((unsigned)((a.rows + NT / TPR - 1) / (NT / TPR)));
  hipLaunchKernelGGL((a.bf16 ? block_norm_kernel<TPR, NV, true> : block_norm_kernel<TPR, NV, false>), grid, dim3(NT), 0, s, a);
}
template <int TPR, int NV>
void launch_bwd(const BlockNorm& a, const Units& u, float* part, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  hipLaunchKernelGGL((a.bf16 ? block_norm_bwd_kernel<TPR, NV, true> : block_norm_bwd_kernel<TPR, NV, false>),
                     dim3((unsigned)u.units), dim3(NT), 0, s, a, u, part);
}

}  // namespace

hipError_t enqueue_block_norm(const BlockNorm& a, hipStream_t s) {
  const Shape f = shape_of(a.C, false);
  const auto go = f.tpr == 8     ? launch<8, 1>
                  : f.tpr == 16  ? launch<16, 1>
                  : f.tpr == 32  ? launch<32, 1>
                  : f.tpr == 64  ? (f.nv == 1 ? launch<64, 1> : launch<64, 2>)
                  : f.tpr == 256 ? (f.nv == 1 ? launch<256, 1> : launch<256, 2>)
                  : f.tpr == 512 ? launch<512, 2>
                                 : launch<1024, 2>;
  go(a, s);
  return hipGetLastError();
}

size_t block_norm_bwd_workspace_bytes(const BlockNorm& a) {
  const Units u = units_of(a);
  return (size_t)u.units * u.sums * a.C * 4;
}

hipError_t enqueue_block_norm_bwd(const BlockNorm& a, void* workspace, hipStream_t s) {
  const Units u = units_of(a);
  float* part = static_cast<float*>(workspace);
  const Shape f = shape_of(a.C, true);
  const auto go = f.tpr == 8     ? launch_bwd<8, 1>
                  : f.tpr == 16  ? launch_bwd<16, 1>
                  : f.tpr == 32  ? launch_bwd<32, 1>
                  : f.tpr == 64  ? (f.nv == 1 ? launch_bwd<64, 1> : launch_bwd<64, 2>)
                  : f.tpr == 256 ? (f.nv == 1 ? launch_bwd<256, 1> : launch_bwd<256, 2>)
                                 : (f.nv <= 2 ? launch_bwd<512, 2> : launch_bwd<512, 4>);
  if (u.units) go(a, u, part, s);
  const int64_t gates = u.gate < 0 ? 0 : a.rows / a.gate_rows;
  const dim3 grid((unsigned)((a.C + 15) / 16), (unsigned)(2 + (gates < 4096 ? gates : 4096)));
  if (u.sums) hipLaunchKernelGGL((a.bf16 ? block_norm_sum_kernel<true> : block_norm_sum_kernel<false>), grid, dim3(256), 0, s, a, u, part);
  return hipGetLastError();
}

}  // namespace ssm
