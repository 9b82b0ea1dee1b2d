// The short causal convolution of every channel over its last W inputs, with
// its activation, the state it leaves and its gradients:
//
//   p_t = bias + sum_j w_j x_{t-W+1+j},  y = silu(p) or p
//   dp = dy silu'(p),  dx_t = sum_j w_j dp_{t+W-1-j},  dw_j = sum_t dp_t x_{t-W+1+j}
//
// where the rows before the first token are those of the state.  Bound by the bytes
// of x and y (and dy and dx), read once but for the rows in front of each run: 8 x 4096
// tokens of 2048 channels of bfloat16 55 us, 4.9 TB/s; gradients of 4 x 4096 58 us, 3.5
// TB/s with the second launch (the activation's slope is as long a wait for the vector unit, and runs of 32
// tokens work out 36 of them).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"

namespace ssm {
namespace {

constexpr int NTH = 256;
constexpr int kAhead = 4;   // tokens whose loads are in flight

// Threads lie side by side over `across` pieces of PC channels (a power of two up
// to 64) and the rest of a workgroup over runs of tokens; each walks its run
// with the last W - 1 inputs in registers.
struct ConvPlan {
  int across, pieces, blocks;   // threads over channels, pieces of PC channels, workgroups over them
  int run;                      // tokens of a run
  int64_t runs, groups;         // runs of a sequence (one at least), workgroups over them
};

struct Place {
  int piece;
  int64_t b, run;
  bool live;
};

__device__ __forceinline__ Place place_of(const ConvPlan& p) {
  const int64_t id = blockIdx.x;
  const int block = (int)(id % p.blocks);
  const int64_t g = id / p.blocks;
  Place at;
  at.piece = block * p.across + threadIdx.x % p.across;
  at.b = g / p.groups;
  at.run = g % p.groups * (NTH / p.across) + threadIdx.x / p.across;
  at.live = at.piece < p.pieces && at.run < p.runs;
  return at;
}

// Weights of PC channels, [W][PC].
template <int W, int PC>
__device__ __forceinline__ void get_weights(const float* weight, int64_t c, float (&w)[W][PC]) {
  float f[PC * W];
  if constexpr (PC * W % 4 == 0) {
#pragma unroll
    for (int i = 0; i < PC * W; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(weight + c * W + i);
      f[i] = q.x, f[i + 1] = q.y, f[i + 2] = q.z, f[i + 3] = q.w;
    }
  } else {
    static_assert(PC % 2 == 0, "pairs of adjacent weights");
#pragma unroll
    for (int i = 0; i < PC * W; i += 2) {
      const float2 q = *reinterpret_cast<const float2*>(weight + c * W + i);
      f[i] = q.x, f[i + 1] = q.y;
    }
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
#pragma unroll
    for (int k = 0; k < PC; ++k) w[j][k] = f[k * W + j];
}

// Row i of the state followed by x, with i counted from the state's first row.
template <int W, bool BF, int PC>
__device__ __forceinline__ Raw<BF, PC> window_row(const Conv& a, int64_t b, int64_t c, int64_t i, int64_t n) {
  Raw<BF, PC> r;
  r.clear();
  if (i < W - 1) {
    if (a.s_in) r.load(a.s_in, (b * (W - 1) + i) * a.D + c);
  } else if (i - (W - 1) < n) {
    r.load(a.x.p, b * a.x.b + (i - (W - 1)) * a.x.t + c);
  }
  return r;
}

template <int W, bool BF, int PC>
__global__ __launch_bounds__(NTH) void conv_kernel(Conv a, ConvPlan p) {
  const Place at = place_of(p);
  if (!at.live) return;
  const int64_t b = at.b, c = (int64_t)at.piece * PC, n = tokens_of(a.lengths, b, a.T);
  float w[W][PC], bias[PC], x[W - 1 + kAhead][PC];
  get_weights<W, PC>(a.weight, c, w);
#pragma unroll
  for (int k = 0; k < PC; ++k) bias[k] = 0.f;
  if (a.bias)
#pragma unroll
    for (int k = 0; k < PC; ++k) bias[k] = a.bias[c + k];
  const int64_t t0 = at.run * p.run, t1 = t0 + p.run < a.T ? t0 + p.run : a.T;
  // The state that is left, before this run writes any: s_out may be s_in, which
  // no other run reads.
  Raw<BF, PC> left[W - 1];
  if (at.run == 0 && a.s_out)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) left[j] = window_row<W, BF, PC>(a, b, c, n + j, n);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) window_row<W, BF, PC>(a, b, c, t0 + j, n).get(x[j]);
  if (at.run == 0 && a.s_out)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) left[j].store(a.s_out, (b * (W - 1) + j) * a.D + c);
  Raw<BF, PC> next[kAhead];
  const auto load = [&](int64_t t) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      next[i].clear();
      if (t + i < n) next[i].load(a.x.p, b * a.x.b + (t + i) * a.x.t + c);
    }
  };
  load(t0);
  for (int64_t t = t0; t < t1; t += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i].get(x[W - 1 + i]);
    if (t + kAhead < t1) load(t + kAhead);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float y[PC];
#pragma unroll
      for (int k = 0; k < PC; ++k) {
        float s = bias[k];
#pragma unroll
        for (int j = 0; j < W; ++j) s = fmaf(w[j][k], x[i + j][k], s);
        if (a.silu) s *= sigmoid<BF>(s);
        y[k] = t + i < n ? s : 0.f;
      }
      Raw<BF, PC> r;
      r.set(y);
      if (t + i < t1) r.store(const_cast<void*>(a.y.p), b * a.y.b + (t + i) * a.y.t + c);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int k = 0; k < PC; ++k) x[j][k] = x[kAhead + j][k];
  }
}

// A run's gradients.  At token s, dp_s gives the gradient of the row W - 1
// before it (of the state's row s in the first run, which goes on to the last of
// those), and ds_out joins it from the row on that the state kept.  The sums of
// dw and dbias over a run are a float32 chain of run tokens, those of a
// workgroup's runs are 64-bit and go to the workspace, [groups][W + 1][D].
template <int W, bool BF, int PC>
__global__ __launch_bounds__(NTH) void conv_bwd_kernel(Conv a, ConvPlan p, float* part) {
  __shared__ float join[NTH][PC + 1];
  const Place at = place_of(p);
  float dw[W + 1][PC] = {};   // the bias's last
  if (at.live) {
    const int64_t b = at.b, c = (int64_t)at.piece * PC, n = tokens_of(a.lengths, b, a.T);
    const int64_t t0 = at.run * p.run, t1 = t0 + p.run < a.T ? t0 + p.run : a.T;
    float w[W][PC], bias[PC], x[W - 1 + kAhead][PC], dp[W - 1 + kAhead][PC];
    get_weights<W, PC>(a.weight, c, w);
#pragma unroll
    for (int k = 0; k < PC; ++k) bias[k] = 0.f;
    if (a.bias)
#pragma unroll
    for (int k = 0; k < PC; ++k) bias[k] = a.bias[c + k];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      window_row<W, BF, PC>(a, b, c, t0 + j, n).get(x[j]);
#pragma unroll
      for (int k = 0; k < PC; ++k) dp[j][k] = 0.f;
    }
    Raw<BF, PC> xn[kAhead], dn[kAhead];
    const auto load = [&](int64_t s) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        xn[i].clear();
        dn[i].clear();
        if (s + i < n) {
          xn[i].load(a.x.p, b * a.x.b + (s + i) * a.x.t + c);
          dn[i].load(a.dy.p, b * a.dy.b + (s + i) * a.dy.t + c);
        }
      }
    };
    const int64_t last = t1 + W - 1;   // (rows of the next run's dp reach into this one)
    const int64_t end = t1 < n ? t1 : n;   // (behind: no gradient that could meet a row that is not finite)
    load(t0);
    for (int64_t s = t0; s < last; s += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        xn[i].get(x[W - 1 + i]);
        dn[i].get(dp[W - 1 + i]);
      }
      if (s + kAhead < last) load(s + kAhead);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (a.silu) {
#pragma unroll
          for (int k = 0; k < PC; ++k) {
            float v = bias[k];
#pragma unroll
            for (int j = 0; j < W; ++j) v = fmaf(w[j][k], x[i + j][k], v);
            const float g = sigmoid(v);
            dp[W - 1 + i][k] *= g * fmaf(v, 1.f - g, 1.f);
          }
        }
        if (s + i >= n)
#pragma unroll
          for (int k = 0; k < PC; ++k) dp[W - 1 + i][k] = 0.f;   // (a bias that is not finite)
        if (s + i < end)
#pragma unroll
          for (int k = 0; k < PC; ++k) {
#pragma unroll
            for (int j = 0; j < W; ++j) dw[j][k] = fmaf(dp[W - 1 + i][k], x[i + j][k], dw[j][k]);
            dw[W][k] += dp[W - 1 + i][k];
          }
        const int64_t row = s + i;   // of the state followed by x
        if (row < last && (row >= t0 + W - 1 || at.run == 0)) {
          float d[PC];
#pragma unroll
          for (int k = 0; k < PC; ++k) {
            d[k] = 0.f;
#pragma unroll
            for (int j = 0; j < W; ++j) d[k] = fmaf(w[j][k], dp[W - 1 + i - j][k], d[k]);
          }
          if (row >= n + W - 1)
#pragma unroll
            for (int k = 0; k < PC; ++k) d[k] = 0.f;   // (a weight that is not finite)
          if (a.ds_out && row >= n && row - n < W - 1) {
            Raw<BF, PC> r;
            float e[PC];
            r.load(a.ds_out, (b * (W - 1) + row - n) * a.D + c);
            r.get(e);
#pragma unroll
            for (int k = 0; k < PC; ++k) d[k] += e[k];
          }
          Raw<BF, PC> r;
          r.set(d);
          if (row >= W - 1)
            r.store(const_cast<void*>(a.y.p), b * a.y.b + (row - (W - 1)) * a.y.t + c);
          else if (a.ds_in)
            r.store(a.ds_in, (b * (W - 1) + row) * a.D + c);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int k = 0; k < PC; ++k) {
          x[j][k] = x[kAhead + j][k];
          dp[j][k] = dp[kAhead + j][k];
        }
    }
  }
  const int64_t group = blockIdx.x / p.blocks;
  const int c0 = (int)(blockIdx.x % p.blocks) * p.across * PC;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int k = 0; k < PC; ++k) join[threadIdx.x][k] = dw[j][k];
    __syncthreads();
    for (int e = threadIdx.x; e < p.across * PC; e += NTH) {
      if (c0 + e >= a.D) continue;
      double s = 0.0;
      for (int r = e / PC; r < NTH; r += p.across) s += join[r][e % PC];
      part[(group * (W + 1) + j) * a.D + c0 + e] = (float)s;
    }
  }
}

// dweight [D, W] and dbias [D] of 16 columns of [W + 1][D]: the workgroups' sums
// in 16 interleaved shares, all in 64 bits.
__global__ __launch_bounds__(256) void conv_sum_kernel(const float* part, float* dweight, float* dbias, int64_t groups,
                                                       int D, int W) {
  __shared__ double lds[16][17];
  const int64_t columns = (int64_t)(W + 1) * D;
  const int64_t col = (int64_t)blockIdx.x * 16 + threadIdx.x % 16;
  const int share = threadIdx.x / 16;
  double s = 0.0;
  if (col < columns)
#pragma unroll 8
    for (int64_t g = share; g < groups; g += 16) s += part[g * columns + col];
  lds[share][threadIdx.x % 16] = s;
  __syncthreads();
  if (threadIdx.x >= 16 || col >= columns) return;
  s = 0.0;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += lds[i][threadIdx.x];
  const int j = (int)(col / D), d = (int)(col % D);
  if (j < W)
    dweight[(int64_t)d * W + j] = (float)s;
  else if (dbias)
    dbias[d] = (float)s;
}

// Channels of a thread.  Us, with 8 / 4: 8 x 4096 tokens of 2048 channels 59.1 / 58.0,
// float32 116 / 106, 512 tokens 8.3 / 7.4.  The gradients keep two windows, the
// weights and their sums, with 8 channels 256 registers and one wave a SIMD: 8 / 4
// / 2, 4 x 4096 tokens 90.3 / 61.7 / 56.6, float32 121 / 96.9 / 90.7.
constexpr int kPiece = 4, kPieceBwd = 2;

// Runs of 16 tokens read 3 rows twice; the gradients also work those out twice, and
// take runs of 32 once there are more than four waves for each SIMD.  Us with 16 / 32: 8 x 4096
// tokens of 2048 channels 55.0 / 57.8, 1 x 4096 9.3 / 10.2; gradients of 1, 2 and 4 x 4096 21.5 / 22.1,
// 35.0 / 30.1, 67.8 / 56.4.
ConvPlan plan_of(const Conv& a, int piece) {
  ConvPlan p;
  p.pieces = a.D / piece;
  p.across = 1;
  while (p.across < 64 && p.across < p.pieces) p.across *= 2;
  p.blocks = (p.pieces + p.across - 1) / p.across;
  const int64_t threads = a.B * p.blocks * p.across;   // of one run
  p.run = piece == kPieceBwd && threads * (a.T / 16) > 262144 ? 32 : 16;
  p.runs = a.T ? (a.T + p.run - 1) / p.run : 1;
  const int side = NTH / p.across;
  p.groups = (p.runs + side - 1) / side;
  return p;
}

template <int W>
void launch_conv(const Conv& a, const ConvPlan& p, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * p.groups * p.blocks));
  hipLaunchKernelGGL((a.bf16 ? conv_kernel<W, true, kPiece> : conv_kernel<W, false, kPiece>), grid, dim3(NTH), 0, s, a, p);
}
template <int W>
void launch_conv_bwd(const Conv& a, const ConvPlan& p, float* part, hipStream_t s) {
  const dim3 grid((unsigned)(a.B * p.groups * p.blocks));
  hipLaunchKernelGGL((a.bf16 ? conv_bwd_kernel<W, true, kPieceBwd> : conv_bwd_kernel<W, false, kPieceBwd>), grid, dim3(NTH), 0, s, a, p, part);
}

}  // namespace

hipError_t enqueue_conv(const Conv& a, hipStream_t s) {
  const ConvPlan p = plan_of(a, kPiece);
  (a.W == 2 ? launch_conv<2> : a.W == 3 ? launch_conv<3> : launch_conv<4>)(a, p, s);
  return hipGetLastError();
}

size_t conv_bwd_workspace_bytes(const Conv& a) {
  const ConvPlan p = plan_of(a, kPieceBwd);
  return (size_t)(a.B * p.groups) * (a.W + 1) * a.D * 4;
}

hipError_t enqueue_conv_bwd(const Conv& a, void* workspace, hipStream_t s) {
  const ConvPlan p = plan_of(a, kPieceBwd);
  float* part = static_cast<float*>(workspace);
  if (a.B) (a.W == 2 ? launch_conv_bwd<2> : a.W == 3 ? launch_conv_bwd<3> : launch_conv_bwd<4>)(a, p, part, s);
  const int64_t columns = (int64_t)(a.W + 1) * a.D;
  hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((columns + 15) / 16)), dim3(256), 0, s, part, a.dweight, a.dbias,
                     a.B * p.groups, a.D, a.W);
  return hipGetLastError();
}

}  // namespace ssm
