// Root-mean-square norm of the rows of [rows, C] with the residual's addition
// in front, an output of the inputs' type or of 8-bit codes with scales, and
// its gradients:
//
//   h = x + residual (rounded to its type),  r = 1 / sqrt(mean(h^2) + eps),
//   y = h r w;   dx = r (dy w - h r^2 mean(dy w h)) + dh,  dw = sum dy h r.
//
// Bound by the bytes of the rows, each read and written once: a row stays in
// registers between its sum and its output.  TPR threads hold a row in NV
// pieces of 8 adjacent columns each (16-byte loads of bfloat16), so a wave
// reads 1 KiB at a time.  Sums are float32: a thread's own, then the wave's
// by lane exchanges, then the waves' through LDS.  32768 rows of 2048 columns
// in bfloat16 with a residual: 90 us, 6.0 TB/s; 256 rows with 8-bit codes 4 us,
// a launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linattn_internal.h"
#include "rows.h"

namespace linattn {
namespace {

constexpr float kE4m3Max = 448.f;

// The scale of values up to `top`.  At least the smallest normal float32: top /
// 448 in fewer bits, or rounded to zero, would leave codes past 448.
__device__ __forceinline__ float scale_of(float top) { return top > 0.f ? fmaxf(top / kE4m3Max, 0x1p-126f) : 1.f; }

// OUT: 0 rows of the inputs' type, 1 codes with a scale per 128 columns, 2
// codes with a scale per row.
template <int TPR, int NV, bool BF, int OUT>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_kernel(Norm a) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  __shared__ float lds[2][16];
  const int at = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  if (row >= a.rows) return;   // all threads of a row together
  const int64_t base = row * a.C;
  float h[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
    if (c < a.C)
      get8<BF>(a.x, base + c, h[v]);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = 0.f;
  }
  if (a.residual) {
    float r[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      if (c < a.C)
        get8<BF>(a.residual, base + c, r[v]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) r[v][j] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] += r[v][j];
      if constexpr (BF) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t u = pair(h[v][2 * j], h[v][2 * j + 1]);
          h[v][2 * j] = __uint_as_float(u << 16);
          h[v][2 * j + 1] = __uint_as_float(u & 0xFFFF0000u);
        }
      }
      if (c < a.C) put8<BF>(a.h, base + c, h[v]);
    }
  }
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(h[v][j], h[v][j], sum);
  const float r = 1.f / sqrtf(over_row<TPR, false>(sum, lds[0]) / (float)a.C + a.eps);
  float top = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
    float wt[8];
    if (c < a.C) {
      get8<false>(a.weight, c, wt);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] = h[v][j] * r * wt[j];
    }
    if constexpr (OUT == 0) {
      if (c < a.C) put8<BF>(a.y, base + c, h[v]);
    } else {
      if constexpr (OUT == 1) top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(h[v][j]));
      if constexpr (OUT == 1) {
        // 16 lanes hold 128 adjacent columns
        top = over_lanes<(TPR < 16 ? TPR : 16), true>(top);
        const float scale = scale_of(top);
        if (c < a.C) {
          if ((at & 15) == 0) a.scales[row * ((a.C + 127) / 128) + c / 128] = scale;
#pragma unroll
          for (int j = 0; j < 8; ++j) h[v][j] /= scale;
        }
      }
    }
  }
  if constexpr (OUT == 2) {
    top = over_row<TPR, true>(top, lds[1]);
    const float scale = scale_of(top);
    if (at == 0) a.scales[row] = scale;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[v][j] /= scale;
  }
  if constexpr (OUT != 0) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      if (c >= a.C) continue;
      uint32_t q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int u = __builtin_amdgcn_cvt_pk_fp8_f32(h[v][4 * j], h[v][4 * j + 1], 0, false);
        u = __builtin_amdgcn_cvt_pk_fp8_f32(h[v][4 * j + 2], h[v][4 * j + 3], u, true);
        q[j] = (uint32_t)u;
      }
      *reinterpret_cast<uint2*>(a.codes + base + c) = make_uint2(q[0], q[1]);
    }
  }
}

// ---- gradients.  A workgroup walks over rows a grid apart and keeps its
// columns' sums of dy h r in registers; the workgroups' sums go to the
// workspace and are added up in the order of the workgroups.  16384 rows of
// 1024 columns in bfloat16: 28 us, 4.7 TB/s, of which the sums 4 us (without the
// next row's loads in flight 45 us); 2048 columns of float32 77 us, 5.2 TB/s.
template <int TPR, int NV, bool BF>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(NormBwd a, float* part) {
  constexpr int NT = TPR > 256 ? TPR : 256, RW = NT / TPR;
  __shared__ float lds[2][2][16];
  __shared__ float join[RW > 1 ? RW : 1][RW > 1 ? TPR * NV * 8 : 1];
  const int at = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  // dweight: eight rows at a time in float32, those sums in 64 bits where the
  // registers hold them.  In one float32 chain the error grows with the rows
  // (2-norm, of 16384 x 1024 1.3e-7, now 1.0e-7; of 2^22 x 64 3.6e-7, now 0.9e-7;
  // the call 28.2 -> 28.6 us).
  constexpr bool WIDE = NV <= 2;
  float dw[NV][8], wt[NV][8];
  double sum[WIDE ? NV : 1][8] = {};
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = (v * TPR + at) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = wt[v][j] = 0.f;
    if (c < a.C) get8<false>(a.weight, c, wt[v]);
  }
  // The next row's loads go out before the present one is worked on, where the
  // registers hold both (2048 rows of 16384 columns, us, with spilled registers
  // and without the loads ahead: bfloat16 66 / 51, float32 198 / 108).
  constexpr bool AHEAD = NV <= 2;
  Raw8<BF> hn[NV], dn[NV], en[NV];
  const auto load = [&](int64_t row) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      const int64_t i = row * a.C + c;
      hn[v].clear();
      dn[v].clear();
      en[v].clear();
      if (row < a.rows && c < a.C) {
        hn[v].load(a.h, i);
        dn[v].load(a.dy, i);
        if (a.dh) en[v].load(a.dh, i);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RW;
  int64_t row = (int64_t)blockIdx.x * RW + slot;
  if (AHEAD) load(row);
  // every wave of a workgroup makes the same turns where rows are shared by waves (RW == 1)
  for (int turn = 0, n = 0; row < a.rows; row += step, turn ^= 1) {
    const int64_t base = row * a.C;
    float h[NV][8], d[NV][8], x[NV][8];
    float hh = 0.f, hd = 0.f;
    if (!AHEAD) load(row);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      hn[v].get(h[v]);
      dn[v].get(d[v]);
      en[v].get(x[v]);
    }
    if (AHEAD) load(row + step);
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hh = fmaf(h[v][j], h[v][j], hh);
        hd = fmaf(h[v][j], d[v][j] * wt[v][j], hd);
      }
    hh = over_row<TPR, false>(hh, lds[turn][0]);
    hd = over_row<TPR, false>(hd, lds[turn][1]);
    const float r = 1.f / sqrtf(hh / (float)a.C + a.eps);
    const float f = r * r * (hd / (float)a.C);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dw[v][j] = fmaf(d[v][j], h[v][j] * r, dw[v][j]);
        x[v][j] = fmaf(r, d[v][j] * wt[v][j] - h[v][j] * f, x[v][j]);
      }
      if (c < a.C) put8<BF>(a.dx, base + c, x[v]);
    }
    if constexpr (WIDE)
      if (++n % 8 == 0)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) sum[v][j] += dw[v][j], dw[v][j] = 0.f;
  }
  if constexpr (WIDE)
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[v][j] = (float)(sum[v][j] + dw[v][j]);
  if constexpr (RW > 1) {
#pragma unroll
    for (int v = 0; v < NV; ++v) put8<false>(join[slot], (v * TPR + at) * 8, dw[v]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.C; c += NT) {
      double q = 0.0;
#pragma unroll
      for (int s = 0; s < RW; ++s) q += join[s][c];
      part[blockIdx.x * a.C + c] = (float)q;
    }
  } else {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * TPR + at) * 8;
      if (c < a.C) put8<false>(part, blockIdx.x * a.C + c, dw[v]);
    }
  }
}

// dweight of 16 columns: the workgroups' sums in 64 interleaved shares of at most
// eight, the shares in 64 bits (all of it in 64 bits: 16384 x 1024 28.6 -> 30.0 us).
__global__ __launch_bounds__(256) void norm_sum_kernel(const float* part, float* dweight, int groups, int64_t C) {
  __shared__ float lds[64][16];
  const int q = threadIdx.x % 4, s = threadIdx.x / 4;
  const int64_t col = (int64_t)blockIdx.x * 16 + 4 * q;   // C is a multiple of 8
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < C)
#pragma unroll 8
    for (int i = s; i < groups; i += 64) {
      const float4 y = *reinterpret_cast<const float4*>(part + i * C + col);
      x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
    }
*reinterpret_cast<float4*>(&lds[s][4 * q]) = make_float4(x[0], x[1], x[2], x[3]);
  __syncthreads();
  if (threadIdx.x < 16 && (int64_t)blockIdx.x * 16 + threadIdx.x < C) {
    double y = 0.0;
#pragma unroll
    for (int i = 0; i < 64; i += 8) {   // eight chains side by side
      double z = 0.0;
#pragma unroll
      for (int j = 0; j < 8; ++j) z += lds[i + j][threadIdx.x];
      y += z;
    }
    dweight[(int64_t)blockIdx.x * 16 + threadIdx.x] = (float)y;
  }
}

// Threads of a row and pieces of each, at most two (16 columns a thread): 8, 16
// and 32 threads hold up to 64, 128 and 256 columns, a wave up to 512, and up to
// 1024 of many rows, then four, eight and sixteen waves up to 4096, 8192 and
// 16384.  Measured, us, a wave / fewer threads: 64 columns of 2^19 rows 96 / 22,
// 128 of 2^18 50 / 22, 256 of 2^17 30 / 22.  Then, us, a wave / four waves:
// 1024 columns of 256 rows 3.4 / 3.0, of 2048 rows 4.5 / 4.8, of 16384 rows 17.2
// / 19.7; 2048 columns of 256 rows 4.5 / 3.1, of 16384 rows 32.7 / 31.2.  Four /
// eight / sixteen: 4096 columns of 4096 float32 rows 32.0 / 32.8 / 32.0; 8192 of
// 2048 rows 35.3 / 33.0 / 34.1; 16384 of 1024 rows, eight / sixteen 35.7 / 34.3.
struct Shape {
  int tpr, nv;
};
Shape shape_of(int64_t rows, int64_t C) {
  const int64_t pieces = C / 8;
  const int tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 64 || (pieces <= 128 && rows >= 2048) ? 64 : pieces <= 512 ? 256 : pieces <= 1024 ? 512 : 1024;
  return {tpr, pieces <= tpr ? 1 : 2};
}

// The gradients keep the next row and the sums of dweight besides: at most two
// pieces a thread up to 8192 columns.  A wave / fewer threads, us: 64 columns of
// 2^19 rows 223 / 35, 256 of 2^17 62 / 37; a wave / four waves: 1024 columns of
// 256 rows 6.1 / 7.0, of 16384 rows 19.4 / 37.7.
Shape bwd_shape_of(int64_t C) {
  const int64_t pieces = C / 8;
  const int tpr = pieces <= 8 ? 8 : pieces <= 16 ? 16 : pieces <= 32 ? 32 : pieces <= 128 ? 64 : pieces <= 512 ? 256 : 512;
  const int64_t need = (pieces + tpr - 1) / tpr;
  return {tpr, need <= 1 ? 1 : need <= 2 ? 2 : 4};
}

template <int TPR, int NV>
void launch_norm(const Norm& a, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  const dim3 grid((unsigned)((a.rows + NT / TPR - 1) / (NT / TPR)));
  const int out = !a.codes ? 0 : a.group ? 1 : 2;
  auto* k = a.bf16 ? (out == 0 ? norm_kernel<TPR, NV, true, 0> : out == 1 ? norm_kernel<TPR, NV, true, 1> : norm_kernel<TPR, NV, true, 2>)
                   : (out == 0 ? norm_kernel<TPR, NV, false, 0> : out == 1 ? norm_kernel<TPR, NV, false, 1> : norm_kernel<TPR, NV, false, 2>);
  hipLaunchKernelGGL(k, grid, dim3(NT), 0, s, a);
}

template <int TPR, int NV>
void launch_norm_bwd(const NormBwd& a, float* part, int groups, hipStream_t s) {
  constexpr int NT = TPR > 256 ? TPR : 256;
  auto* k = a.bf16 ? norm_bwd_kernel<TPR, NV, true> : norm_bwd_kernel<TPR, NV, false>;
  hipLaunchKernelGGL(k, dim3((unsigned)groups), dim3(NT), 0, s, a, part);
}

// Workgroups of the gradients, never more than there are rows for them: two
// for each CU, one of more than four waves, for each writes its sums of all
// columns.  Us, with one / two / four: 16384 rows of 1024 columns -- / 26.3 /
// 28.5; 4096 float32 rows of 8192 95.8 / 102 / 122.  Two rows for each at
// least costs small calls more than it saves (64 x 1024 6.1 -> 6.9 us).
int bwd_groups(const NormBwd& a, const Shape& f) {
  const int rw = f.tpr >= 256 ? 1 : 256 / f.tpr, most = f.tpr >= 512 ? 256 : 512;
  const int64_t want = (a.rows + rw - 1) / rw;
  return (int)(want < most ? want : most);
}

}  // namespace

hipError_t enqueue_norm(const Norm& a, hipStream_t s) {
  const Shape f = shape_of(a.rows, a.C);
  const auto launch = f.tpr == 8     ? launch_norm<8, 1>
                      : f.tpr == 16  ? launch_norm<16, 1>
                      : f.tpr == 32  ? launch_norm<32, 1>
                      : f.tpr == 64  ? (f.nv == 1 ? launch_norm<64, 1> : launch_norm<64, 2>)
                      : f.tpr == 256 ? (f.nv == 1 ? launch_norm<256, 1> : launch_norm<256, 2>)
                      : f.tpr == 512 ? launch_norm<512, 2>
                                     : launch_norm<1024, 2>;
  launch(a, s);
  return hipGetLastError();
}

size_t norm_bwd_workspace_bytes(const NormBwd& a) { return (size_t)bwd_groups(a, bwd_shape_of(a.C)) * a.C * 4; }

hipError_t enqueue_norm_bwd(const NormBwd& a, void* workspace, hipStream_t s) {
  const Shape f = bwd_shape_of(a.C);
  const int groups = bwd_groups(a, f);
  float* part = static_cast<float*>(workspace);
  const auto launch = f.tpr == 8     ? launch_norm_bwd<8, 1>
                      : f.tpr == 16  ? launch_norm_bwd<16, 1>
                      : f.tpr == 32  ? launch_norm_bwd<32, 1>
                      : f.tpr == 64  ? (f.nv == 1 ? launch_norm_bwd<64, 1> : launch_norm_bwd<64, 2>)
                      : f.tpr == 256 ? (f.nv == 1 ? launch_norm_bwd<256, 1> : launch_norm_bwd<256, 2>)
                                     : (f.nv <= 2 ? launch_norm_bwd<512, 2> : launch_norm_bwd<512, 4>);
  if (groups) launch(a, part, groups, s);
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((a.C + 15) / 16)), dim3(256), 0, s, part, a.dweight, groups, a.C);
  return hipGetLastError();
}

}  // namespace linattn
