// Linear attention with one decay for each head: the token-by-token steps and
// the launches of a call.
#include "linattn_plan.h"
#include "linattn_sweep.h"

namespace linattn {
namespace {

constexpr int NTH = kStepThreads;

// A few tokens (decoding): the recurrence itself in float32,
//   M <- a M + k_t^T v_t,   o_t = is q_t M,
// with the state's 64 columns of a block in registers: thread (x, y) holds
// rows y, y + 16, .. of columns 4x..4x+3.  Bound by the state's bytes, read
// and written once as whole 256-byte rows: one token of 256 x 32 heads of 64 x
// 64, 51 us, 5.4 TB/s; of 12 heads 4 us, a launch.
//
// The decay is carried in two parts, a = hi + lo: rounded to float32 it would
// be off the same way at every token, and a state that lives for 1 / (1 - a)
// tokens by as many times 2^-25 (6e-5 after 4096 tokens with a = 1 - 10^-5).
// Both parts are positive, so that an infinite state stays what it is.
template <int KX, bool BF, bool OBF>
__global__ __launch_bounds__(NTH) void step_kernel(Sweep a, int vblocks) {
  __shared__ float qk[2][kStepTokens][16 * KX];
  __shared__ float part[4][64];
  const int64_t pair = blockIdx.x / vblocks;
  const int v0 = (int)(blockIdx.x % vblocks) * kVBlock;
  const int64_t b = pair / a.H, h = pair % a.H;
  const int tid = threadIdx.x, x = tid & 15, y = tid >> 4, w = tid >> 6;
  const int n = v0 + 4 * x;
  const bool live = n < a.V;
  const int T = (int)tokens_of(a, b);
  const double decay = exp((double)a.log_decay[h]);
  float hi = (float)decay;
  if ((double)hi >= decay && hi > 0.f) hi = __uint_as_float(__float_as_uint(hi) - 1);   // the next float32 below
  const float lo = (float)(decay - (double)hi);

  const auto value = [](const void* p, int64_t i) {
    if constexpr (BF)
      return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
    else
      return static_cast<const float*>(p)[i];
  };
  float4 M[KX];
#pragma unroll
  for (int i = 0; i < KX; ++i) {
    const int c = y + 16 * i;
    M[i] = live && a.s_in && c < a.K ? *reinterpret_cast<const float4*>(a.s_in + pair * a.K * a.V + (int64_t)c * a.V + n)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int e = tid; e < T * 16 * KX; e += NTH) {
    const int t = e / (16 * KX), c = e % (16 * KX);
    qk[0][t][c] = c < a.K ? value(a.q.p, b * a.q.b + t * a.q.t + h * a.q.h + c) * a.is : 0.f;
    qk[1][t][c] = c < a.K ? value(a.k.p, b * a.k.b + t * a.k.t + h * a.k.h + c) : 0.f;
  }
  __syncthreads();
  for (int t = 0; t < T; ++t) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f), o = v;
    if (live) {
      const int64_t at = b * a.v.b + t * a.v.t + h * a.v.h + n;
      v = make_float4(value(a.v.p, at), value(a.v.p, at + 1), value(a.v.p, at + 2), value(a.v.p, at + 3));
    }
#pragma unroll
    for (int i = 0; i < KX; ++i) {
      const float k = qk[1][t][y + 16 * i], q = qk[0][t][y + 16 * i];
      M[i].x = fmaf(hi, M[i].x, fmaf(lo, M[i].x, k * v.x));
      M[i].y = fmaf(hi, M[i].y, fmaf(lo, M[i].y, k * v.y));
      M[i].z = fmaf(hi, M[i].z, fmaf(lo, M[i].z, k * v.z));
      M[i].w = fmaf(hi, M[i].w, fmaf(lo, M[i].w, k * v.w));
      o.x = fmaf(q, M[i].x, o.x);
      o.y = fmaf(q, M[i].y, o.y);
      o.z = fmaf(q, M[i].z, o.z);
      o.w = fmaf(q, M[i].w, o.w);
    }
    o = make_float4(wkv6::rows_sum(o.x), wkv6::rows_sum(o.y), wkv6::rows_sum(o.z), wkv6::rows_sum(o.w));
    if ((tid & 63) < 16) *reinterpret_cast<float4*>(&part[w][4 * x]) = o;
    __syncthreads();
    if (tid < 64 && v0 + tid < a.V) {
      const float r = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
      const int64_t at = b * a.o.b + t * a.o.t + h * a.o.h + v0 + tid;
      if constexpr (OBF)
        static_cast<__bf16*>(const_cast<void*>(a.o.p))[at] = (__bf16)r;
      else
        static_cast<float*>(const_cast<void*>(a.o.p))[at] = r;
    }
    __syncthreads();
  }
  for (int t = T; t < (int)a.T; ++t)
    if (tid < 64 && v0 + tid < a.V) {
      const int64_t at = b * a.o.b + t * a.o.t + h * a.o.h + v0 + tid;
      if constexpr (OBF)
        static_cast<uint16_t*>(const_cast<void*>(a.o.p))[at] = 0;
      else
        static_cast<float*>(const_cast<void*>(a.o.p))[at] = 0.f;
    }
  if (a.s_out && live)
#pragma unroll
    for (int i = 0; i < KX; ++i) {
      const int c = y + 16 * i;
      if (c < a.K) *reinterpret_cast<float4*>(a.s_out + pair * a.K * a.V + (int64_t)c * a.V + n) = M[i];
    }
}

// A call without tokens hands the state on (a kernel: a recorded memory copy
// or clear has no place in a captured graph of the caller's).
__global__ __launch_bounds__(NTH) void state_copy_kernel(const float4* from, float4* to, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * NTH + threadIdx.x; i < n; i += (int64_t)gridDim.x * NTH)
    to[i] = from ? from[i] : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <int KX>
hipError_t launch_steps(const Sweep& a, hipStream_t s) {
  const int vblocks = vblocks_of(a);
  const dim3 grid((unsigned)(a.B * a.H * vblocks));
  if (!a.bf16)
    hipLaunchKernelGGL((step_kernel<KX, false, false>), grid, dim3(NTH), 0, s, a, vblocks);
  else if (a.out_bf16)
    hipLaunchKernelGGL((step_kernel<KX, true, true>), grid, dim3(NTH), 0, s, a, vblocks);
  else
    hipLaunchKernelGGL((step_kernel<KX, true, false>), grid, dim3(NTH), 0, s, a, vblocks);
  return hipGetLastError();
}

}  // namespace

hipError_t enqueue_state_copy(const float* from, float* to, int64_t n, hipStream_t s) {
  if (from == to || n == 0) return hipSuccess;
  const int64_t want = (n / 4 + NTH - 1) / NTH;
  hipLaunchKernelGGL(state_copy_kernel, dim3((unsigned)(want < 4096 ? want : 4096)), dim3(NTH), 0, s,
                     reinterpret_cast<const float4*>(from), reinterpret_cast<float4*>(to), n / 4);
  return hipGetLastError();
}

size_t sweep_workspace_bytes(const Sweep* a, int n) { return planned_workspace_bytes(a, n); }

hipError_t enqueue_sweeps(const Sweep* a, int n, void* workspace, hipStream_t s) {
  if (steps(a, n)) return a->K <= 64 ? launch_steps<4>(*a, s) : launch_steps<8>(*a, s);
  if (const Split of = split(a, n); of.n[0]) {
    const hipError_t e = enqueue_sweeps(of.a[0], of.n[0], workspace, s);
    return e == hipSuccess ? enqueue_sweeps(of.a[1], of.n[1], workspace, s) : e;
  }
  SweepPlan p = plan(a, n);
  if (p.segments > 1) p.ws = static_cast<float*>(workspace);
  const auto launch = widest(a, n) <= 64 ? launch_sweeps64 : launch_sweeps128;
  // A sweep that leaves its state where another one takes its own from goes
  // last, after it (with segments, all states are read before the sweeps).
  bool after = false;
  for (int i = 0; i + 1 < n; ++i) after = after || (a[n - 1].s_out && a[n - 1].s_out == a[i].s_in);
  if (!after || p.segments > 1) return launch(p, s);
  p.sweeps = n - 1;
  const hipError_t e = launch(p, s);
  if (e != hipSuccess) return e;
  p.sweeps = 1;
  p.a[0] = a[n - 1];
  return launch(p, s);
}

}  // namespace linattn
