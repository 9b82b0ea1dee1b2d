// The selective scan forwards: prompts over blocks of tokens (ssm_scan.h), and
// a few tokens at a time with the state in registers.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_scan.h"

namespace ssm {
namespace {

// ---- prompts.  A workgroup stages the steps and inputs of its channels and B
// and C of a block of tokens in LDS, each wave goes through its share of the
// channels, and the sums over the states come back through LDS to be gated and
// stored by the threads that loaded the same places (a thread overwrites only rows that
// it has read itself, so that one barrier parts staging from the walk and one the walk from the
// output).  AHEAD: the next block is staged into a second buffer, and the one after it loaded, before
// a block's walk, which saves a barrier for each block and hides the loads; calls of many workgroups
// hide them by each other.
//
// bf16, 16 states, gate: 8 x 4096 tokens of 2048 channels 403 us, 0.38 ps a token and state
// (0.54 GB moved at 1.35 TB/s: bound by the vector instructions, 12.2 a token and state with the
// shares of softplus and gate, 290 us of them at 3 clocks each and 8.7 an exp); 8192 tokens of 1536 channels 139, where
// 192 workgroups leave a quarter of the CUs without one.  (float32, 16 channels: 8 registers are spilled.)
//
// Waves a SIMD that LDS leaves room for, up to 4, for which the registers are made to do (128 each:
// 8 x 4096 tokens of 2048 channels 441 -> 400 us).  Two buffers leave room for one or two
// workgroups of 8 waves, which need no such bound.
template <class S, bool AHEAD>
constexpr int waves_of() {
  constexpr int floats = (S::NG > 1 ? 3 : 2) * S::DW * S::LD + 2 * S::TB * S::N + 2 * S::DW * S::N + 2 * S::DW;
  constexpr int waves = 160 * 1024 / (4 * floats) * S::NW / 4;
  return AHEAD ? 1 : waves < 4 ? waves : 4;
}

template <class S, bool AHEAD, bool BF>
__global__ __launch_bounds__(S::NT, (waves_of<S, AHEAD>())) void scan_kernel(Scan a) {
  constexpr int BUFFERS = AHEAD ? 2 : 1;
  __shared__ float4 delta4[BUFFERS][S::DW * S::LD / 4], ux4[BUFFERS][S::DW * S::LD / 4];
  __shared__ float4 y4[S::NG > 1 ? BUFFERS : 1][S::NG > 1 ? S::DW * S::LD / 4 : 1];
  __shared__ float4 B4[BUFFERS][S::TB * S::N / 4], C4[BUFFERS][S::TB * S::N / 4];
  __shared__ float4 a4[S::DW * S::N / 4], carry4[S::DW * S::N / 4];
  __shared__ float tables[2][S::DW];
  float* const a2 = reinterpret_cast<float*>(a4);
  float* const carry = reinterpret_cast<float*>(carry4);

  const Where w = where_of<S::DW>(a.B, a.D, a.G);
  if (!w.live) return;
  const int tid = threadIdx.x, wave = tid / 64, q = tid % 64 / 16, l = tid % 16;
  const int64_t b = w.b, n = tokens_of(a.lengths, b, a.T);

  for (int i = tid; i < S::DW * S::N; i += S::NT) {
    const int c = i / S::N, s = i % S::N;
    const bool in = c < w.channels && s < a.N;
    const int64_t at = (int64_t)(w.c0 + c) * a.N + s;
    a2[i] = in ? a.A[at] * kLog2e : 0.f;
    carry[i] = in && a.s_in ? a.s_in[b * a.D * a.N + at] : 0.f;
  }

  for (int i = tid; i < 2 * S::DW; i += S::NT) {
    const float* const from = i < S::DW ? a.skip : a.bias;
    tables[i / S::DW][i % S::DW] = from && i % S::DW < w.channels ? from[w.c0 + i % S::DW] : 0.f;
  }
  using Mine = Pieces<S, !AHEAD>;
  const auto live = [&](const Mine& me, int i, int64_t t0) {
    return me.c < w.channels && me.token(i) < S::TB && t0 + me.token(i) < n;
  };
  const auto row = [&](const Mine& me, const Tensor& t, int64_t at) { return b * t.b + at * t.t + w.c0 + me.c; };
  __syncthreads();   // the tables

  Raw<BF, S::PC> rx[S::TURNS], rdt[S::TURNS], now[S::TURNS], rz[S::TURNS];
  Raw8<BF> rB[S::BTURNS], rC[S::BTURNS];
  const auto load = [&](int64_t t0) {
    const Mine me(tid);
#pragma unroll
    for (int i = 0; i < S::TURNS; ++i) {
      rx[i].clear();
      rdt[i].clear();
      if (live(me, i, t0)) {
        rx[i].load(a.x.p, row(me, a.x, t0 + me.token(i)));
        rdt[i].load(a.dt.p, row(me, a.dt, t0 + me.token(i)));
      }
    }
#pragma unroll
    for (int i = 0; i < S::BTURNS; ++i) {
      const int p = me.state_piece(i), t = S::piece_token(p), s = S::piece_state(p);
      rB[i].clear();
      rC[i].clear();
      if (p < S::BPIECES && t0 + t < n && s < a.N) {
        rB[i].load(a.b.p, b * a.b.b + (t0 + t) * a.b.t + w.g * a.b.h + s);
        rC[i].load(a.c.p, b * a.c.b + (t0 + t) * a.c.t + w.g * a.c.h + s);
      }
    }
  };
  // The inputs of the output's factor and skip.
  const auto load_out = [&](const Mine& me, int64_t t0, int i) {
    if (!live(me, i, t0)) return;
    now[i].load(a.x.p, row(me, a.x, t0 + me.token(i)));
    if (a.z.p) rz[i].load(a.z.p, row(me, a.z, t0 + me.token(i)));
  };

  const auto stage = [&](int64_t t0, int buffer) {
    float* const delta = reinterpret_cast<float*>(delta4[buffer]);
    float* const ux = reinterpret_cast<float*>(ux4[buffer]);
    float* const Bs = reinterpret_cast<float*>(B4[buffer]);
    float* const Cs = reinterpret_cast<float*>(C4[buffer]);
    const Mine me(tid);
    const int c = me.c;
    const float* const bias = tables[1] + c;
#pragma unroll
    for (int i = 0; i < S::TURNS; ++i) {
      const int t = me.token(i);
      if (t >= S::TB) continue;
      const bool in = live(me, i, t0);
      float x[S::PC], v[S::PC];
      rx[i].get(x);
      rdt[i].get(v);
#pragma unroll
      for (int k = 0; k < S::PC; ++k) v[k] += bias[k];
      if (a.softplus)   // (one branch around all of them: their chains overlap)
#pragma unroll
        for (int k = 0; k < S::PC; ++k) v[k] = softplus(v[k]);
#pragma unroll
      for (int k = 0; k < S::PC; ++k) {
        const float d = in ? v[k] : 0.f;
        delta[(c + k) * S::LD + S::at(t)] = d;
        ux[(c + k) * S::LD + S::at(t)] = d * x[k];
      }
    }
#pragma unroll
    for (int i = 0; i < S::BTURNS; ++i) {
      const int p = me.state_piece(i), t = S::piece_token(p), s = S::piece_state(p);
      if (p >= S::BPIECES) continue;
      float x[8], y[8];
      rB[i].get(x);
      rC[i].get(y);
#pragma unroll
      for (int k = 0; k < 8; k += S::NL < 4 ? 2 : 4) {
        if constexpr (S::NL < 4) {
          *reinterpret_cast<float2*>(Bs + S::at(t, s + k)) = make_float2(x[k], x[k + 1]);
          *reinterpret_cast<float2*>(Cs + S::at(t, s + k)) = make_float2(y[k], y[k + 1]);
        } else {
          *reinterpret_cast<float4*>(Bs + S::at(t, s + k)) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          *reinterpret_cast<float4*>(Cs + S::at(t, s + k)) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
        }
      }
    }
  };

  if (AHEAD && n) {
    load(0);
    stage(0, 0);
    if (S::TB < n) load(S::TB);
    __syncthreads();
  }
  for (int64_t t0 = 0; t0 < n; t0 += S::TB) {
    const int buffer = AHEAD ? (int)(t0 / S::TB % 2) : 0;
    float* const delta = reinterpret_cast<float*>(delta4[buffer]);
    float* const ux = reinterpret_cast<float*>(ux4[buffer]);
    float* const ys = S::NG > 1 ? reinterpret_cast<float*>(y4[S::NG > 1 ? buffer : 0]) : ux;   // the sums of C h
    float* const Bs = reinterpret_cast<float*>(B4[buffer]);
    float* const Cs = reinterpret_cast<float*>(C4[buffer]);
    if constexpr (AHEAD) {
      const Mine me(tid);
#pragma unroll
      for (int i = 0; i < S::TURNS; ++i) load_out(me, t0, i);
      if (t0 + S::TB < n) stage(t0 + S::TB, 1 - buffer);
      if (t0 + 2 * S::TB < n) load(t0 + 2 * S::TB);
    } else {
      load(t0);
      stage(t0, 0);
      __syncthreads();
    }
#pragma unroll 1
    for (int g = 0; g * S::NS < a.N; ++g) {
#pragma unroll 1
      for (int d = wave; d < w.channels; d += S::NW) {
        const int states = d * S::N + g * S::NS + q * S::NL;
        float dl[S::R], in[S::R], an[S::NL], h[S::NL], y[S::R], v[S::R][S::NL];
        get_tokens<S>(delta + d * S::LD, l, dl);
        get_tokens<S>(ux + d * S::LD, l, in);
        get_states<S::NL>(a2 + states, an);
        get_states<S::NL>(carry + states, h);
        asm volatile("" ::: "memory");   // B and C are read for every channel: registers for them would halve the waves
        get_block<S>(Bs, g, q, l, v);
        Walk<S> k;
        k.run(dl, in, an, v, h);
        if (l == kLanes - 1) put_states<S::NL>(carry + states, k.end);
        asm volatile("" ::: "memory");
        get_block<S>(Cs, g, q, l, v);
#pragma unroll
        for (int r = 0; r < S::R; ++r) {
          y[r] = 0.f;
#pragma unroll
          for (int i = 0; i < S::NL; ++i) {
            k.before[i] = fmaf(k.e[r][i], k.before[i], k.u[r][i]);
            y[r] = fmaf(v[r][i], k.before[i], y[r]);
          }
        }
        put_sums<S>(ys + d * S::LD, q, l, y, g > 0);
      }
    }
    __syncthreads();
    const Mine out(tid);
    const float* const skip = tables[0] + out.c;
#pragma unroll
    for (int i = 0; i < S::TURNS; ++i) {
      const int t = out.token(i);
      if (t >= S::TB || out.c >= w.channels || t0 + t >= a.T) continue;
      const bool in = t0 + t < n;
      Raw<BF, S::PC> r;
      r.clear();
      if (in) {
        float x[S::PC], y[S::PC];
        if (!AHEAD) load_out(out, t0, i);
        now[i].get(x);
#pragma unroll
        for (int k = 0; k < S::PC; ++k) y[k] = fmaf(skip[k], x[k], ys[(out.c + k) * S::LD + S::at(t)]);
        if (a.z.p) {
          rz[i].get(x);
#pragma unroll
          for (int k = 0; k < S::PC; ++k) y[k] *= x[k] * sigmoid<BF>(x[k]);
        }
        r.set(y);
      }
      r.store(const_cast<void*>(a.y.p), row(out, a.y, t0 + t));
    }
  }
  // rows behind the last block's
  if (const Mine me(tid); me.c < w.channels) {
    Raw<BF, S::PC> zero;
    zero.clear();
    for (int64_t t = (n + S::TB - 1) / S::TB * S::TB + me.token(0); t < a.T; t += S::NT / (S::DW / S::PC))
      zero.store(const_cast<void*>(a.y.p), row(me, a.y, t));
  }
  __syncthreads();
  if (a.s_out)
    for (int i = tid; i < S::DW * S::N; i += S::NT) {
      const int d = i / S::N, s = i % S::N;
      if (d < w.channels && s < a.N) a.s_out[b * a.D * a.N + (int64_t)(w.c0 + d) * a.N + s] = carry[i];
    }
}

// ---- a few tokens.  SL adjacent states of a channel for each thread, in registers,
// and N / SL threads side by side for a channel (shared by lanes of one wave).  Bound
// by the bytes of the states and, from a few tokens on, by the vector instructions.
//
// One token's state, h exp(x) + u with x = delta A.  A decay rounded to float32
// would be off the same way at every token, and a state that lives for thousands of
// tokens by as many times 2^-25: down to exp(-0.35) it is taken as 1 + m, m = expm1(x)
// = x (1 + x/2 (1 + x/3 (...))), to x^8 / 8! which leaves 2^-26 of x, and the state rounds
// once.  Below, a state lives for three tokens.
__device__ __forceinline__ float moved(float h, float x, float u) {
  float m = fmaf(x, 1.f / 40320.f, 1.f / 5040.f);
  m = fmaf(m, x, 1.f / 720.f);
  m = fmaf(m, x, 1.f / 120.f);
  m = fmaf(m, x, 1.f / 24.f);
  m = fmaf(m, x, 1.f / 6.f);
  m = fmaf(m, x, 0.5f);
  m = fmaf(m * x, x, x);
  const bool near = fabsf(x) < 0.35f;
  return fmaf(near ? m : exp_whole(x), h, u) + (near ? h : 0.f);
}

template <bool BF>
__device__ __forceinline__ float value(const void* p, int64_t i) {
  if constexpr (BF)
    return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else
    return static_cast<const float*>(p)[i];
}
constexpr int kStepThreads = 256;

template <int SL, int LN, bool BF>   // states of a lane, lanes of a channel: a power of two
__global__ __launch_bounds__(kStepThreads) void step_kernel(Scan a, int64_t across) {
  const int64_t id = (int64_t)blockIdx.x % across * kStepThreads + threadIdx.x;
  const int64_t b = blockIdx.x / across;
  const int64_t d = id / LN;
  const int s = (int)(id % LN) * SL;
  if (d >= a.D) return;   // all lanes of a channel together
  const bool in = s < a.N;
  const int64_t at = d * a.N + s, state = b * a.D * a.N + at;
  const int g = (int)(d / (a.D / a.G));
  const int n = (int)tokens_of(a.lengths, b, a.T);
  float A[SL], h[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) A[i] = h[i] = 0.f;
  if (in) get_states<SL>(a.A + at, A);
  if (in && a.s_in) get_states<SL>(a.s_in + state, h);
  const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
  for (int t = 0; t < (int)a.T; ++t) {
    float y = 0.f;
    if (t < n) {
      float B[SL], C[SL];
#pragma unroll
      for (int i = 0; i < SL; ++i) B[i] = C[i] = 0.f;
      if (in) {
        Raw<BF, SL> r;
        r.load(a.b.p, b * a.b.b + t * a.b.t + g * a.b.h + s);
        r.get(B);
        r.load(a.c.p, b * a.c.b + t * a.c.t + g * a.c.h + s);
        r.get(C);
      }
      const float x = value<BF>(a.x.p, b * a.x.b + t * a.x.t + d);
      const float z = a.z.p ? value<BF>(a.z.p, b * a.z.b + t * a.z.t + d) : 0.f;
      float v = value<BF>(a.dt.p, b * a.dt.b + t * a.dt.t + d) + bias;
      if (a.softplus) v = softplus(v);
      const float ux = v * x;
#pragma unroll
      for (int i = 0; i < SL; ++i) {
        h[i] = moved(h[i], v * A[i], ux * B[i]);
        y = fmaf(C[i], h[i], y);
      }
      y = fmaf(skip, x, linattn::over_lanes<LN, false>(y));
      if (a.z.p) y *= z * sigmoid<BF>(z);
    }
    if (s == 0) {
      const int64_t to = b * a.y.b + t * a.y.t + d;
      if constexpr (BF)
        static_cast<uint16_t*>(const_cast<void*>(a.y.p))[to] = (uint16_t)linattn::pair(y, 0.f);
      else
        static_cast<float*>(const_cast<void*>(a.y.p))[to] = y;
    }
  }
  // (Past the caches: the next reader of a state is the next token's call, all other layers' states
  // later.  256 x 4096 channels of 16 states, bf16: 35.6 -> 30.1 us.)
  using Four = float __attribute__((ext_vector_type(4)));
  if (in && a.s_out)
#pragma unroll
    for (int i = 0; i < SL; i += 4)
      __builtin_nontemporal_store(Four{h[i], h[i + 1], h[i + 2], h[i + 3]}, reinterpret_cast<Four*>(a.s_out + state + i));
}

template <int LN>
void launch_steps(const Scan& a, hipStream_t s) {
  // us, with 4 / 8 (before the states went past the caches) one token of 256 x 4096 channels of 16 states
  // 40.2 / 35.7, 8 tokens 141 / 105
  constexpr int SL = 8;
  const int64_t across = ((int64_t)a.D * LN + kStepThreads - 1) / kStepThreads;
  hipLaunchKernelGGL((a.bf16 ? step_kernel<SL, LN, true> : step_kernel<SL, LN, false>), dim3((unsigned)(across * a.B)),
                     dim3(kStepThreads), 0, s, a, across);
}

template <class S, bool AHEAD>
void launch(const Scan& a, hipStream_t s) {
  hipLaunchKernelGGL((a.bf16 ? scan_kernel<S, AHEAD, true> : scan_kernel<S, AHEAD, false>), dim3((unsigned)grid_of<S::DW>(a)),
                     dim3(S::NT), 0, s, a);
}

// Channels and waves of a workgroup, with the number of workgroups of 8 channels; us for
// 2048 tokens of 16 states with 8 channels and two buffers by 8 waves / 8 by 4 waves / 16 by 4
// waves:
//   256: 35 / 59 / 87    512: 67 / 72 / 87    600: 99 / 93 / 116    1024: 150 / 121 / 127
//   2048: 300 / 224 / 204
// Up to two workgroups for each CU there are waves enough only with 8 of them each, and the
// second buffer hides the staging; from there on more channels share what is staged of B and C.
// Of 32 states the rows of 16 channels leave room for two waves a SIMD: 402 with 8 channels,
// 410 with 16.  Of 64 states B and C of a block, 64 KB, leave one workgroup of 8 waves a CU either
// way; 8 channels with two buffers and 32 with one: 512: 193 / 368, 1024: 385 / 386, but 64 x 48
// tokens of 2048 channels 376 / 169.
template <int NL, int R, int NG>
void launch_blocks(const Scan& a, hipStream_t s) {
  const int64_t groups = a.B * blocks_of<8>(a.D, a.G);
  if (groups <= (NG == 4 ? 1024 : 512)) return launch<Shape<NL, R, NG, 8, 8, 4>, true>(a, s);
  if constexpr (NG == 4) {
    launch<Shape<NL, R, NG, 32, 8, 8>, false>(a, s);
  } else if constexpr (NG == 2) {
    launch<Shape<NL, R, NG, 8, 4, 4>, false>(a, s);
  } else {
    if (groups <= 1024)
      launch<Shape<NL, R, NG, 8, 4, 4>, false>(a, s);
    else
      launch<Shape<NL, R, NG, 16, 4, 8>, false>(a, s);
  }
}

// Up to so many tokens go token by token.  Either way with 64 x 2048 channels: 8 tokens 16.0 us,
// by blocks 36.8; 10 tokens 19.5 / 37.0; but 1 x 2048 channels, 10 tokens: 11.2 / 9.4, 16 tokens: 16.4 / 9.5.
constexpr int kTokens = 8;

// Tokens of a block are 16 R: 64 x 32 tokens of 2048 channels with R of 2, 4 and 8 38 / 51 / 83 us,
// of 64 tokens with 4 and 8 53 / 85; prompts of 8 x 4096 tokens with 4 and 8 507 / 400.
template <int R>
void launch_tokens(const Scan& a, hipStream_t s) {
  (a.N <= 8 ? launch_blocks<2, R, 1> : a.N <= 16 ? launch_blocks<4, R, 1> : a.N <= 32 ? launch_blocks<4, R, 2> : launch_blocks<4, R, 4>)(a, s);
}

}  // namespace

hipError_t enqueue_scan(const Scan& a, hipStream_t s) {
  if (a.T <= kTokens)
    (a.N <= 8 ? launch_steps<1> : a.N <= 16 ? launch_steps<2> : a.N <= 32 ? launch_steps<4> : launch_steps<8>)(a, s);
  else
    (a.T <= 32 ? launch_tokens<2> : a.T <= 64 ? launch_tokens<4> : launch_tokens<8>)(a, s);
  return hipGetLastError();
}

}  // namespace ssm
