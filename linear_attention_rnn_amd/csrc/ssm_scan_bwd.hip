// Gradients of the selective scan.  With m_t = sum_n C_t h_t + D x_t, s = silu(z)
// (1 without z) and dm = dy s, the adjoint of the state runs from the last token
// to the first:
//
//   g_t = C_t dm_t + exp(delta_{t+1} A) g_{t+1},  q_t = exp(delta_t A) g_t h_{t-1}
//   dB_t = sum_d g delta x,   dC_t = sum_d dm h,  dz = dy m silu'(z)
//   dx = delta sum_n g B + D dm,   ddelta = x sum_n g B + sum_n A q,   dA = sum_t delta q
//
// A workgroup has up to DW channels of a batch item.  It goes through the blocks
// of tokens forwards once, which leaves the state at the start of each in the
// workspace, then backwards: there each wave walks a channel forwards (ssm_scan.h), keeps
// decays and states of the block in registers, and comes back with the adjoint, whose
// decays over lanes are combined the same way.  Sums over channels stay in
// registers while a wave goes through its channels, then the waves add theirs up
// in order; the workgroups' sums are added up by a second kernel.
//
// Bound by the vector instructions, 39.6 per token and state (of 16, with the shares of softplus
// and gate; a third of them in the way forwards), at two waves a SIMD: decays, inputs, states and
// sums of a lane's tokens fill 256 registers; 16 channels of 17 to 32 states spill 17 to 19 of them.  bf16, 16 states,
// gate: 4 x 4096 tokens of 2048 channels 833 us, 1.6 ps a token and state; with the 35 us that add up dB and dC.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "ssm_scan.h"

namespace ssm {
namespace {

// The workspace.
struct Sums {
  float* states;   // [B, D, blocks of tokens][N as the lanes hold it]: at the start of each but the first
  float* bc;       // [B, blocks of channels, T][2][N]: dB and dC
  float* A;        // [B, D, N]
  float* skip;     // [B, D]
  float* bias;     // [B, D]
};

template <class S>
struct Layout {
  size_t states, bc, A, skip, bias, bytes;
  int64_t blocks;   // of tokens
  explicit Layout(const Scan& a) {
    blocks = (a.T + S::TB - 1) / S::TB;
    size_t at = 0;
    const auto take = [&](size_t floats) {
      const size_t from = at;
      at += (floats + 3) / 4 * 16;
      return from;
    };
    states = take((size_t)a.B * a.D * S::N * blocks);
    bc = take((size_t)a.B * blocks_of<S::DW>(a.D, a.G) * a.T * 2 * a.N);
    A = take((size_t)a.B * a.D * a.N);
    skip = take((size_t)a.B * a.D);
    bias = take((size_t)a.B * a.D);
    bytes = at;
  }
  Sums in(void* ws) const {
    char* p = static_cast<char*>(ws);
    const auto f = [&](size_t at) { return reinterpret_cast<float*>(p + at); };
    return {f(states), f(bc), f(A), f(skip), f(bias)};
  }
};

template <class S, bool BF>
__global__ __launch_bounds__(S::NT) void scan_bwd_kernel(Scan a, Sums ws, int64_t blocks) {
  // With several groups of states the inputs of the next are not overwritten.
  constexpr int ROWS = S::NG > 1 ? 6 : 4;
  __shared__ float4 rows4[ROWS][S::DW * S::LD / 4];
  __shared__ float4 B4[S::TB * S::N / 4], C4[S::TB * S::N / 4];
  __shared__ float4 a4[S::DW * S::N / 4], carry4[S::DW * S::N / 4], back4[S::DW * S::N / 4], dA4[S::DW * S::N / 4];
  __shared__ float tables[2][S::DW];
  __shared__ float4 sums4[S::NW / 2][2][S::TB * S::NS / 4];
  float* const sums = reinterpret_cast<float*>(sums4);
  float* const delta = reinterpret_cast<float*>(rows4[0]);
  float* const ux = reinterpret_cast<float*>(rows4[1]);
  float* const dm = reinterpret_cast<float*>(rows4[2]);
  float* const qa = reinterpret_cast<float*>(rows4[3]);                            // the sums of A q / log 2,
  float* const gbs = reinterpret_cast<float*>(rows4[S::NG > 1 ? ROWS - 2 : 1]);    // of g B
  float* const ys = reinterpret_cast<float*>(rows4[S::NG > 1 ? ROWS - 1 : 2]);     // and of C h
  float* const Bs = reinterpret_cast<float*>(B4);
  float* const Cs = reinterpret_cast<float*>(C4);
  float* const a2 = reinterpret_cast<float*>(a4);
  float* const carry = reinterpret_cast<float*>(carry4);   // the state at the start of the block
  float* const back = reinterpret_cast<float*>(back4);     // the adjoint of that at its end
  float* const dA = reinterpret_cast<float*>(dA4);

  const Where w = where_of<S::DW>(a.B, a.D, a.G);
  if (!w.live) return;
  const int tid = threadIdx.x, wave = tid / 64, q = tid % 64 / 16, l = tid % 16;
  const int64_t b = w.b, n = tokens_of(a.lengths, b, a.T);
  const int64_t last = (n + S::TB - 1) / S::TB - 1;   // block; -1: none

  for (int i = tid; i < S::DW * S::N; i += S::NT) {
    const int c = i / S::N, s = i % S::N;
    const bool in = c < w.channels && s < a.N;
    const int64_t at = (int64_t)(w.c0 + c) * a.N + s;
    a2[i] = in ? a.A[at] * kLog2e : 0.f;
    carry[i] = in && a.s_in ? a.s_in[b * a.D * a.N + at] : 0.f;
    back[i] = in && a.ds_out ? a.ds_out[b * a.D * a.N + at] : 0.f;
    dA[i] = 0.f;
  }
  for (int i = tid; i < 2 * S::DW; i += S::NT) {
    const float* const from = i < S::DW ? a.skip : a.bias;
    tables[i / S::DW][i % S::DW] = from && i % S::DW < w.channels ? from[w.c0 + i % S::DW] : 0.f;
  }
  // The state at the start of block k of the workgroup's channel d.
  const auto start = [&](int d, int64_t k) { return ws.states + ((b * a.D + w.c0 + d) * blocks + k) * S::N; };

  const auto live = [&](const Pieces<S>& me, int i, int64_t t0) {
    return me.c < w.channels && me.token(i) < S::TB && t0 + me.token(i) < n;
  };
  const auto row = [&](const Pieces<S>& me, const Tensor& t, int64_t at) { return b * t.b + at * t.t + w.c0 + me.c; };
  using Piece = Raw<BF, S::PC>;

  // A block's steps and inputs, and with ALL its C and gradients of y.
  const auto stage = [&](int64_t t0, auto ALL) {
    constexpr bool all = decltype(ALL)::value;
    const Pieces<S> me(tid);
    const int c = me.c;
    const float* const bias = tables[1] + c;
    Piece rx[S::TURNS], rdt[S::TURNS], rdy[S::TURNS], rz[S::TURNS];
    Raw8<BF> rB[S::BTURNS], rC[S::BTURNS];
#pragma unroll
    for (int i = 0; i < S::TURNS; ++i) {
      rx[i].clear();
      rdt[i].clear();
      rdy[i].clear();
      rz[i].clear();
      if (!live(me, i, t0)) continue;
      rx[i].load(a.x.p, row(me, a.x, t0 + me.token(i)));
      rdt[i].load(a.dt.p, row(me, a.dt, t0 + me.token(i)));
      if constexpr (all) {
        rdy[i].load(a.dy.p, row(me, a.dy, t0 + me.token(i)));
        if (a.z.p) rz[i].load(a.z.p, row(me, a.z, t0 + me.token(i)));
      }
    }
#pragma unroll
    for (int i = 0; i < S::BTURNS; ++i) {
      const int p = me.state_piece(i), t = S::piece_token(p), s = S::piece_state(p);
      rB[i].clear();
      rC[i].clear();
      if (p >= S::BPIECES || t0 + t >= n || s >= a.N) continue;
      rB[i].load(a.b.p, b * a.b.b + (t0 + t) * a.b.t + w.g * a.b.h + s);
      if constexpr (all) rC[i].load(a.c.p, b * a.c.b + (t0 + t) * a.c.t + w.g * a.c.h + s);
    }
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
      if constexpr (all) {
        rdy[i].get(v);
        rz[i].get(x);
        if (a.z.p)
#pragma unroll
          for (int k = 0; k < S::PC; ++k) v[k] *= x[k] * sigmoid(x[k]);
#pragma unroll
        for (int k = 0; k < S::PC; ++k) dm[(c + k) * S::LD + S::at(t)] = v[k];
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
          if (all) *reinterpret_cast<float2*>(Cs + S::at(t, s + k)) = make_float2(y[k], y[k + 1]);
        } else {
          *reinterpret_cast<float4*>(Bs + S::at(t, s + k)) = make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
          if (all) *reinterpret_cast<float4*>(Cs + S::at(t, s + k)) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
        }
      }
    }
  };

  // ---- forwards: the states at the starts of the blocks
  for (int64_t k = 0; k < last; ++k) {
    __syncthreads();
    stage(k * S::TB, std::false_type());
    __syncthreads();
#pragma unroll 1
    for (int g = 0; g * S::NS < a.N; ++g) {
#pragma unroll 1
      for (int d = wave; d < w.channels; d += S::NW) {
        const int states = d * S::N + g * S::NS + q * S::NL;
        float dl[S::R], in[S::R], an[S::NL], h[S::NL], Bv[S::R][S::NL];
        get_tokens<S>(delta + d * S::LD, l, dl);
        get_tokens<S>(ux + d * S::LD, l, in);
        get_states<S::NL>(a2 + states, an);
        get_states<S::NL>(carry + states, h);
        asm volatile("" ::: "memory");   // B is read for every channel: registers for it would cost waves
        get_block<S>(Bs, g, q, l, Bv);
        Walk<S> f;
        f.run(dl, in, an, Bv, h);
        if (l == kLanes - 1) {
          put_states<S::NL>(carry + states, f.end);
          put_states<S::NL>(start(d, k + 1) + g * S::NS + q * S::NL, f.end);
        }
      }
    }
  }

  // ---- backwards
  float dskip[S::PC] = {}, dbias[S::PC] = {};
  for (int64_t k = last; k >= 0; --k) {
    const int64_t t0 = k * S::TB;
    __syncthreads();
    stage(t0, std::true_type());
    __syncthreads();
#pragma unroll 1
    for (int g = 0; g * S::NS < a.N; ++g) {
      float dB[S::R][S::NL], dC[S::R][S::NL];
#pragma unroll
      for (int r = 0; r < S::R; ++r)
#pragma unroll
        for (int i = 0; i < S::NL; ++i) dB[r][i] = dC[r][i] = 0.f;
#pragma unroll 1
      for (int d = wave; d < w.channels; d += S::NW) {
        const int states = d * S::N + g * S::NS + q * S::NL;
        float dl[S::R], in[S::R], dv[S::R], an[S::NL], h0[S::NL], h[S::R][S::NL], v[S::R][S::NL], y[S::R];
        get_tokens<S>(delta + d * S::LD, l, dl);
        get_tokens<S>(ux + d * S::LD, l, in);
        get_tokens<S>(dm + d * S::LD, l, dv);
        get_states<S::NL>(a2 + states, an);
        if (k == last && last > 0) {
          get_states<S::NL>(carry + states, h0);   // left by the way forwards
        } else if (k > 0) {
          get_states<S::NL>(start(d, k) + g * S::NS + q * S::NL, h0);
        } else {
          const int at = g * S::NS + q * S::NL;
          const float* const s = a.s_in + (b * a.D + w.c0 + d) * a.N + at;
#pragma unroll
          for (int i = 0; i < S::NL; ++i) h0[i] = a.s_in && at + i < a.N ? s[i] : 0.f;
        }
        asm volatile("" ::: "memory");
        get_block<S>(Bs, g, q, l, v);
        Walk<S> f;
        f.run(dl, in, an, v, h0);
        asm volatile("" ::: "memory");
        const int mine = ((g * 4 + q) * S::R) * S::STEP + l * S::NL;   // B and C of the lane
#pragma unroll
        for (int r = 0; r < S::R; ++r) {
          float Cr[S::NL];
          get_states<S::NL>(Cs + mine + r * S::STEP, Cr);
          y[r] = 0.f;
#pragma unroll
          for (int i = 0; i < S::NL; ++i) {
            h[r][i] = fmaf(f.e[r][i], r ? h[r - 1][i] : f.before[i], f.u[r][i]);
            y[r] = fmaf(Cr[i], h[r][i], y[r]);
            dC[r][i] = fmaf(dv[r], h[r][i], dC[r][i]);
          }
        }
        put_sums<S>(ys + d * S::LD, q, l, y, g > 0);
        asm volatile("" ::: "memory");
        // the adjoint that reaches the lane from the ones behind it
        float G[S::NL], P[S::NL], end[S::NL], gr[S::NL], total = f.sum;
        get_states<S::NL>(back + states, end);
#pragma unroll
        for (int i = 0; i < S::NL; ++i) {
          G[i] = 0.f;
          P[i] = __builtin_amdgcn_exp2f(f.sum * an[i]);
        }
#pragma unroll
        for (int r = S::R - 1; r >= 0; --r) {
          float Cr[S::NL];
          get_states<S::NL>(Cs + mine + r * S::STEP, Cr);
#pragma unroll
          for (int i = 0; i < S::NL; ++i) G[i] = f.e[r][i] * fmaf(Cr[i], dv[r], G[i]);
        }
        const auto join = [&](auto step) {
          constexpr int K = decltype(step)::value;
          total += behind<K>(total);
          add_before<-K>(G, P);
          if constexpr (K < 8)
#pragma unroll
            for (int i = 0; i < S::NL; ++i) P[i] *= behind<K>(P[i]);
        };
        join(std::integral_constant<int, 1>());
        join(std::integral_constant<int, 2>());
        join(std::integral_constant<int, 4>());
        join(std::integral_constant<int, 8>());
#pragma unroll
        for (int i = 0; i < S::NL; ++i) {
          G[i] = fmaf(__builtin_amdgcn_exp2f(total * an[i]), end[i], G[i]);
          gr[i] = behind_or(G[i], end[i]);
        }
        if (l == 0) put_states<S::NL>(back + states, G);
        // Back over the lane's tokens.  Steps behind the sequence are zero, and 0 times a state that is not finite
        // would go into dA: the state in front of them counts as zero.  (An instruction for each token and state,
        // 1% of the time for 4 x 4096 tokens of 2048 channels; a way of its own for the blocks in which a sequence
        // ends saved half of that, nothing where there are 8 channels, and was twice the code.)
        const int left = (int)(n - t0 < S::TB ? n - t0 : S::TB) - l * S::R;
        float gb[S::R], qs[S::R], da[S::NL];
#pragma unroll
        for (int i = 0; i < S::NL; ++i) da[i] = 0.f;
        asm volatile("" ::: "memory");
#pragma unroll
        for (int r = S::R - 1; r >= 0; --r) {
          float Br[S::NL], Cr[S::NL];
          get_states<S::NL>(Bs + mine + r * S::STEP, Br);
          get_states<S::NL>(Cs + mine + r * S::STEP, Cr);
          gb[r] = qs[r] = 0.f;
#pragma unroll
          for (int i = 0; i < S::NL; ++i) {
            gr[i] = fmaf(Cr[i], dv[r], gr[i]);
            dB[r][i] = fmaf(in[r], gr[i], dB[r][i]);
            gb[r] = fmaf(gr[i], Br[i], gb[r]);
            gr[i] *= f.e[r][i];
            const float p = gr[i] * (left <= r ? 0.f : r ? h[r - 1][i] : f.before[i]);
            qs[r] = fmaf(p, an[i], qs[r]);
            da[i] = fmaf(p, dl[r], da[i]);
          }
        }
        put_sums<S>(gbs + d * S::LD, q, l, gb, g > 0);
        put_sums<S>(qa + d * S::LD, q, l, qs, g > 0);
#pragma unroll
        for (int i = 0; i < S::NL; ++i) {   // the last lane has the row's sum
          da[i] += before<1>(da[i]);
          da[i] += before<2>(da[i]);
          da[i] += before<4>(da[i]);
          da[i] += before<8>(da[i]);
        }
        if (l == kLanes - 1) {
          float all[S::NL];
          get_states<S::NL>(dA + states, all);
#pragma unroll
          for (int i = 0; i < S::NL; ++i) all[i] += da[i];
          put_states<S::NL>(dA + states, all);
        }
      }
      // The waves' dB and dC: the upper half of the waves hand theirs to the lower,
      // whose sums are added up in the waves' order.
      constexpr int HALF = S::NW / 2;
      float* const mine = sums + wave % HALF * 2 * S::TB * S::NS;
      if (S::NG > 1) __syncthreads();   // (the group before has been read)
#pragma unroll
      for (int step = 0; step < 2; ++step) {
        if (wave / HALF == 1 - step)
#pragma unroll
          for (int r = 0; r < S::R; ++r) {
            float* const pB = mine + (q * S::R + r) * S::STEP + l * S::NL;
            float* const pC = pB + S::TB * S::NS;
            if (step) {
              float x[S::NL];
              get_states<S::NL>(pB, x);
#pragma unroll
              for (int i = 0; i < S::NL; ++i) dB[r][i] += x[i];
              get_states<S::NL>(pC, x);
#pragma unroll
              for (int i = 0; i < S::NL; ++i) dC[r][i] += x[i];
            }
            put_states<S::NL>(pB, dB[r]);
            put_states<S::NL>(pC, dC[r]);
          }
        __syncthreads();
      }
      const int thread = anew(tid);
      float* const bc = ws.bc + ((b * blocks_of<S::DW>(a.D, a.G) + w.block) * a.T + t0) * 2 * a.N;
#pragma unroll
      for (int i = 0; i < (8 * S::TB + S::NT - 1) / S::NT; ++i) {   // NL adjacent states of a token, of B, then of C
        const int e = thread + i * S::NT, c = e / (4 * S::TB);
        const int t = e % kLanes * S::R + e / kLanes % S::R, s = g * S::NS + e / S::TB % 4 * S::NL;
        if (e >= 8 * S::TB || s >= a.N || t0 + t >= n) continue;
        float x[S::NL], y[S::NL];
        get_states<S::NL>(sums + e * S::NL, x);
#pragma unroll
        for (int v = 1; v < HALF; ++v) {
          get_states<S::NL>(sums + v * 2 * S::TB * S::NS + e * S::NL, y);
#pragma unroll
          for (int k = 0; k < S::NL; ++k) x[k] += y[k];
        }
        put_states<S::NL>(bc + ((int64_t)t * 2 + c) * a.N + s, x);
      }
    }
    const Pieces<S> me(tid);
    const int c = me.c;
    const float* const skip = tables[0] + c;
    const float* const bias = tables[1] + c;
#pragma unroll
    for (int i = 0; i < S::TURNS; ++i) {
      const int t = me.token(i);
      if (t >= S::TB || c >= w.channels || t0 + t >= a.T) continue;
      Piece r[3];
      r[0].clear();
      r[1].clear();
      r[2].clear();
      if (t0 + t < n) {
        float x[S::PC], v[S::PC], d[S::PC], z[S::PC], o[3][S::PC];
        Piece in[4];
        in[0].load(a.x.p, row(me, a.x, t0 + t));
        in[1].load(a.dt.p, row(me, a.dt, t0 + t));
        in[2].load(a.dy.p, row(me, a.dy, t0 + t));
        in[3].clear();
        if (a.z.p) in[3].load(a.z.p, row(me, a.z, t0 + t));
        in[0].get(x);
        in[1].get(v);
        in[2].get(d);
        in[3].get(z);
#pragma unroll
        for (int e = 0; e < S::PC; ++e) {
          const int at = (c + e) * S::LD + S::at(t);
          const float gb = gbs[at];
          float g = d[e];
          if (a.z.p) {
            const float s = sigmoid(z[e]);
            o[2][e] = d[e] * fmaf(skip[e], x[e], ys[at]) * (s * fmaf(z[e], 1.f - s, 1.f));
            g *= z[e] * s;
          }
          o[1][e] = fmaf(x[e], gb, qa[at] * 0.69314718f);
          if (a.softplus) o[1][e] *= sigmoid(v[e] + bias[e]);
          o[0][e] = fmaf(delta[at], gb, skip[e] * g);
          dskip[e] = fmaf(g, x[e], dskip[e]);
          dbias[e] += o[1][e];
        }
        r[0].set(o[0]);
        r[1].set(o[1]);
        if (a.z.p) r[2].set(o[2]);
      }
      r[0].store(const_cast<void*>(a.dx.p), row(me, a.dx, t0 + t));
      r[1].store(const_cast<void*>(a.ddt.p), row(me, a.ddt, t0 + t));
      if (a.z.p) r[2].store(const_cast<void*>(a.dz.p), row(me, a.dz, t0 + t));
    }
  }

  // rows behind the last block's
  if (const Pieces<S> me(tid); me.c < w.channels) {
    Piece zero;
    zero.clear();
    for (int64_t t = (last + 1) * S::TB + me.token(0); t < a.T; t += S::NT / (S::DW / S::PC)) {
      zero.store(const_cast<void*>(a.dx.p), row(me, a.dx, t));
      zero.store(const_cast<void*>(a.ddt.p), row(me, a.ddt, t));
      if (a.z.p) zero.store(const_cast<void*>(a.dz.p), row(me, a.dz, t));
    }
  }
  __syncthreads();
  for (int i = tid; i < S::DW * S::N; i += S::NT) {
    const int d = i / S::N, s = i % S::N;
    if (d >= w.channels || s >= a.N) continue;
    const int64_t at = b * a.D * a.N + (int64_t)(w.c0 + d) * a.N + s;
    ws.A[at] = dA[i];
    if (a.ds_in) a.ds_in[at] = back[i];
  }
  // dD and dbias: the threads' sums of a channel in 64 bits
  float* const join = reinterpret_cast<float*>(rows4);   // S::PC floats of every thread
  static_assert(S::PC * S::NT <= ROWS * S::DW * S::LD, "the rows hold them");
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < S::PC; ++e) join[tid * S::PC + e] = v ? dbias[e] : dskip[e];
    __syncthreads();
    for (int d = tid; d < w.channels; d += S::NT) {
      double s = 0.0;
      for (int i = d / S::PC; i < S::NT; i += S::DW / S::PC) s += join[i * S::PC + d % S::PC];
      (v ? ws.bias : ws.skip)[b * a.D + w.c0 + d] = (float)s;
    }
  }
}

// dB and dC: the blocks' sums, in 64 bits; zero where no token counts.  A workgroup
// has 16 pairs of adjacent states and the blocks in 16 interleaved shares.
template <bool BF>
__global__ __launch_bounds__(256) void bc_sum_kernel(Scan a, const float* bc, int per) {
  __shared__ double lds[16][32 + 1];
  const int pairs = a.N / 2, share = threadIdx.x / 16, at = threadIdx.x % 16;
  const int64_t all = a.B * a.G * a.T * a.N;
  for (int64_t first = (int64_t)blockIdx.x * 16; first < all; first += (int64_t)gridDim.x * 16) {
    const int64_t id = first + at;   // over [B, G, T, 2, N / 2]
    const int s = (int)(id % pairs) * 2, c = (int)(id / pairs % 2);
    const int64_t t = id / (2 * pairs) % a.T, bg = id / (2 * pairs) / a.T;
    const bool live = id < all;
    double x = 0.0, y = 0.0;
    if (live && t < tokens_of(a.lengths, bg / a.G, a.T)) {
      const float* p = bc + (bg * per * a.T + t) * 2 * a.N + c * a.N + s;
#pragma unroll 4
      for (int i = share; i < per; i += 16) {
        const float2 f = *reinterpret_cast<const float2*>(p + (int64_t)i * a.T * 2 * a.N);
        x += f.x;
        y += f.y;
      }
    }
    __syncthreads();   // (the pairs before have been added up)
    lds[share][2 * at] = x;
    lds[share][2 * at + 1] = y;
    __syncthreads();
    if (share || !live) continue;
    x = y = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      x += lds[i][2 * at];
      y += lds[i][2 * at + 1];
    }
    const Tensor& to = c ? a.dc : a.db;
    const int64_t out = bg / a.G * to.b + t * to.t + bg % a.G * to.h + s;
    if constexpr (BF)
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(const_cast<void*>(to.p)) + out) = linattn::pair((float)x, (float)y);
    else
      *reinterpret_cast<float2*>(static_cast<float*>(const_cast<void*>(to.p)) + out) = make_float2((float)x, (float)y);
  }
}

// dA, dD and dbias: the batch items' sums.
__global__ __launch_bounds__(256) void table_sum_kernel(Scan a, Sums ws) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x, all = (int64_t)a.D * a.N;
  const float* p;
  float* to;
  int64_t at, step;
  if (id < all)
    p = ws.A, to = a.dA, at = id, step = all;
  else if (id < all + a.D)
    p = ws.skip, to = a.dskip, at = id - all, step = a.D;
  else if (id < all + 2 * a.D)
    p = ws.bias, to = a.dbias, at = id - all - a.D, step = a.D;
  else
    return;
  if (!to) return;
  double s = 0.0;
#pragma unroll 8
  for (int64_t b = 0; b < a.B; ++b) s += p[b * step + at];
  to[at] = (float)s;
}

template <class S>
hipError_t launch(const Scan& a, void* workspace, hipStream_t s) {
  const Layout<S> lay(a);
  const Sums ws = lay.in(workspace);
  if (a.B) {
    hipLaunchKernelGGL((a.bf16 ? scan_bwd_kernel<S, true> : scan_bwd_kernel<S, false>),
                       dim3((unsigned)grid_of<S::DW>(a)), dim3(S::NT), 0, s, a, ws, lay.blocks);
    const int64_t pairs = a.B * a.G * a.T * a.N;
    if (pairs)
      hipLaunchKernelGGL((a.bf16 ? bc_sum_kernel<true> : bc_sum_kernel<false>), dim3((unsigned)std::min<int64_t>((pairs + 15) / 16, 1 << 20)),
                         dim3(256), 0, s, a, ws.bc, (int)(blocks_of<S::DW>(a.D, a.G) / a.G));
  }
  const int64_t all = (int64_t)a.D * (a.N + 2);
  hipLaunchKernelGGL(table_sum_kernel, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, a, ws);
  return hipGetLastError();
}

// Calls f with the instance that a call runs on.  Channels of a workgroup: more of
// them share B, C and the sums of dB and dC, as long as there are workgroups for three
// quarters of the CUs.  Us for 1024 tokens of 16 states with 8 / 16 / 32 channels:
//   64 workgroups of 32: 102 / 135 / 198    128: 191 / 140 / 202    192: 299 / 268 / 206
//   256: 405 / 282 / 214    512: 810 / 558 / 425
// More than 16 states leave no room in LDS for 32 channels, 32 of them with 16 channels:
// 652 -> 495 with 512 workgroups of 8.  Tokens of a block are 16 R: 64 x 64 tokens of 2048
// channels with R of 4 and 8 409 / 507 us, 64 x 100 tokens 662 / 524; more than 32 states
// have no room for R = 8.
template <int NL, int R, int NG, int MOST, class F>
auto with_channels(const Scan& a, F f) {
  if constexpr (MOST == 32)
    if (a.B * blocks_of<32>(a.D, a.G) >= 192) return f(Shape<NL, R, NG, 32, 8, 8>());
  if (a.B * blocks_of<16>(a.D, a.G) >= 192) return f(Shape<NL, R, NG, 16, 8, 4>());
  return f(Shape<NL, R, NG, 8, 8, 2>());
}
template <class F>
auto with_shape(const Scan& a, F f) {
  if (a.N > 32) return with_channels<4, 4, 4, 16>(a, f);
  if (a.T <= 64)
    return a.N <= 8 ? with_channels<2, 4, 1, 32>(a, f) : a.N <= 16 ? with_channels<4, 4, 1, 32>(a, f) : with_channels<4, 4, 2, 16>(a, f);
  return a.N <= 8 ? with_channels<2, 8, 1, 32>(a, f) : a.N <= 16 ? with_channels<4, 8, 1, 32>(a, f) : with_channels<4, 8, 2, 16>(a, f);
}

}  // namespace

size_t scan_bwd_workspace_bytes(const Scan& a) {
  return with_shape(a, [&](auto s) { return Layout<decltype(s)>(a).bytes; });
}

hipError_t enqueue_scan_bwd(const Scan& a, void* workspace, hipStream_t stream) {
  return with_shape(a, [&](auto s) { return launch<decltype(s)>(a, workspace, stream); });
}

}  // namespace ssm
