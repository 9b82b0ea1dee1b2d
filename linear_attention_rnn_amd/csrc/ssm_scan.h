// The selective scan over blocks of tokens, shared by the forward kernel and
// the gradients.  Per channel d and state n, with the step delta_t = softplus(dt_t
// + bias):
//
//   h_t = exp(delta_t A) h_{t-1} + delta_t x_t B_t,   y_t = sum_n C_t h_t
//
// A wave holds one channel over a block of 16 R tokens: lane (q, l) = (lane /
// 16, lane % 16) has the R tokens from l R on and the NL states from q NL on, so
// that four lanes hold a token's states.  B and C of its tokens and states are the
// same for every channel of a group; they are read from LDS for each, since
// registers for them would halve the waves (441 -> 400 us for 8 x 4096 tokens of 2048
// channels).  Per channel:
//   1. decays e = exp(delta A) and inputs u = delta x B of the lane, its own
//      state H from zero, its decay P = exp(A sum delta);
//   2. the 16 lanes' (P, H) are combined in four doubling steps within a row of
//      16 lanes, and the state at the block's start joins them, decayed by exp(A
//      (sum of all steps up to there)): one rounding for a block, where the product of a
//      token's decays would be off the same way at every token;
//   3. the lane goes through its tokens again from the state in front of them.
// Decays and inputs stay in registers between 1 and 3: 2 more instructions for
// each token and state than a walk over the tokens, and the scan's, for 16 times
// as many lanes.  Bound by the vector instructions: per token and state about 8, an
// exp among them that takes four times as long as another one, and about 70 per token and
// channel for softplus and gate.  A lone wave issues one in 5 to 8 clocks, four waves of a
// SIMD one in 3: so the kernels take few registers before they save instructions.  More
// than 16 states go group after group, whose registers are then those of 16.
#pragma once

#include "ssm_device.h"

namespace ssm {
namespace {

constexpr int kLanes = 16;   // lanes over a block's tokens

// Sizes of one instance: NL states and R tokens a lane, up to NG groups of 4 NL
// states one after another, DW channels and NW waves a workgroup, PC channels that
// a thread loads of a token.
template <int NL_, int R_, int NG_, int DW_, int NW_, int PC_>
struct Shape {
  static constexpr int NL = NL_, R = R_, NG = NG_, DW = DW_, NW = NW_, PC = PC_;
  static constexpr int NS = 4 * NL, N = NG * NS, TB = kLanes * R, NT = 64 * NW;
  static constexpr int V = R < 4 ? R : 4;       // tokens of one access to a channel's row
  static constexpr int LD = TB + 4;             // floats of a channel's row
  static constexpr int PIECES = TB * (DW / PC);
  static constexpr int TURNS = (PIECES + NT - 1) / NT;
  static constexpr int BPIECES = TB * (N / 8);  // of 8 states of a token
  static constexpr int BTURNS = (BPIECES + NT - 1) / NT;
  // Where token t of a block lies in a channel's row: the lanes' first four tokens
  // side by side, then their next, so that a wave reads whole lines; the next are
  // shifted by four lanes, so that adjacent tokens of a thread's neighbours meet in
  // no bank.
  static __device__ __forceinline__ int at(int t) {
    if constexpr (R <= 4)
      return t;
    else
      return t % R / 4 * (4 * kLanes) + half(t / R, t % R) + t % 4;
  }
  static __device__ __forceinline__ int half(int l, int r) { return (l ^ (r & 4)) * 4; }
  // Where B and C of token t, states from n on, lie: group after group, lanes side
  // by side.
  static __device__ __forceinline__ int at(int t, int n) { return (n / NL * R + t % R) * STEP + t / R * NL + n % NL; }
  static constexpr int STEP = kLanes * NL;   // from one of a lane's tokens to the next
  // Token and first state of a thread's piece of B and C: those of a wave lie side by
  // side in LDS.
  static __device__ __forceinline__ int piece_token(int p) { return p % kLanes * R + p / kLanes % R; }
  static __device__ __forceinline__ int piece_state(int p) { return p / TB * 8; }
};

// A lane's tokens of a channel's row.
template <class S>
__device__ __forceinline__ void get_tokens(const float* row, int l, float (&x)[S::R]) {
#pragma unroll
  for (int i = 0; i < S::R; i += S::V) {
    const float* p = row + i / 4 * (4 * kLanes) + (S::R > 4 ? S::half(l, i) : l * S::V);
    if constexpr (S::V == 4) {
      const float4 f = *reinterpret_cast<const float4*>(p);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    } else {
      const float2 f = *reinterpret_cast<const float2*>(p);
      x[i] = f.x, x[i + 1] = f.y;
    }
  }
}

template <int NL>
__device__ __forceinline__ void get_states(const float* p, float (&x)[NL]) {
  if constexpr (NL == 2) {
    const float2 f = *reinterpret_cast<const float2*>(p);
    x[0] = f.x, x[1] = f.y;
  } else {
#pragma unroll
    for (int i = 0; i < NL; i += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + i);
      x[i] = f.x, x[i + 1] = f.y, x[i + 2] = f.z, x[i + 3] = f.w;
    }
  }
}
// B or C of a lane's tokens in group g.
template <class S>
__device__ __forceinline__ void get_block(const float* p, int g, int q, int l, float (&x)[S::R][S::NL]) {
#pragma unroll
  for (int r = 0; r < S::R; ++r) get_states<S::NL>(p + ((g * 4 + q) * S::R + r) * S::STEP + l * S::NL, x[r]);
}
template <int NL>
__device__ __forceinline__ void put_states(float* p, const float (&x)[NL]) {
  if constexpr (NL == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int i = 0; i < NL; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  }
}

// Sums over the four lanes of a token's states, put into the lane's channel row
// at its tokens, or added to what earlier groups of states left there.  The lane exchanges add up two
// tokens at a time.
template <class S>
__device__ __forceinline__ void put_sums(float* row, int q, int l, const float (&y)[S::R], bool add) {
  const auto put = [&](float* at, float z) { *at = S::NG > 1 && add ? *at + z : z; };
  if constexpr (S::R == 2) {
    const float w = halves_sum(y[0], y[1]);
    const float z = rows16_sum(w, w);   // rows 0, 1: the first token, 2, 3: the second
    if (q % 2 == 0) put(row + 2 * l + q / 2, z);
  } else {
#pragma unroll
    for (int i = 0; i < S::R; i += 4) {
      const float z = rows16_sum(halves_sum(y[i], y[i + 1]), halves_sum(y[i + 2], y[i + 3]));
      // rows 0 to 3 hold tokens 0, 2, 1, 3
      put(row + i / 4 * (4 * kLanes) + S::half(l, i) + (q % 2 * 2 + q / 2), z);
    }
  }
}

// A channel's decays and inputs of a lane, and the state in front of its
// tokens.  h0: the state at the block's start; returns in `end` (of the last lane)
// that at its end.
template <class S>
struct Walk {
  float e[S::R][S::NL], u[S::R][S::NL];
  float before[S::NL], end[S::NL];
  float sum, total;   // of the lane's steps, and of all up to its last token

  __device__ __forceinline__ void run(const float (&delta)[S::R], const float (&ux)[S::R], const float (&a2)[S::NL],
                                      const float (&B)[S::R][S::NL], const float (&h0)[S::NL]) {
    float H[S::NL], P[S::NL];
    sum = delta[0];
#pragma unroll
    for (int r = 1; r < S::R; ++r) sum += delta[r];
#pragma unroll
    for (int r = 0; r < S::R; ++r)
#pragma unroll
      for (int i = 0; i < S::NL; ++i) {
        e[r][i] = __builtin_amdgcn_exp2f(delta[r] * a2[i]);
        u[r][i] = ux[r] * B[r][i];
        H[i] = r ? fmaf(e[r][i], H[i], u[r][i]) : u[r][i];
      }
#pragma unroll
    for (int i = 0; i < S::NL; ++i) P[i] = __builtin_amdgcn_exp2f(sum * a2[i]);
    total = sum;
    scan<1>(H, P);
    scan<2>(H, P);
    scan<4>(H, P);
    scan<8>(H, P);
#pragma unroll
    for (int i = 0; i < S::NL; ++i) {
      end[i] = fmaf(__builtin_amdgcn_exp2f(total * a2[i]), h0[i], H[i]);
      before[i] = before_or(end[i], h0[i]);
    }
  }

 private:
  // (A lane with none before it gets P = 0, which nothing but 0 is multiplied by
  // from there on.)
  template <int K>
  __device__ __forceinline__ void scan(float (&H)[S::NL], float (&P)[S::NL]) {
    total += ssm::before<K>(total);
    add_before<K>(H, P);
    if constexpr (K < 8)
#pragma unroll
      for (int i = 0; i < S::NL; ++i) P[i] *= ssm::before<K>(P[i]);
  }
};

// x, but what is computed from it is computed where it is used: addresses of the
// phases around the walk over the channels would keep dozens of registers through
// it, which cost waves.
__device__ __forceinline__ int anew(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A thread's pieces of a block: S::PC channels from c on of the tokens token(i).
template <class S, bool ANEW = true>
struct Pieces {
  int tid, c;
  __device__ __forceinline__ explicit Pieces(int thread) : tid(ANEW ? anew(thread) : thread), c(tid % (S::DW / S::PC) * S::PC) {}
  __device__ __forceinline__ int token(int i) const { return (tid + i * S::NT) / (S::DW / S::PC); }   // from S::TB on: none
  // The number of its pieces of B and C: from the other half of the threads on, where
  // there are fewer pieces of either kind than threads.
  __device__ __forceinline__ int state_piece(int i) const { return (tid ^ (S::NT / 2)) + i * S::NT; }
};

// Where a workgroup works: a batch item, a group and up to DW of its channels.
// Workgroups of neighbouring channels, which share lines of the rows, are on one
// XCD: consecutive numbers go to the XCDs in turn.
struct Where {
  int64_t b;
  int g, c0, channels;   // group, first channel, channels (a multiple of 8)
  int64_t block;         // number of the block of channels, from 0 in every batch item
  bool live;
};
template <int DW>
__host__ __device__ __forceinline__ int64_t blocks_of(int D, int G) {
  return (int64_t)G * ((D / G + DW - 1) / DW);
}
template <int DW>
__device__ __forceinline__ Where where_of(int64_t B, int D, int G) {
  const int per = (D / G + DW - 1) / DW;
  const int64_t all = B * G * per, side = (all + 7) / 8;
  const int64_t id = blockIdx.x % 8 * side + blockIdx.x / 8;
  Where w;
  w.live = id < all;
  w.b = id / (G * per);
  w.block = id % (G * per);
  w.g = (int)(w.block / per);
  const int at = (int)(w.block % per) * DW;
  w.c0 = w.g * (D / G) + at;
  w.channels = D / G - at < DW ? D / G - at : DW;
  return w;
}
// Workgroups of a launch.
template <int DW>
int64_t grid_of(const Scan& a) {
  return (a.B * blocks_of<DW>(a.D, a.G) + 7) / 8 * 8;
}

}  // namespace
}  // namespace ssm
