// Internal interface between the C ABI layer (linattn_api.cpp) and the HIP
// kernels of the linear-attention operators.  Not installed; not part of the
// public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace linattn {

constexpr int kChunk = 64;       // tokens of a chunk
// Calls of at most so many tokens run token by token (us, so and in chunks: 2
// tokens of 16 x 32 heads of 64 x 64 5.2 / 8.8, 8 tokens 8.6 / 9.0, 12 10.8 /
// 9.0; of 12 heads 3.7 / 6.6, 6.6 / 6.7, 8.6 / 6.7).
constexpr int kStepTokens = 8;
constexpr int kVBlock = 64;      // value channels one workgroup handles
constexpr int kStepThreads = 256;   // of a workgroup of the token-by-token calls

// Threads of a workgroup of the sweeps of up to KP (64 or 128) key channels.
// LDS holds one float32 workgroup of more than 64 key channels at a time, so
// that one gets a second set of four waves: the outputs' value channels and the
// state's key channels are shared out between the two (gradients of K = 128, V =
// 64, 2 x 777 tokens: 64.6 -> 61.6 us; prompts of 128 x 128: 100.5 -> 95.4).
// With K = 64 two workgroups fit, and eight waves of one are slower (60 -> 74 us).
constexpr int sweep_threads(int KP, bool bf16) { return KP == 128 && !bf16 ? 512 : 256; }

// A [B, T, H, D] tensor: base and distances in elements (channels adjacent).
struct Tensor {
  const void* p;
  int64_t b, t, h;
};

// One sweep of the recurrence over all sequences, forwards or from the last
// token to the first.  With M the state as the sweep meets it (multiplied by
// the decay once already where the sweep runs backwards), per token in sweep
// order:
//
//   forward:   M <- a M + us k^T v;   o = q (is a M_before + ps k^T v)
//   backward:  o = q (is M + ps k^T v);   M <- a (M + us k^T v)
//
// and earlier tokens of the sweep reach later ones through M.  The forward
// operator is the forward sweep with us = 1, is = ps = scale; its gradients
// are three sweeps over other triples of tensors.
struct Sweep {
  int64_t B, T, H;
  int K, V;                 // channels of q and k; of v and o
  Tensor q, k, v, o;
  const float* log_decay;   // [H]
  const int32_t* lengths;   // [B] or null
  float us, is, ps;
  const float* s_in;        // [B, H] states of K * V floats, or null
  float* s_out;             // the same, or null
  bool s_transposed;        // states are stored [V][K] (the sweep's K, V) instead of [K][V]
  bool reverse;
  bool bf16;                // q, k, v
  bool out_bf16;
};

__host__ __device__ inline int vblocks_of(const Sweep& a) { return (a.V + kVBlock - 1) / kVBlock; }

// Up to three sweeps over the same sequences, types and product K V, run side
// by side: none reads what another writes, except that the last one's s_out
// may be another one's s_in.
constexpr int kSweeps = 3;
size_t sweep_workspace_bytes(const Sweep* a, int n);
// `workspace`: sweep_workspace_bytes bytes, or null where that is 0.
hipError_t enqueue_sweeps(const Sweep* a, int n, void* workspace, hipStream_t stream);

// How sweeps are laid over the card.
struct SweepPlan {
  Sweep a[kSweeps];
  int sweeps;
  float* ws;        // [sweeps][B H][segments] states of segments; null for one segment
  int segments;     // of each sequence
  int seg_tokens;   // tokens of a segment, a multiple of 64
  int vblocks;      // blocks of 64 value channels, the most of the sweeps
  int blocks;       // blocks of value channels of all sweeps
  int64_t pairs;    // B H
  int64_t items;    // pairs * segments
};
// Workgroups of a launch over `items` items: eight of them side by side, see the
// kernel.
inline int64_t sweep_groups(const SweepPlan& p, int64_t items) { return (items + 7) / 8 * 8 * p.blocks; }
hipError_t launch_sweeps64(const SweepPlan& p, hipStream_t s);    // K <= 64 in all sweeps
hipError_t launch_sweeps128(const SweepPlan& p, hipStream_t s);

// n floats from `from` (zeros where it is null) to `to`; n is a multiple of 4.
hipError_t enqueue_state_copy(const float* from, float* to, int64_t n, hipStream_t stream);

struct Rope {
  int64_t B, T, H;
  int D, R;
  Tensor q, k, q_out, k_out;   // k.p null: q alone
  const int32_t* positions;    // [B, T] or null
  int64_t start;
  const double* freqs;         // [R / 2]
  bool interleaved, inverse, bf16;
};
hipError_t enqueue_rope(const Rope& a, hipStream_t stream);

struct Norm {
  int64_t rows, C;
  const void* x;
  const void* residual;   // or null
  const float* weight;
  float eps;
  void* h;                // or null
  void* y;                // normalised rows, or null with codes
  uint8_t* codes;
  float* scales;
  int group;              // columns that share a scale: 128, or 0 for the row
  bool bf16;
};
hipError_t enqueue_norm(const Norm& a, hipStream_t stream);

struct NormBwd {
  int64_t rows, C;
  const void* dy;
  const void* h;
  const void* dh;   // or null
  const float* weight;
  float eps;
  void* dx;
  float* dweight;
  bool bf16;
};
size_t norm_bwd_workspace_bytes(const NormBwd& a);
hipError_t enqueue_norm_bwd(const NormBwd& a, void* workspace, hipStream_t stream);

}  // namespace linattn
