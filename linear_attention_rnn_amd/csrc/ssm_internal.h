// Internal interface between the C ABI layer (ssm_api.cpp) and the HIP kernels
// of the selective state space layer.  Not installed; not part of the public
// ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "linattn_internal.h"

namespace ssm {

using linattn::Tensor;   // [B, T, places, channels]: base and distances in elements

struct Conv {
  int64_t B, T;
  int D, W;
  Tensor x, y;              // y: dx in the gradients
  Tensor dy;                // gradients only
  const float* weight;      // [D, W]
  const float* bias;        // [D] or null
  const int32_t* lengths;   // [B] or null
  const void* s_in;         // [B, W - 1, D] of x's type, or null
  void* s_out;              // the same, or null
  const void* ds_out;       // gradients: of s_out, or null
  void* ds_in;              // of s_in, or null
  float* dweight;
  float* dbias;             // or null
  bool silu, bf16;
};
hipError_t enqueue_conv(const Conv& a, hipStream_t stream);
size_t conv_bwd_workspace_bytes(const Conv& a);
hipError_t enqueue_conv_bwd(const Conv& a, void* workspace, hipStream_t stream);

struct Scan {
  int64_t B, T;
  int D, N, G;
  Tensor x, dt, b, c, z, y;   // z.p may be null; y: null in the gradients
  const float* A;             // [D, N]
  const float* skip;          // [D] or null
  const float* bias;          // [D] or null
  bool softplus;
  const int32_t* lengths;     // [B] or null
  const float* s_in;          // [B, D, N] or null
  float* s_out;               // the same, or null
  bool bf16;
  // gradients
  Tensor dy, dx, ddt, db, dc, dz;   // dz.p null with z.p
  const float* ds_out;              // or null
  float* ds_in;                     // or null
  float* dA;
  float* dskip;                     // or null
  float* dbias;                     // or null
};
hipError_t enqueue_scan(const Scan& a, hipStream_t stream);
size_t scan_bwd_workspace_bytes(const Scan& a);
hipError_t enqueue_scan_bwd(const Scan& a, void* workspace, hipStream_t stream);

enum Activation { kNone = 0, kSilu = 1, kSigmoid = 2 };

struct BlockNorm {
  int64_t rows, C;
  const void* x;
  const void* residual;    // or null
  const void* gate;        // [rows / gate_rows, C] or null
  int64_t gate_rows;       // rows that share a row of the gate
  const float* post;       // or null
  const float* pre;        // or null
  float scale, eps;
  Activation act;
  void* h;
  void* y;                 // null without pre
  bool bf16;
  // gradients (h: the forward's)
  const void* dy;          // null without pre
  const void* dh;          // or null
  void* dx;
  void* dresidual;         // or null
  void* dgate;             // null without gate
  float* dpost;
  float* dpre;
};
hipError_t enqueue_block_norm(const BlockNorm& a, hipStream_t stream);
size_t block_norm_bwd_workspace_bytes(const BlockNorm& a);
hipError_t enqueue_block_norm_bwd(const BlockNorm& a, void* workspace, hipStream_t stream);

}  // namespace ssm
