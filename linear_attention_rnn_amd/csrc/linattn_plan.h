// How the attention calls are laid over the card: host arithmetic only, shared
// by the argument checks, the launches and the tests that run without a GPU.
#pragma once

#include <algorithm>

#include "linattn_internal.h"

namespace linattn {

inline bool steps(const Sweep* a, int n) { return n == 1 && a->T <= kStepTokens && !a->reverse && !a->s_transposed; }

// The most key channels of the sweeps: they run with 64 or 128 for all.
inline int widest(const Sweep* a, int n) {
  int K = 0;
  for (int i = 0; i < n; ++i) K = std::max(K, a[i].K);
  return K;
}

// Sweeps of at most and of more than 64 key channels in launches of their own,
// the last sweep's second: float32 gradients of more than one round of
// workgroups, for the narrow ones take two thirds of the time and two fit a CU.
// Us, together / so, of 4 x 1000 tokens, 32 heads of 128 x 64 (640 workgroups)
// 321 / 210, 15 x 2064, 8 of 32 x 96 (480) 440 / 369, 14 x 40, 12 of 128 x 32 36.9
// / 28.0; with fewer than 256 (2 x 777, 8 of 128 x 64) 58 / 73; in bfloat16, 8 x
// 512 tokens, 16 of 64 x 128 53 / 62, 15 x 2064, 8 of 32 x 96 171 / 200.
struct Split {
  Sweep a[2][kSweeps];
  int n[2] = {0, 0};
};
inline Split split(const Sweep* a, int n) {
  Split s;
  int64_t groups = 0;
  bool wide = false, narrow = false;
  for (int i = 0; i < n; ++i) {
    groups += vblocks_of(a[i]) * a->B * a->H;
    (a[i].K > 64 ? wide : narrow) = true;
  }
  if (a->bf16 || !wide || !narrow || groups <= 256) return s;
  const bool last = a[n - 1].K > 64;
  for (int i = 0; i < n; ++i) {
    const int g = (a[i].K > 64) == last;
    s.a[g][s.n[g]++] = a[i];
  }
  return s;
}

inline SweepPlan plan(const Sweep* a, int n) {
  SweepPlan p = {};
  p.sweeps = n;
  p.vblocks = 1;
  for (int i = 0; i < n; ++i) {
    p.a[i] = a[i];
    const int vb = vblocks_of(a[i]);
    p.vblocks = std::max(p.vblocks, vb);
    p.blocks += vb;
  }
  p.pairs = a->B * a->H;
  const int64_t chunks = (a->T + kChunk - 1) / kChunk, groups = p.pairs * p.blocks;
  // Segments cost a second pass over keys and values, so they are for calls
  // that leave CUs idle: below 160 workgroups, up to two for each of the 256
  // CUs, and with lengths, which leave later segments short or empty, up to the
  // next multiple (float32 gradients of 24 heads, 72 workgroups: 7 segments 82,
  // 8 101; 7 x 4880 tokens of 16 heads with lengths: 4 segments 201, 5 174).
  // Otherwise measured, us, with 1 / 4 / 8 / 16 / 64 segments: 192 workgroups
  // (gradients, 64 chunks) 101 / 108 / 119 / 129 / 240; 64 of them (64 chunks)
  // 155 / 77 / 73 / 78 / 116; 32 (128 chunks of K = V = 128) 301 / 139 / 88 / 81 /
  // 121; 2 (256 chunks) 380 / 171 / 95 / 58 / 36, and 41 with 128.  They have
  // three chunks at least, for calls of eight (8 heads, us, two / three / four
  // chunks: of 512 tokens 15.3 / 15.9 / 19.4, of 1024 17.1 / 16.5 / 19.9, of 4096
  // 24.3 / 22.5 / 24.3; 5 chunks, one segment / two: 15.0 / 18.6); two where
  // chunks take longer, in float32.  A CU holds one workgroup of the float32
  // sweeps of more than 64 key channels at a time, so those stay in one round
  // of 256 (gradients of K = 128, V = 64, 13 chunks: 73 us with 3 segments, 80
  // with 5).
  int64_t G = groups >= 160 ? 1 : (512 + (a->lengths ? groups - 1 : 0)) / groups;
  if (!a->bf16 && widest(a, n) > 64 && G > 1) G = 256 / groups;
  G = std::max<int64_t>(1, std::min(G, !a->bf16 ? chunks / 2 : chunks < 8 ? 1 : (chunks + 2) / 3));
  const int64_t per = (chunks + G - 1) / G;
  p.seg_tokens = (int)(per * kChunk);
  p.segments = (int)((chunks + per - 1) / per);
  p.items = p.pairs * p.segments;
  return p;
}

// What segments of a plan keep: [sweeps][B H][segments] states.
inline size_t planned_workspace_bytes(const Sweep* a, int n) {
  if (steps(a, n)) return 0;
  if (const Split s = split(a, n); s.n[0])
    return std::max(planned_workspace_bytes(s.a[0], s.n[0]), planned_workspace_bytes(s.a[1], s.n[1]));
  const SweepPlan p = plan(a, n);
  if (p.segments == 1) return 0;
  return (size_t)n * p.items * (widest(a, n) <= 64 ? 64 : 128) * kVBlock * p.vblocks * 4;
}

// Work-items of the largest launch of a call; a launch holds fewer than 2^32.
inline int64_t largest_launch(const Sweep* a, int n) {
  if (steps(a, n)) return a->B * a->H * vblocks_of(*a) * kStepThreads;
  if (const Split s = split(a, n); s.n[0])
    return std::max(largest_launch(s.a[0], s.n[0]), largest_launch(s.a[1], s.n[1]));
  const SweepPlan p = plan(a, n);
  return sweep_groups(p, p.items) * sweep_threads(widest(a, n) <= 64 ? 64 : 128, a->bf16);
}

}  // namespace linattn
