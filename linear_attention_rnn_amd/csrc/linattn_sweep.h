// Linear attention with one decay for each head: the chunked sweep on matrix
// cores and its segment carries.  Included by the files that instantiate
// it (linattn_sweep64.hip, linattn_sweep128.hip).
//
// Mathematics, for a chunk of n <= 64 tokens in sweep order with the state M
// (K x V) entering it, a the decay, d = 0 for the forward sweep and 1 for the
// reversed one (whose state carries one decay more):
//
//   o_j = is a^(j+1-d) q_j M  +  sum_{i<=j} ps a^(j-i) (q_j . k_i) v_i
//   M  <- a^n M  +  sum_i k_i^T (us a^(n-1-i+d) v_i)
//
// All exponents are >= 0, so every factor is at most 1 for a decay a <= 1.
//
// A workgroup of four waves (eight: see sweep_threads()) runs one (batch item,
// head, block of 64 value channels, segment).  Wave w computes the outputs of tokens
// 16w..16w+15 (all 64 channels, transposed: O^T[n][t]) and keeps the state's
// columns of its strip of 16 value channels in registers.  MFMA operands chain
// without a detour: scores come out as K Q^T tiles whose accumulator lanes are,
// tile pairs taken together, the operand lanes of the product with V^T; the
// state's accumulators are the operand lanes of the product with q.  Only the
// state crosses waves, through LDS as ready-made operand fragments.
//
// The rows of an MFMA tile may be any 16 channels as long as both sides of a
// product agree: "tile pairs" (2u, 2u+1) hold channels 32u + 8(m/4) + m%4 and
// those + 4 in row m, so that a lane's values of both tiles are 8 adjacent
// channels: a 16-byte operand of q, and 16-byte stores of bfloat16 outputs.
//
// Operand parts: bfloat16 inputs are one part, float32 inputs three.  MP parts
// carry what arises in between (scores times decays, the state as it meets
// q): one where the output is bfloat16 too (each adds a rounding of the size
// of the output's own, 2^-8, to the part of the output it carries), three
// where it is float32.  Two parts would leave the output's own rounding alone
// (errors of 1.66e-3, one part 2.35e-3) and cost prompts of 256 heads 124 -> 132
// us, prompts of 128 x 128 88 -> 106, gradients of 64 heads 108 -> 128.  The
// decayed values of the state's update are always three parts, so that outputs
// do not depend on whether the state is asked for (with two parts where it is
// not: the prompts 124 and 82 us, the gradients 103).
//
// What bounds it.  256 heads of 4096 tokens and 64 channels in bfloat16: 125 us,
// 4.3 TB/s, where a kernel that only loads and stores the same 128-byte pieces 4
// KiB apart takes 118 us; with each head's rows adjacent 110 us, 4.9 TB/s (a
// copy: 5.1).  The gradients of the same 324 us for 1.41 GB (the sweeps run both
// ways, so q, k, v and d_o come from memory nearly twice), 4.4 TB/s.  With fewer
// workgroups than CUs a chunk's own chain of steps sets the time, 3450 cycles of
// K = V = 64 and 5400 of K = 128 (float32: three to four times that, for six
// products of parts).
#pragma once

#include "linattn_internal.h"
#include "wkv6_device.h"

namespace linattn {
namespace {

using wkv6::bf16x4;
using wkv6::bf16x8;
using wkv6::ex2;
using wkv6::f32x4;
using wkv6::ld_tr;
using wkv6::lds_barrier;
using wkv6::mma;
using wkv6::Op;
using wkv6::Rsrc;
using wkv6::swz;

constexpr int kPlane = 64 * 64;   // a part of 64 rows of 64 channels

// log2 of the decay, finite: the factor of any distance > 0 is 0 at -4096.
__device__ __forceinline__ float log2_decay(float ld) { return ld < -2839.f ? -4096.f : ld * 1.44269504f; }

// The decay over d tokens; 0 where d is negative.
__device__ __forceinline__ float decayed(float gl, int d) {
  const float e = ex2(gl * (d < 0 ? 0 : d));
  return d < 0 ? 0.f : e;
}

// The decay a^n of a state over n tokens, in two float32 parts: rounded to one
// it would be off by up to 2^-25 the same way at every step, and a state that
// lives for 1 / (1 - a^n) steps by as many times that (after 4096 chunks with
// decays of 1e-6 to 3.2e-4 a token 4e-5 to 9e-5).  Both parts are positive, so
// that an infinite state stays what it is.
//
// SEGMENT: a decay above 1 grows out of float32 over a long segment (over a chunk
// it must not).  Then it is applied as three factors that do not: a state of 0
// stays 0, and any other one, of 2^-149 or more, becomes infinite.
template <bool SEGMENT>
struct Decay {
  float hi, lo;   // or the third root and 0
  bool large;
  __device__ __forceinline__ Decay(float ld, float n) {
    const double e = (double)ld * n;
    double a = exp(e);
    large = a > 3.4028234663852886e38;
    if (SEGMENT && large) a = exp(fmin(e, 250.0) / 3.0);
    float h = (float)a;
    if (!large && (double)h >= a && h > 0.f) h = __uint_as_float(__float_as_uint(h) - 1);   // the next float32 below
    hi = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(h)));   // the same for a workgroup
    lo = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(large ? 0.f : (float)(a - (double)h))));
  }
  __device__ __forceinline__ f32x4 operator()(f32x4 m) const {
    if (SEGMENT && large) return m * hi * hi * hi;
#pragma unroll
    for (int r = 0; r < 4; ++r) m[r] = fmaf(hi, m[r], lo * m[r]);   // (hi m rounded would drop lo m)
    return m;
  }
};

__device__ __forceinline__ int64_t tokens_of(const Sweep& a, int64_t b) {
  if (!a.lengths) return a.T;
  const int64_t n = a.lengths[b];
  return n < 0 ? 0 : n > a.T ? a.T : n;
}

// A tensor's rows of one (batch item, head) as a sweep meets them, 64 at a
// time: `at` points at the chunk's first row in memory order (before the
// tensor's start where a reversed sweep's last chunk is short; those rows are
// masked) and moves by a constant from chunk to chunk, so that a lane's
// offsets never change.
struct Rows {
  const char* at;
  int64_t step;   // bytes from a chunk to the next
  int stride;     // bytes from a row to the next one of the sweep, ...
  int base;       // ... and of row 0

  __device__ __forceinline__ void start(const Tensor& x, int64_t b, int64_t h, int64_t lo, int64_t len, bool rev, int isz) {
    const int64_t row = x.t * isz, first = rev ? len - lo - kChunk : lo;
    at = static_cast<const char*>(x.p) + (b * x.b + h * x.h) * isz + first * row;
    step = rev ? -kChunk * row : kChunk * row;
    stride = rev ? -(int)row : (int)row;
    base = rev ? (kChunk - 1) * (int)row : 0;
  }
  // byte offset of row j, channel c; out of range for channels behind the last
  __device__ __forceinline__ int offset(int j, int c, int D, int isz) const {
    return c < D ? base + j * stride + c * isz : wkv6::kOffNone;
  }
  __device__ __forceinline__ Rsrc rsrc() const {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(at), (short)0, wkv6::kOffNone, wkv6::kRsrcFlags);
  }
};

// Eight adjacent channels as loaded: 16 bytes of bfloat16 or 32 of float32.
template <bool BF>
struct Raw8 {
  uint4 q[BF ? 1 : 2];
};

template <bool BF>
__device__ __forceinline__ Raw8<BF> load8(Rsrc r, int off) {
  Raw8<BF> x;
  x.q[0] = wkv6::bload16(r, off);
  if constexpr (!BF) x.q[1] = wkv6::bload16(r, off + 16);
  return x;
}

template <bool BF>
__device__ __forceinline__ Op<BF ? 1 : 3> operand(const Raw8<BF>& x) {
  if constexpr (BF) {
    Op<1> o;
    o.p[0] = __builtin_bit_cast(bf16x8, x.q[0]);
    return o;
  } else {
    float f[8];
    __builtin_memcpy(f, x.q, 32);
    return wkv6::split8<3>(f);
  }
}

template <bool BF>
__device__ __forceinline__ void stage8(__bf16* plane, int stride, int off, const Raw8<BF>& x) {
  const Op<BF ? 1 : 3> o = operand<BF>(x);
#pragma unroll
  for (int s = 0; s < (BF ? 1 : 3); ++s) *reinterpret_cast<bf16x8*>(plane + s * stride + off) = o.p[s];
}

template <int S>
__device__ __forceinline__ Op<S> read8(const __bf16* p, int stride, int off) {
  Op<S> o;
#pragma unroll
  for (int s = 0; s < S; ++s) o.p[s] = *reinterpret_cast<const bf16x8*>(p + s * stride + off);
  return o;
}

// Two transposed reads: slots 0..3 from the rows of `o0`, 4..7 from those of `o1`.
template <int S>
__device__ __forceinline__ Op<S> read_tr(const __bf16* p, int stride, int o0, int o1) {
  Op<S> o;
#pragma unroll
  for (int s = 0; s < S; ++s) {
    const bf16x4 a = ld_tr(p + s * stride + o0), b = ld_tr(p + s * stride + o1);
    o.p[s] = bf16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  }
  return o;
}

// Where a segment's state lies in the workspace: the wave's accumulators as
// they are, [block of values][wave][J][e][lane][r], so that a lane moves 16
// bytes at a time (element by element, 32 loads of a 128 x 64 state took as
// long as a chunk).
template <int KP>
__device__ __forceinline__ int64_t segment_state(const SweepPlan& p, int sweep, int64_t pair, int seg) {
  return ((sweep * p.pairs + pair) * p.segments + seg) * (KP * kVBlock * p.vblocks);
}

// Up to so many segments, each adds up the earlier ones' states by itself;
// more get theirs from the carry kernel.  Measured, us, so and with the kernel:
// 4 segments (float32, 6 x 1023 tokens, V = 96) 59.7 / 64.0, 3 (float32
// gradients, K = 128) 64.8 / 67.9; 16 (8192 tokens of 16 heads of 128 x 128)
// 79.8 / 73.7, 128 40.3 / 31.0.
constexpr int kJoin = 8;

// Waves a SIMD: three of the bfloat16 sweeps of 64 key channels (168 registers,
// 24 or 41 KB of LDS a workgroup; a fourth would spill), else two, by registers
// (bfloat16 of 128 key channels: 218) or LDS (float32: 74 KB of 64 key channels;
// 123 KB of 128, eight waves of one workgroup).
template <int KP, bool BF>
constexpr int occupancy() {
  return KP == 64 && BF ? 3 : 2;
}

template <int KP, bool BF, int MP, bool OBF, bool SUMMARY>
__global__ __launch_bounds__(sweep_threads(KP, BF), (occupancy<KP, BF>())) void sweep_kernel(SweepPlan p) {
  constexpr int NT = sweep_threads(KP, BF), PARTS = NT / 256;
  constexpr int NI = BF ? 1 : 3;             // parts of an input operand
  constexpr int ISZ = BF ? 2 : 4;
  constexpr int NJ = KP / 32;                // groups of 32 key channels
  constexpr int KPL = (KP / 64) * kPlane;    // one part of the keys
  constexpr int KR = KP * 8 / NT;            // key chunks of 8 channels a thread loads
  constexpr int VR = 512 / NT;
  constexpr int MJ = NJ / PARTS, OU = 2 / PARTS;
  __shared__ __bf16 Kp[NI * KPL];
  __shared__ __bf16 Vp[NI * kPlane];
  __shared__ __bf16 Sp[SUMMARY ? 8 : MP * KP * 64];

  // The sweeps and blocks of values of one item, which read the same rows, are
  // 8 apart, so that they run on one XCD and share its L2.  None is without
  // work: workgroups go to the shader engines in turn whatever they do, and
  // idle ones in a pattern left some engines two rounds and others none
  // (float32 gradients of K = 64, V = 96: 144 us, now 82).
  const int64_t item = (int64_t)(blockIdx.x / (8 * p.blocks)) * 8 + blockIdx.x % 8;
  int sweep = 0, vb = blockIdx.x / 8 % p.blocks;
  for (int i = 0; i + 1 < kSweeps && vb >= vblocks_of(p.a[sweep]); ++i) vb -= vblocks_of(p.a[sweep++]);
  const int v0 = vb * kVBlock;
  const Sweep& a = p.a[sweep];
  const bool rev = a.reverse;
  if (item >= p.items) return;
  const int segs = SUMMARY ? p.segments - 1 : p.segments;
  const int64_t pair = item / segs;
  const int seg = (int)(item % segs);
  const int64_t b = pair / a.H, h = pair % a.H;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = wave >> 2, w = wave & 3;        // of the state: strip w, its key groups MJ * part..
  const int tb = part ? 3 - w : w;                 // of the outputs: tokens 16 tb.., values 32 OU part..
  const float ld = a.log_decay[h], gl = log2_decay(ld);

  const int64_t len = tokens_of(a, b);
  const int64_t lo = (int64_t)seg * p.seg_tokens;
  const int64_t hi = lo + p.seg_tokens < len ? lo + p.seg_tokens : len;
  const int nch = lo < hi ? (int)((hi - lo + kChunk - 1) / kChunk) : 0;

  const Decay<false> whole(ld, kChunk), last(ld, (float)(hi - lo - (int64_t)(nch - 1) * kChunk));   // of a chunk, of the last one

  // ---- the entering state: rows c = 32J + 8g + 4e + r, column n of strip w
  f32x4 M[MJ][2];
  const int sn = v0 + 32 * (w >> 1) + 8 * (li >> 2) + 4 * (w & 1) + (li & 3);
  const int KV = a.K * a.V;
  const int cs = a.s_transposed ? 1 : a.V, ns = a.s_transposed ? a.K : 1;
  const auto state_offset = [&](int J, int e, int r) {
    const int c = 32 * (MJ * part + J) + 8 * g + 4 * e + r;
    return c < a.K && sn < a.V ? (c * cs + sn * ns) * 4 : wkv6::kOffNone;
  };
  // Workspace, per segment: first its own state, which the carry kernel turns
  // into the entering one; the last place holds s_in, for s_out may be s_in.
  const auto place = [&](int s) {
    return reinterpret_cast<f32x4*>(p.ws + segment_state<KP>(p, sweep, pair, s)) + ((vb * 4 + w) * NJ + MJ * part) * 2 * 64 + lane;
  };
  const auto read_in = [&](f32x4 (&m)[MJ][2]) {
    // (unconditional buffer loads: a branch around each would wait for each)
    const float* s_from = a.s_in ? a.s_in + pair * KV : nullptr;
    const Rsrc rs = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(s_from), (short)0, s_from ? KV * 4 : 0, wkv6::kRsrcFlags);
#pragma unroll
    for (int J = 0; J < MJ; ++J)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          m[J][e][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, state_offset(J, e, r), 0, 0));
  };
  const auto write = [&](f32x4* to, const f32x4 (&m)[MJ][2]) {
#pragma unroll
    for (int i = 0; i < 2 * MJ; ++i) to[64 * i] = m[i / 2][i % 2];
  };
  f32x4 Sin[SUMMARY ? MJ : 1][2];
  if constexpr (SUMMARY) {
    if (seg == 0) read_in(Sin);
#pragma unroll
    for (int J = 0; J < MJ; ++J) M[J][0] = M[J][1] = f32x4{0.f, 0.f, 0.f, 0.f};
  } else if (!p.ws) {
    read_in(M);
  } else {
    const bool join = p.segments <= kJoin;
    const f32x4* from = place(join ? p.segments - 1 : seg);
#pragma unroll
    for (int i = 0; i < 2 * MJ; ++i) M[i / 2][i % 2] = from[64 * i];
    if (join && seg > 0) {
      const Decay<true> decay(ld, (float)p.seg_tokens);   // (what enters a segment behind the last token is not used)
      for (int s = 0; s < seg; ++s) {
        from = place(s);
#pragma unroll
        for (int i = 0; i < 2 * MJ; ++i) M[i / 2][i % 2] = decay(M[i / 2][i % 2]) + from[64 * i];
      }
    }
  }

  // ---- factors of whole chunks
  const float f_inter = ex2(gl * (16 * tb + li + (rev ? 0 : 1))) * a.is;   // column t = 16tb + li
  float dg[4], of[4];   // tile of the wave's own tokens; the tile before it
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int d = li - 4 * g - r;
    dg[r] = decayed(gl, d) * a.ps;
    of[r] = ex2(gl * (16 + d)) * a.ps;
  }
  const float a16 = ex2(gl * 16.f);
  // Scores of later keys are cleared, not multiplied by 0: a key that is not
  // finite must not reach the tokens before it (gradients of 64 heads 104.0 ->
  // 104.6 us, with a branch or a select 104.2 to 109).
  uint32_t live[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) live[r] = li < 4 * g + r ? 0u : ~0u;
  float uf[2][8];   // tokens 32u + 8g + j in the state's update
  const auto update_factors = [&](int nt) {
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int d = nt - 1 + (rev ? 1 : 0) - (32 * u + 8 * g + j);
        uf[u][j] = decayed(gl, d) * a.us;
      }
  };
  update_factors(kChunk);

  // ---- loads of a chunk of nt tokens (none: everything out of range)
  Raw8<BF> kr[KR], vr[VR], qr[SUMMARY ? 1 : NJ];
  Rows rk, rv, rq, ro;
  int ok[KR], ov[VR], oq[NJ] = {}, oo[OU] = {};
  constexpr int OSZ = OBF ? 2 : 4;
  rk.start(a.k, b, h, lo, len, rev, ISZ);
  rv.start(a.v, b, h, lo, len, rev, ISZ);
#pragma unroll
  for (int x = 0; x < KR; ++x) ok[x] = rk.offset((tid + x * NT) / (KP / 8), (tid + x * NT) % (KP / 8) * 8, a.K, ISZ);
#pragma unroll
  for (int x = 0; x < VR; ++x) ov[x] = rv.offset((tid + x * NT) / 8, v0 + tid % 8 * 8, a.V, ISZ);
  if constexpr (!SUMMARY) {
    rq.start(a.q, b, h, lo, len, rev, ISZ);
    ro.start(a.o, b, h, lo, len, rev, OSZ);
#pragma unroll
    for (int J = 0; J < NJ; ++J) oq[J] = rq.offset(16 * tb + li, 32 * J + 8 * g, a.K, ISZ);
#pragma unroll
    for (int u = 0; u < OU; ++u) oo[u] = ro.offset(16 * tb + li, v0 + 32 * (OU * part + u) + 8 * g, a.V, OSZ);
  }
  const auto load = [&](int nt) {
    const Rsrc bk = rk.rsrc(), bv = rv.rsrc();
#pragma unroll
    for (int x = 0; x < KR; ++x) kr[x] = load8<BF>(bk, (tid + x * NT) / (KP / 8) < nt ? ok[x] : wkv6::kOffNone);
#pragma unroll
    for (int x = 0; x < VR; ++x) vr[x] = load8<BF>(bv, (tid + x * NT) / 8 < nt ? ov[x] : wkv6::kOffNone);
    rk.at += rk.step;
    rv.at += rv.step;
    if constexpr (!SUMMARY) {
      const Rsrc bq = rq.rsrc();
#pragma unroll
      for (int J = 0; J < NJ; ++J)
        qr[J] = load8<BF>(bq, 16 * tb + li < nt ? oq[J] : wkv6::kOffNone);
      rq.at += rq.step;
    }
  };
  const auto tokens = [&](int c) {
    const int64_t left = hi - lo - (int64_t)c * kChunk;
    return (int)(left < 0 ? 0 : left < kChunk ? left : kChunk);
  };
  if (nch > 0) load(tokens(0));

  const bool last_seg = hi == len;
  for (int c = 0; c < nch; ++c) {
    const int nt = tokens(c);
    // ---- keys, values and the state to LDS
#pragma unroll
    for (int x = 0; x < KR; ++x) {
      const int id = tid + x * NT, row = id / (KP / 8), c8 = id % (KP / 8);
      stage8<BF>(Kp + (c8 >> 3) * kPlane, KPL, swz(row, (c8 & 7) * 8), kr[x]);
    }
#pragma unroll
    for (int x = 0; x < VR; ++x) {
      const int id = tid + x * NT;
      stage8<BF>(Vp, kPlane, swz(id / 8, id % 8 * 8), vr[x]);
    }
    Op<NI> qf[NJ];
    if constexpr (!SUMMARY) {
#pragma unroll
      for (int J = 0; J < NJ; ++J) qf[J] = operand<BF>(qr[J]);
#pragma unroll
      for (int J = 0; J < MJ; ++J) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = M[J][e >> 2][e & 3];
        const Op<MP> o = wkv6::split8<MP>(f);
#pragma unroll
        for (int s = 0; s < MP; ++s)
          *reinterpret_cast<bf16x8*>(Sp + ((s * 4 + w) * NJ + MJ * part + J) * 512 + lane * 8) = o.p[s];
      }
    }
    lds_barrier();
    load(tokens(c + 1));
    __builtin_amdgcn_sched_barrier(0);   // the loads go out now

    if constexpr (!SUMMARY) {
      {
        // ---- the state's part: O^T[n][t] = sum_c M[c][n] q_t[c]
        f32x4 acc[2 * OU];
#pragma unroll
        for (int s = 0; s < 2 * OU; ++s) {
          acc[s] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int J = 0; J < NJ; ++J)
            acc[s] = mma<MP, NI>(read8<MP>(Sp, 4 * NJ * 512, ((2 * OU * part + s) * NJ + J) * 512 + lane * 8), qf[J], acc[s]);
          acc[s] *= f_inter;
        }
        // ---- the chunk's own part, two tiles of 16 tokens i at a time
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          if (2 * u <= tb) {
            float pr[8];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int I = 2 * u + e;
              f32x4 sc = {0.f, 0.f, 0.f, 0.f};
              if (I <= tb) {
#pragma unroll
                for (int J = 0; J < NJ; ++J)
                  sc = mma<NI, NI>(read8<NI>(Kp + (J >> 1) * kPlane, KPL, swz(16 * I + li, 32 * (J & 1) + 8 * g)), qf[J], sc);
                const float far = I + 2 == tb ? a16 : I + 3 == tb ? a16 * a16 : 1.f;
#pragma unroll
                for (int r = 0; r < 4; ++r) sc[r] *= I == tb ? dg[r] : of[r] * far;
                if (I == tb) {
#pragma unroll
                  for (int r = 0; r < 4; ++r) sc[r] = __uint_as_float(__float_as_uint(sc[r]) & live[r]);
                }
              }
#pragma unroll
              for (int r = 0; r < 4; ++r) pr[4 * e + r] = sc[r];
            }
            const Op<MP> pf = wkv6::split8<MP>(pr);
#pragma unroll
            for (int s = 0; s < 2 * OU; ++s) {
              const int row = 32 * u + 4 * g + (li >> 2), col = 4 * (OU * part + (s >> 1)) + (li & 3);
              const Op<NI> vf = read_tr<NI>(Vp, kPlane, row * 64 + ((col ^ (row & 7)) << 3) + 4 * (s & 1),
                                            (row + 16) * 64 + ((col ^ (row & 7)) << 3) + 4 * (s & 1));
              acc[s] = mma<NI, MP>(vf, pf, acc[s]);
            }
          }
        }
        // ---- store: row t, channels v0 + 32u + 8g..+7
        const Rsrc bo = ro.rsrc();
        ro.at += ro.step;
#pragma unroll
        for (int u = 0; u < OU; ++u) {
          const int off = 16 * tb + li < nt ? oo[u] : wkv6::kOffNone;
          const f32x4 x = acc[2 * u], y = acc[2 * u + 1];
          if constexpr (OBF) {
            typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
            const u32x4 q = {__builtin_bit_cast(unsigned int, wkv6::round_pair(x[0], x[1])),
                             __builtin_bit_cast(unsigned int, wkv6::round_pair(x[2], x[3])),
                             __builtin_bit_cast(unsigned int, wkv6::round_pair(y[0], y[1])),
                             __builtin_bit_cast(unsigned int, wkv6::round_pair(y[2], y[3]))};
            __builtin_amdgcn_raw_buffer_store_b128(q, bo, off, 0, 0);
          } else {
            wkv6::bstoref4(bo, off, x[0], x[1], x[2], x[3]);
            wkv6::bstoref4(bo, off + 16, y[0], y[1], y[2], y[3]);
          }
        }
      }
    }

    // ---- the state's update
    if (SUMMARY || c + 1 < nch || (a.s_out && last_seg)) {
      if (nt < kChunk) update_factors(nt);
      const Decay<false>& decay = nt < kChunk ? last : whole;
#pragma unroll
      for (int J = 0; J < MJ; ++J)
#pragma unroll
        for (int e = 0; e < 2; ++e) M[J][e] = decay(M[J][e]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (32 * u < nt) {
          const int row = 32 * u + 8 * g + (li >> 2);   // and + 4
          const auto at_col = [&](int col, int half, int add) {
            return (row + add) * 64 + ((col ^ ((row + add) & 7)) << 3) + 4 * half;
          };
          const int vc = 4 * (w >> 1) + (li & 3);
          const Op<NI> vo = read_tr<NI>(Vp, kPlane, at_col(vc, w & 1, 0), at_col(vc, w & 1, 4));
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[j] = (float)vo.p[0][j];
            if constexpr (NI == 3) f[j] += (float)vo.p[1][j] + (float)vo.p[2][j];
            f[j] *= uf[u][j];
          }
          const Op<3> vf = wkv6::split8<3>(f);
#pragma unroll
          for (int J = 0; J < MJ; ++J)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int kj = MJ * part + J, kc = 4 * (kj & 1) + (li & 3);
              M[J][e] = mma<NI, 3>(read_tr<NI>(Kp + (kj >> 1) * kPlane, KPL, at_col(kc, e, 0), at_col(kc, e, 4)), vf, M[J][e]);
            }
        }
      }
    }
    lds_barrier();
  }

  // ---- hand on the state
  if constexpr (SUMMARY) {
    write(place(seg), M);
    if (seg == 0) write(place(p.segments - 1), Sin);
  } else if (a.s_out && ((last_seg && lo < hi) || (len == 0 && seg == 0))) {
    const Rsrc rt = __builtin_amdgcn_make_buffer_rsrc(a.s_out + pair * KV, (short)0, KV * 4, wkv6::kRsrcFlags);
#pragma unroll
    for (int J = 0; J < MJ; ++J)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(M[J][e][r]), rt, state_offset(J, e, r), 0, 0);
  }

  // ---- rows behind the sequence: zero, each segment those of its own places
  if constexpr (!SUMMARY) {
    const int64_t z0 = len > lo ? len : lo, z1 = lo + p.seg_tokens < a.T ? lo + p.seg_tokens : a.T;
    for (int64_t t = z0 + tid / 8; t < z1; t += NT / 8) {
      const int n = v0 + tid % 8 * 8;
      if (n < a.V) {
        char* q = static_cast<char*>(const_cast<void*>(a.o.p)) + (b * a.o.b + h * a.o.h + t * a.o.t + n) * OSZ;
#pragma unroll
        for (int x = 0; x < OSZ / 2; ++x) reinterpret_cast<uint4*>(q)[x] = make_uint4(0, 0, 0, 0);
      }
    }
  }
}

// The segments' own states, as the summaries left them, become the states
// that enter the segments: M_0 = s_in, M_{s+1} = a^(a segment's tokens) M_s + U_s
// (what enters a segment behind the last token is not used).
// Bound by the latency of the chain's loads: 8 us for 16 heads x 16 segments
// of 128 x 128 (34 MB).
constexpr int kAhead = 8;
constexpr int kCarryThreads = 128;
template <int KP>
__global__ __launch_bounds__(kCarryThreads) void carry_kernel(SweepPlan p) {
  const Sweep& a = p.a[blockIdx.z];
  const int64_t pair = blockIdx.x, next = KP * kVBlock * p.vblocks / 4;
  const Decay<true> decay(a.log_decay[pair % a.H], (float)p.seg_tokens);
  f32x4* at = reinterpret_cast<f32x4*>(p.ws + segment_state<KP>(p, blockIdx.z, pair, 0)) + blockIdx.y * kCarryThreads + threadIdx.x;
  f32x4 m = at[(p.segments - 1) * next];
  for (int s0 = 0; s0 < p.segments; s0 += kAhead) {
    f32x4 u[kAhead];   // loaded together: the chain through m must not wait for memory
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s0 + i + 1 < p.segments) u[i] = at[(s0 + i) * next];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int s = s0 + i;
      if (s >= p.segments) break;
      at[s * next] = m;
      if (s + 1 < p.segments) m = decay(m) + u[i];
    }
  }
}

template <int KP, bool BF, int MP, bool OBF>
hipError_t launch(const SweepPlan& of, hipStream_t s) {
  SweepPlan p = of;
  p.blocks = 0;
  for (int i = 0; i < p.sweeps; ++i) p.blocks += vblocks_of(p.a[i]);
  const auto grid = [&](int64_t items) { return dim3((unsigned)sweep_groups(p, items)); };
  if (p.segments > 1) {
    SweepPlan q = p;
    q.items = p.pairs * (p.segments - 1);
    const unsigned parts = (unsigned)(KP * kVBlock * p.vblocks / (4 * kCarryThreads));
    hipLaunchKernelGGL((sweep_kernel<KP, BF, MP, OBF, true>), grid(q.items), dim3(sweep_threads(KP, BF)), 0, s, q);
    if (p.segments > kJoin) hipLaunchKernelGGL(carry_kernel<KP>, dim3((unsigned)p.pairs, parts, p.sweeps), dim3(kCarryThreads), 0, s, p);
  }
  hipLaunchKernelGGL((sweep_kernel<KP, BF, MP, OBF, false>), grid(p.items), dim3(sweep_threads(KP, BF)), 0, s, p);
  return hipGetLastError();
}

template <int KP>
hipError_t launch_types(const SweepPlan& p, hipStream_t s) {
  if (!p.a[0].bf16) return launch<KP, false, 3, false>(p, s);
  if (!p.a[0].out_bf16) return launch<KP, true, 3, false>(p, s);
  return launch<KP, true, 1, true>(p, s);
}

}  // namespace

}  // namespace linattn
