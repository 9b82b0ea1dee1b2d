// C ABI of the linear-attention operators: argument checks, workspace,
// launch.  The declarations and their contract live in include/linattn.h.
#include "linattn.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <string>

#include "linattn_internal.h"
#include "linattn_plan.h"
#include "wkv6_host.h"

namespace {

using linattn::Tensor;
using wkv6::set_error;

int invalid(const std::string& m) { return set_error(WKV6_ERR_INVALID_ARG, m); }
int unsupported(const std::string& m) { return set_error(WKV6_ERR_UNSUPPORTED, m); }

// Bytes that a call touches through one pointer: rows of `row` bytes, `sb`,
// `st` and `sh` bytes apart between batch items, tokens and heads.
struct Span {
  const char* name;
  uintptr_t at;
  int64_t nb, nt, nh, sb, st, sh, row;
  bool out;
  int64_t bytes() const { return (nb - 1) * sb + (nt - 1) * st + (nh - 1) * sh + row; }
};

Span flat(const char* name, const void* p, int64_t bytes, bool out) {
  return {name, reinterpret_cast<uintptr_t>(p), 1, 1, 1, 0, 0, 0, bytes, out};
}

bool same_place(const Span& a, const Span& b) {
  return a.at == b.at && a.nb == b.nb && a.nt == b.nt && a.nh == b.nh && a.sb == b.sb && a.st == b.st && a.sh == b.sh &&
         a.row == b.row;
}

// Dimensions of more than one place, from the largest distance on.
struct Dims {
  int n = 0;
  int64_t step[3], count[3];
  explicit Dims(const Span& a) {
    const int64_t c[3] = {a.nb, a.nt, a.nh}, s[3] = {a.sb, a.st, a.sh};
    for (int i = 0; i < 3; ++i) {
      if (c[i] <= 1) continue;
      int at = n++;
      for (; at > 0 && step[at - 1] < s[i]; --at) step[at] = step[at - 1], count[at] = count[at - 1];
      step[at] = s[i];
      count[at] = c[i];
    }
  }
  // bytes from the first to the end of the last row within dimension i
  int64_t width(int i, int64_t row) const {
    for (; i < n; ++i) row += (count[i] - 1) * step[i];
    return row;
  }
};

// Whether rows of a (of `ra` bytes) and of b (of `rb`, starting `d` bytes
// later) share bytes, from dimension i on: place by place as long as their
// distances are the same, then by all that the remaining dimensions reach over.
bool share_rows(const Dims& a, const Dims& b, int i, int64_t ra, int64_t rb, int64_t d) {
  if (i == a.n || i == b.n || a.step[i] != b.step[i]) return d < a.width(i, ra) && -d < b.width(i, rb);
  const int64_t s = a.step[i], wa = a.width(i + 1, ra), wb = b.width(i + 1, rb);
  if (s == 0 || wa > s || wb > s) return true;   // not told apart
  // b's place is m steps after a's: only a few m can meet
  const int64_t m0 = -(d / s) - 2;
  for (int64_t m = m0; m <= m0 + 4; ++m) {
    if (m <= -a.count[i] || m >= b.count[i]) continue;
    const int64_t e = d + m * s;
    if (e < wa && -e < wb && share_rows(a, b, i + 1, ra, rb, e)) return true;
  }
  return false;
}

// Whether two spans share bytes.  Disjoint ranges do not; slices of one buffer,
// side by side, are told apart exactly, also where heads of different sizes lie
// side by side within a token; everything else counts as sharing.
bool share(const Span& a, const Span& b) {
  if (a.at + (uint64_t)a.bytes() <= b.at || b.at + (uint64_t)b.bytes() <= a.at) return false;
  const Dims da(a), db(b);
  return share_rows(da, db, 0, a.row, b.row, (int64_t)(b.at - a.at));
}

// Whether an output's rows are all different places: its distances, from the
// smallest on, each reach past what lies within.
bool distinct(const Span& a) {
  const Dims d(a);
  for (int i = 0; i < d.n; ++i)
    if (d.step[i] < d.width(i + 1, a.row)) return false;
  return true;
}

// allowed: pairs of indexes (output, input) that may be the same place
int check_overlaps(const Span* s, int n, const int (*allowed)[2], int na) {
  for (int i = 0; i < n; ++i) {
    if (!s[i].out || !s[i].at) continue;
    if (!distinct(s[i])) return invalid(std::string(s[i].name) + ": its rows share elements");
    for (int j = 0; j < n; ++j) {
      if (j == i || !s[j].at || (s[j].out && j > i) || !share(s[i], s[j])) continue;
      bool ok = false;
      for (int k = 0; k < na; ++k) ok = ok || (allowed[k][0] == i && allowed[k][1] == j && same_place(s[i], s[j]));
      if (!ok) return invalid(std::string(s[i].name) + " overlaps " + s[j].name);
    }
  }
  return WKV6_OK;
}

// What a C entry returns where the host's memory gives out (an error text, the
// list of pools): no exception leaves it.
int no_memory() { return WKV6_ERR_HIP; }

// (tables that are read value by value may start at any of them: `align`)
int present(const char* name, const void* p, int align = 16) {
  if (!p) return invalid(std::string("null pointer: ") + name);
  if (reinterpret_cast<uintptr_t>(p) % align)
    return set_error(WKV6_ERR_MISALIGNED, "pointer not " + std::to_string(align) + "-byte aligned: " + name);
  return WKV6_OK;
}

int optional(const char* name, const void* p, int align = 16) { return p ? present(name, p, align) : WKV6_OK; }

int known_dtype(int dtype) {
  return dtype == WKV6_DTYPE_F32 || dtype == WKV6_DTYPE_BF16 ? WKV6_OK : invalid("unknown dtype");
}

int size_of(int dtype) { return dtype == WKV6_DTYPE_BF16 ? 2 : 4; }

// One tensor of a [B, T, H, D] call: its distances (3 values, or null:
// contiguous), checked, and its span.  `chunked`: rows are read a chunk at a time.
int tensor(const char* name, const void* p, const int64_t* d, int64_t B, int64_t T, int64_t H, int64_t D, int dtype,
           bool out, bool chunked, Tensor* t, Span* s) {
  int st = present(name, p);
  if (st != WKV6_OK) return st;
  const int z = size_of(dtype);
  *t = {p, T * H * D, H * D, D};
  if (d) *t = {p, d[0], d[1], d[2]};
  int64_t* const dist[3] = {&t->b, &t->t, &t->h};
  const int64_t most[3] = {B, T, H};
  for (int i = 0; i < 3; ++i) {
    if (most[i] <= 1) *dist[i] = 0;   // a dimension of one place: its distance does not matter
    if (*dist[i] < 0) return invalid(std::string(name) + ": negative stride");
    // sums of the three parts stay under 2^63: each is at most 2^60
    if (*dist[i] && most[i] - 1 > (int64_t(1) << 60) / z / *dist[i])
      return unsupported(std::string(name) + ": sizes exceed the supported index range");
    if (*dist[i] * z % 16)
      return set_error(WKV6_ERR_MISALIGNED, std::string(name) + ": a stride is not a multiple of 16 bytes");
  }
  // a chunk's rows are addressed with 32-bit byte offsets
  if (chunked && T > 1 && t->t > (INT_MAX - 8192) / linattn::kChunk / z)
    return unsupported(std::string(name) + ": token stride exceeds the supported index range");
  *s = {name, reinterpret_cast<uintptr_t>(p), B, T, H, t->b * z, t->t * z, t->h * z, D * z, out};
  return WKV6_OK;
}

// Sizes of the attention calls.
int check_sizes(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int out_dtype) {
  if (B < 0 || T < 0 || H < 1) return invalid("sizes must be B, T >= 0 and H >= 1");
  int st = known_dtype(dtype);
  if (st == WKV6_OK) st = known_dtype(out_dtype);
  if (st != WKV6_OK) return st;
  if (dtype == WKV6_DTYPE_F32 && out_dtype != WKV6_DTYPE_F32)
    return unsupported("float32 inputs give float32 outputs");
  if (K < 8 || V < 8 || K > LINATTN_MAX_HEAD || V > LINATTN_MAX_HEAD || K % 8 || V % 8)
    return unsupported("K and V must be multiples of 8 from 8 to 128");
  if (B == 0) return WKV6_OK;
  if (H > (1 << 21) || B > (1 << 21) / H)
    return unsupported("B * H exceeds the supported number of (batch, head) pairs (2^21)");
  if (T > INT_MAX - linattn::kChunk) return unsupported("T exceeds the supported range");
  return WKV6_OK;
}

// A launch holds fewer than 2^32 work-items.
int check_launches(const linattn::Sweep* a, int n) {
  if (linattn::largest_launch(a, n) >= (int64_t(1) << 32))
    return unsupported("B * H exceeds the (batch, head) pairs of these head sizes that a launch holds");
  return WKV6_OK;
}

linattn::Sweep base_sweep(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const float* log_decay,
                          const int32_t* lengths, int dtype, int out_dtype) {
  linattn::Sweep a = {};
  a.B = B;
  a.T = T;
  a.H = H;
  a.K = (int)K;
  a.V = (int)V;
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.us = a.is = a.ps = 1.f;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  a.out_bf16 = out_dtype == WKV6_DTYPE_BF16;
  return a;
}

// The workspace of a call: the caller's, or the pool's for as long as this
// object lives (given back in stream order).
struct Workspace {
  void* p = nullptr;
  bool owned = false;
  hipStream_t stream;
  explicit Workspace(hipStream_t s) : stream(s) {}
  int take(void* given, size_t have, size_t need) {
    if (!need) return WKV6_OK;
    if (given) {
      if (reinterpret_cast<uintptr_t>(given) % 16)
        return set_error(WKV6_ERR_MISALIGNED, "pointer not 16-byte aligned: workspace");
      if (have < need) return invalid("the workspace is too small");
      p = given;
      return WKV6_OK;
    }
    const hipError_t e = wkv6::workspace_alloc(&p, need, stream);
    if (e != hipSuccess) return set_error(WKV6_ERR_HIP, std::string("workspace allocation: ") + hipGetErrorString(e));
    owned = true;
    return WKV6_OK;
  }
  int done(hipError_t e) {
    const hipError_t ef = owned ? hipFreeAsync(p, stream) : hipSuccess;
    owned = false;
    if (e != hipSuccess) return set_error(WKV6_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
    if (ef != hipSuccess) return set_error(WKV6_ERR_HIP, std::string("workspace release: ") + hipGetErrorString(ef));
    return WKV6_OK;
  }
};

int finished(hipError_t e) {
  return e == hipSuccess ? WKV6_OK : set_error(WKV6_ERR_HIP, std::string("kernel launch: ") + hipGetErrorString(e));
}

// The gradients' three sweeps.  dq is the forward operator on (d_o, v, k)
// with the state transposed, dk and dv are reversed ones on (v, d_o, q) and
// (k, q, d_o) whose state is the adjoint of the forward state.
void bwd_sweeps(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const float* log_decay, float scale,
                const int32_t* lengths, const float* s_in, const float* ds_out, float* ds_in, const Tensor* t, int dtype,
                int grad_dtype, linattn::Sweep (&out)[3]) {
  enum { Q, KK, VV, DO, DQ, DK, DV };
  linattn::Sweep a = base_sweep(B, T, H, V, K, log_decay, lengths, dtype, grad_dtype);
  a.q = t[DO];
  a.k = t[VV];
  a.v = t[KK];
  a.o = t[DQ];
  a.is = a.ps = scale;
  a.s_in = s_in;
  a.s_transposed = true;
  out[0] = a;
  a.q = t[VV];
  a.k = t[DO];
  a.v = t[Q];
  a.o = t[DK];
  a.is = 1.f;
  a.us = a.ps = scale;
  a.s_in = ds_out;
  a.reverse = true;
  out[1] = a;
  linattn::Sweep d = base_sweep(B, T, H, K, V, log_decay, lengths, dtype, grad_dtype);
  d.q = t[KK];
  d.k = t[Q];
  d.v = t[DO];
  d.o = t[DV];
  d.us = d.ps = scale;
  d.s_in = ds_out;
  d.s_out = ds_in;
  d.reverse = true;
  out[2] = d;
}

int norm_sizes(int64_t rows, int64_t C, float eps, int dtype) {
  if (rows < 0 || C < 1) return invalid("sizes must be rows >= 0 and C >= 1");
  const int st = known_dtype(dtype);
  if (st != WKV6_OK) return st;
  if (!(std::isfinite(eps) && eps >= 0.f)) return invalid("eps must be finite and >= 0");
  if (C % 8 || C > LINATTN_MAX_COLUMNS) return unsupported("C must be a multiple of 8 up to 16384");
  // a launch holds fewer than 2^32 work-items: 64 for each of many rows of up
  // to 1024 columns, else up to 1024
  if (rows > (C <= 1024 ? 1 << 25 : 1 << 21))
    return unsupported("rows exceed the supported number (2^25, or 2^21 of more than 1024 columns)");
  return WKV6_OK;
}

}  // namespace

extern "C" {

int linattn_abi_version(void) { return LINATTN_ABI_VERSION; }

size_t linattn_fwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int out_dtype,
                                   int state_out) try {
  set_error(WKV6_OK, "");
  if (check_sizes(B, T, H, K, V, dtype, out_dtype) != WKV6_OK || B == 0 || T == 0) return 0;
  const int32_t some = 0;   // (calls with lengths take as much as others or more)
  linattn::Sweep a = base_sweep(B, T, H, K, V, nullptr, &some, dtype, out_dtype);
  float any = 0.f;
  a.s_out = state_out ? &any : nullptr;
  if (check_launches(&a, 1) != WKV6_OK) return 0;
  return linattn::sweep_workspace_bytes(&a, 1);
} catch (...) {
  return 0;
}

int linattn_fwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const void* q, const void* k, const void* v,
                const float* log_decay, float scale, const int32_t* lengths, const float* s_in, void* o, float* s_out,
                const int64_t* strides, int dtype, int out_dtype, void* workspace, size_t workspace_bytes,
                void* stream) try {
  set_error(WKV6_OK, "");
  int st = check_sizes(B, T, H, K, V, dtype, out_dtype);
  if (st != WKV6_OK || B == 0) return st;
  linattn::Sweep a = base_sweep(B, T, H, K, V, log_decay, lengths, dtype, out_dtype);
  if (T > 0 && (st = check_launches(&a, 1)) != WKV6_OK) return st;
  const int64_t sbytes = B * H * K * V * 4;
  Span s[9];
  int n = 0;
  if ((st = optional("s_in", s_in)) != WKV6_OK || (st = optional("s_out", s_out)) != WKV6_OK) return st;
  s[n++] = flat("s_in", s_in, sbytes, false);
  s[n++] = flat("s_out", s_out, sbytes, true);
  if (T > 0) {
    const bool chunked = !linattn::steps(&a, 1);
    if ((st = tensor("q", q, strides, B, T, H, K, dtype, false, chunked, &a.q, &s[n++])) != WKV6_OK ||
        (st = tensor("k", k, strides ? strides + 3 : nullptr, B, T, H, K, dtype, false, chunked, &a.k, &s[n++])) != WKV6_OK ||
        (st = tensor("v", v, strides ? strides + 6 : nullptr, B, T, H, V, dtype, false, chunked, &a.v, &s[n++])) != WKV6_OK ||
        (st = tensor("o", o, strides ? strides + 9 : nullptr, B, T, H, V, out_dtype, true, chunked, &a.o, &s[n++])) != WKV6_OK ||
        (st = present("log_decay", log_decay, 4)) != WKV6_OK || (st = optional("lengths", lengths)) != WKV6_OK)
      return st;
    s[n++] = flat("log_decay", log_decay, H * 4, false);
    s[n++] = flat("lengths", lengths, B * 4, false);
  } else if (!s_out) {
    return WKV6_OK;
  }
  const int allowed[1][2] = {{1, 0}};
  if ((st = check_overlaps(s, n, allowed, 1)) != WKV6_OK) return st;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (T == 0) return finished(linattn::enqueue_state_copy(s_in, s_out, B * H * K * V, hs));
  a.is = a.ps = scale;
  a.s_in = s_in;
  a.s_out = s_out;
  Workspace ws(hs);
  if ((st = ws.take(workspace, workspace_bytes, linattn::sweep_workspace_bytes(&a, 1))) != WKV6_OK) return st;
  return ws.done(linattn::enqueue_sweeps(&a, 1, ws.p, hs));
} catch (...) {
  return no_memory();
}

size_t linattn_bwd_workspace_bytes(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int grad_dtype,
                                   int state_grad) try {
  set_error(WKV6_OK, "");
  if (check_sizes(B, T, H, K, V, dtype, grad_dtype) != WKV6_OK || B == 0 || T == 0) return 0;
  const Tensor none[7] = {};
  linattn::Sweep w[3];
  float any = 0.f;
  const int32_t some = 0;
  bwd_sweeps(B, T, H, K, V, nullptr, 1.f, &some, nullptr, nullptr, state_grad ? &any : nullptr, none, dtype, grad_dtype, w);
  if (check_launches(w, 3) != WKV6_OK) return 0;
  return linattn::sweep_workspace_bytes(w, 3);
} catch (...) {
  return 0;
}

int linattn_bwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const void* q, const void* k, const void* v,
                const float* log_decay, float scale, const int32_t* lengths, const float* s_in, const void* d_o,
                const float* ds_out, void* dq, void* dk, void* dv, float* ds_in, const int64_t* strides, int dtype,
                int grad_dtype, void* workspace, size_t workspace_bytes, void* stream) try {
  set_error(WKV6_OK, "");
  int st = check_sizes(B, T, H, K, V, dtype, grad_dtype);
  if (st != WKV6_OK || B == 0) return st;
  Tensor t[7] = {};
  linattn::Sweep w[3];
  bwd_sweeps(B, T, H, K, V, log_decay, scale, lengths, s_in, ds_out, ds_in, t, dtype, grad_dtype, w);
  if (T > 0 && (st = check_launches(w, 3)) != WKV6_OK) return st;
  const int64_t sbytes = B * H * K * V * 4;
  Span s[12];
  int n = 0;
  if ((st = optional("s_in", s_in)) != WKV6_OK || (st = optional("ds_out", ds_out)) != WKV6_OK ||
      (st = optional("ds_in", ds_in)) != WKV6_OK)
    return st;
  s[n++] = flat("s_in", s_in, sbytes, false);
  s[n++] = flat("ds_out", ds_out, sbytes, false);
  s[n++] = flat("ds_in", ds_in, sbytes, true);
  if (T > 0) {
    const void* p[7] = {q, k, v, d_o, dq, dk, dv};
    const char* names[7] = {"q", "k", "v", "d_o", "dq", "dk", "dv"};
    const int64_t D[7] = {K, K, V, V, K, K, V};
    for (int i = 0; i < 7; ++i)
      if ((st = tensor(names[i], p[i], strides ? strides + 3 * i : nullptr, B, T, H, D[i], i < 4 ? dtype : grad_dtype,
                       i >= 4, true, &t[i], &s[n++])) != WKV6_OK)
        return st;
    if ((st = present("log_decay", log_decay, 4)) != WKV6_OK || (st = optional("lengths", lengths)) != WKV6_OK) return st;
    s[n++] = flat("log_decay", log_decay, H * 4, false);
    s[n++] = flat("lengths", lengths, B * 4, false);
  } else if (!ds_in) {
    return WKV6_OK;
  }
  const int allowed[1][2] = {{2, 1}};
  if ((st = check_overlaps(s, n, allowed, 1)) != WKV6_OK) return st;
  const hipStream_t hs = static_cast<hipStream_t>(stream);
  if (T == 0) return finished(linattn::enqueue_state_copy(ds_out, ds_in, B * H * K * V, hs));
  bwd_sweeps(B, T, H, K, V, log_decay, scale, lengths, s_in, ds_out, ds_in, t, dtype, grad_dtype, w);
  Workspace ws(hs);
  if ((st = ws.take(workspace, workspace_bytes, linattn::sweep_workspace_bytes(w, 3))) != WKV6_OK) return st;
  return ws.done(linattn::enqueue_sweeps(w, 3, ws.p, hs));
} catch (...) {
  return no_memory();
}

int linattn_rope(int64_t B, int64_t T, int64_t H, int64_t D, int64_t R, const void* q, const void* k, void* q_out,
                 void* k_out, const int32_t* positions, int64_t start, const double* freqs, int layout, int inverse,
                 const int64_t* strides, int dtype, void* stream) try {
  set_error(WKV6_OK, "");
  if (B < 0 || T < 0 || H < 1) return invalid("sizes must be B, T >= 0 and H >= 1");
  int st = known_dtype(dtype);
  if (st != WKV6_OK) return st;
  if (layout != LINATTN_ROPE_HALF && layout != LINATTN_ROPE_INTERLEAVED) return invalid("unknown layout");
  if (D < 8 || D > LINATTN_MAX_HEAD || D % 8) return unsupported("D must be a multiple of 8 from 8 to 128");
  if (R < 2 || R > D || R % 2) return unsupported("R must be even, from 2 to D");
  if (B == 0 || T == 0) return WKV6_OK;
  if (H > (1 << 20) || T > (1 << 27) || B > (1 << 27) / T) return unsupported("B * T (2^27) or H (2^20) exceeds the supported range");
  if (start > (int64_t(1) << 52) || start < -(int64_t(1) << 52)) return unsupported("start exceeds the supported range");
  if ((k == nullptr) != (k_out == nullptr)) return invalid("k and k_out are both given or both null");
  linattn::Rope a = {};
  Span s[6];
  int n = 0;
  const void* p[4] = {q, k, q_out, k_out};
  const char* names[4] = {"q", "k", "q_out", "k_out"};
  Tensor* to[4] = {&a.q, &a.k, &a.q_out, &a.k_out};
  for (int i = 0; i < 4; ++i) {
    if (i % 2 && !k) {
      s[n++] = flat(names[i], nullptr, 0, false);
      continue;
    }
    if ((st = tensor(names[i], p[i], strides ? strides + 3 * i : nullptr, B, T, H, D, dtype, i >= 2, false, to[i],
                     &s[n++])) != WKV6_OK)
      return st;
  }
  if ((st = present("freqs", freqs)) != WKV6_OK || (st = optional("positions", positions, 4)) != WKV6_OK) return st;
  s[n++] = flat("positions", positions, B * T * 4, false);
  s[n++] = flat("freqs", freqs, R / 2 * 8, false);
  const int allowed[2][2] = {{2, 0}, {3, 1}};
  if ((st = check_overlaps(s, n, allowed, 2)) != WKV6_OK) return st;
  a.B = B;
  a.T = T;
  a.H = H;
  a.D = (int)D;
  a.R = (int)R;
  a.positions = positions;
  a.start = start;
  a.freqs = freqs;
  a.interleaved = layout == LINATTN_ROPE_INTERLEAVED;
  a.inverse = inverse != 0;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return finished(linattn::enqueue_rope(a, static_cast<hipStream_t>(stream)));
} catch (...) {
  return no_memory();
}

}  // extern "C"

namespace {

int norm_call(int64_t rows, int64_t C, const void* x, const void* residual, const float* weight, float eps, void* h,
              void* y, uint8_t* codes, float* scales, int group, int dtype, void* stream) {
  int st = norm_sizes(rows, C, eps, dtype);
  if (st != WKV6_OK || rows == 0) return st;
  if ((residual == nullptr) != (h == nullptr)) return invalid("residual and h are both given or both null");
  const bool q8 = !y;
  const int64_t bytes = rows * C * size_of(dtype), groups = group ? (C + 127) / 128 : 1;
  if ((st = present("x", x)) != WKV6_OK || (st = optional("residual", residual)) != WKV6_OK ||
      (st = present("weight", weight)) != WKV6_OK || (st = optional("h", h)) != WKV6_OK ||
      (st = q8 ? present("codes", codes) : present("y", y)) != WKV6_OK || (q8 && (st = present("scales", scales)) != WKV6_OK))
    return st;
  const Span s[6] = {flat("x", x, bytes, false),
                     flat("residual", residual, bytes, false),
                     flat("weight", weight, C * 4, false),
                     flat("h", h, bytes, true),
                     q8 ? flat("codes", codes, rows * C, true) : flat("y", y, bytes, true),
                     flat("scales", scales, rows * groups * 4, true)};
  const int allowed[2][2] = {{3, 0}, {3, 1}};
  if ((st = check_overlaps(s, 6, allowed, 2)) != WKV6_OK) return st;
  linattn::Norm a = {};
  a.rows = rows;
  a.C = C;
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.eps = eps;
  a.h = h;
  a.y = y;
  a.codes = codes;
  a.scales = scales;
  a.group = group;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return finished(linattn::enqueue_norm(a, static_cast<hipStream_t>(stream)));
}

linattn::NormBwd norm_bwd_args(int64_t rows, int64_t C, int dtype) {
  linattn::NormBwd a = {};
  a.rows = rows;
  a.C = C;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return a;
}

}  // namespace

extern "C" {

int linattn_rms_norm(int64_t rows, int64_t C, const void* x, const void* residual, const float* weight, float eps,
                     void* h, void* y, int dtype, void* stream) try {
  set_error(WKV6_OK, "");
  if (rows > 0 && !y) return invalid("null pointer: y");
  return norm_call(rows, C, x, residual, weight, eps, h, y, nullptr, nullptr, 0, dtype, stream);
} catch (...) {
  return no_memory();
}

int linattn_rms_norm_q8(int64_t rows, int64_t C, const void* x, const void* residual, const float* weight, float eps,
                        void* h, void* codes, float* scales, int group, int dtype, void* stream) try {
  set_error(WKV6_OK, "");
  if (group != 0 && group != 128) return invalid("group must be 0 or 128");
  return norm_call(rows, C, x, residual, weight, eps, h, nullptr, static_cast<uint8_t*>(codes), scales, group, dtype,
                   stream);
} catch (...) {
  return no_memory();
}

size_t linattn_rms_norm_bwd_workspace_bytes(int64_t rows, int64_t C, int dtype) try {
  set_error(WKV6_OK, "");
  if (norm_sizes(rows, C, 0.f, dtype) != WKV6_OK) return 0;
  return linattn::norm_bwd_workspace_bytes(norm_bwd_args(rows, C, dtype));
} catch (...) {
  return 0;
}

int linattn_rms_norm_bwd(int64_t rows, int64_t C, const void* dy, const void* h, const void* dh, const float* weight,
                         float eps, void* dx, float* dweight, int dtype, void* workspace, size_t workspace_bytes,
                         void* stream) try {
  set_error(WKV6_OK, "");
  int st = norm_sizes(rows, C, eps, dtype);
  if (st != WKV6_OK) return st;
  if ((st = present("dweight", dweight)) != WKV6_OK) return st;
  linattn::NormBwd a = norm_bwd_args(rows, C, dtype);
  if (rows > 0) {
    if ((st = present("dy", dy)) != WKV6_OK || (st = present("h", h)) != WKV6_OK || (st = optional("dh", dh)) != WKV6_OK ||
        (st = present("weight", weight)) != WKV6_OK || (st = present("dx", dx)) != WKV6_OK)
      return st;
    const int64_t bytes = rows * C * size_of(dtype);
    const Span s[6] = {flat("dy", dy, bytes, false),       flat("dh", dh, bytes, false),
                       flat("h", h, bytes, false),         flat("weight", weight, C * 4, false),
                       flat("dx", dx, bytes, true),        flat("dweight", dweight, C * 4, true)};
    const int allowed[2][2] = {{4, 0}, {4, 1}};
    if ((st = check_overlaps(s, 6, allowed, 2)) != WKV6_OK) return st;
  }
  a.dy = dy;
  a.h = h;
  a.dh = dh;
  a.weight = weight;
  a.eps = eps;
  a.dx = dx;
  a.dweight = dweight;
  Workspace ws(static_cast<hipStream_t>(stream));
  if ((st = ws.take(workspace, workspace_bytes, linattn::norm_bwd_workspace_bytes(a))) != WKV6_OK) return st;
  return ws.done(linattn::enqueue_norm_bwd(a, ws.p, ws.stream));
} catch (...) {
  return no_memory();
}

}  // extern "C"
