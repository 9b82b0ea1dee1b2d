// What the C entries of linattn.h and ssm.h check before a call and how they
// take its workspace: host code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "linattn_internal.h"
#include "wkv6.h"
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
// contiguous), checked, and its span.
int place(const char* name, const void* p, const int64_t* d, int64_t B, int64_t T, int64_t H, int64_t D, int dtype,
          bool out, Tensor* t, Span* s) {
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
  *s = {name, reinterpret_cast<uintptr_t>(p), B, T, H, t->b * z, t->t * z, t->h * z, D * z, out};
  return WKV6_OK;
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

}  // namespace
