// Drives the argument checks of linattn.h under AddressSanitizer and
// UndefinedBehaviorSanitizer (host code only): sizes and strides near the
// int64 limits must neither overflow nor reach the (stub) kernel side, and
// the overlap rules must tell slices that lie side by side from ones that
// share elements.  Exits 0 when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "linattn.h"

extern int g_linattn_enqueued;

namespace {

int failures = 0;

void expect(bool ok, const char* what, int line) {
  if (!ok) {
    std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, wkv6_last_error());
    ++failures;
  }
}

void outcome(int status, int want, int before, int line) {
  expect(status == want, "status", line);
  expect((std::strlen(wkv6_last_error()) > 0) == (want != WKV6_OK), "message", line);
  expect(g_linattn_enqueued - before == (want == WKV6_OK ? 1 : 0), "calls enqueued", line);
}
#define EXPECT(call, want)                        \
  do {                                            \
    const int before = g_linattn_enqueued;        \
    outcome((call), (want), before, __LINE__);    \
  } while (0)

char* P(int i) { return reinterpret_cast<char*>(uintptr_t(0x1000000000ull) * (i + 1)); }
float* F(int i) { return reinterpret_cast<float*>(P(i)); }
char ws[4096] __attribute__((aligned(16)));

int fwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const int64_t* strides = nullptr, const char* o = P(5),
        const char* q = P(0), int dtype = 1, int out = 1) {
  return linattn_fwd(B, T, H, K, V, q, P(1), P(2), F(3), 1.f, nullptr, F(4), const_cast<char*>(o), F(6), strides, dtype,
                     out, ws, sizeof(ws), nullptr);
}

}  // namespace

int main() {
  const int64_t big = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  EXPECT(fwd(2, 9, 2, 64, 64), WKV6_OK);
  const int64_t odd[] = {0, 1, 7, 8, 64, 128, 129, big, low, -1, big - 7, int64_t(1) << 32, int64_t(1) << 62};
  for (int64_t a : odd)
    for (int64_t b : odd)
      for (int64_t c : odd) {
        // every combination returns a status without undefined behaviour
        const int before = g_linattn_enqueued;
        const int st[] = {fwd(a, b, c, 64, 64), fwd(1, b, 1, a, c), linattn_rope(a, b, c, 64, 64, P(0), P(1), P(2), P(3), nullptr, 0, reinterpret_cast<double*>(P(4)), 0, 0, nullptr, 1, nullptr),
                          linattn_rms_norm(a, b, P(0), nullptr, F(1), 0.f, nullptr, P(2), (int)(c & 1), nullptr)};
        for (int s : st) expect(s >= 0 && s <= 3, "a documented status", __LINE__);
        expect(g_linattn_enqueued >= before, "count", __LINE__);
        int64_t d[12] = {a, b, c, 9 * 128, 128, 64, 9 * 128, 128, 64, 9 * 128, 128, 64};
        const int s1 = fwd(2, 9, 2, 64, 64, d);
        int64_t e[12] = {9 * 128, 128, 64, 9 * 128, 128, 64, 9 * 128, 128, 64, a, b, c};
        const int s2 = fwd(2, 9, 2, 64, 64, e);
        expect(s1 >= 0 && s1 <= 3 && s2 >= 0 && s2 <= 3, "a documented status", __LINE__);
        (void)linattn_fwd_workspace_bytes(a, b, c, 64, 64, 1, 1, 1);
        (void)linattn_bwd_workspace_bytes(a, b, c, 64, 64, 1, 1, 1);
        (void)linattn_rms_norm_bwd_workspace_bytes(a, b, 0);
      }
  // slices of one buffer [B, T, 4, H, 64]: o beside q, and o one head into q
  {
    const int64_t t = 4 * 128, b = 9 * t;
    int64_t d[12] = {b, t, 64, b, t, 64, b, t, 64, b, t, 64};
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0) + 128 * 2, P(0)), WKV6_OK);
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0) + 3 * 128 * 2, P(0)), WKV6_OK);
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0) + 64 * 2, P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0), P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0) + (3 * 128 + 64) * 2, P(0)), WKV6_ERR_INVALID_ARG);   // reaches the next token's q
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0), P(0) + 128 * 2), WKV6_OK);
    d[9] = b + 8;   // other distances
    EXPECT(fwd(2, 9, 2, 64, 64, d, P(0) + 128 * 2, P(0)), WKV6_ERR_INVALID_ARG);
    int64_t e[12] = {b, t, 64, b, t, 64, b, t, 64, b, 2 * t, 64};
    EXPECT(fwd(1, 9, 2, 64, 64, e, P(0) + 128 * 2, P(0)), WKV6_ERR_INVALID_ARG);
  }
  // the same for single tokens, and for slices [B, 2, H, T, 64] with heads before tokens
  {
    const int64_t b = 4 * 128;
    int64_t d[12] = {b, 8, 64, b, 8, 64, b, 8, 64, b, 8, 64};
    EXPECT(fwd(20, 1, 2, 64, 64, d, P(0) + 128 * 2, P(0)), WKV6_OK);
    EXPECT(fwd(20, 1, 2, 64, 64, d, P(0) + 64 * 2, P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(20, 1, 2, 64, 64, d, P(0) + (3 * b + 128) * 2, P(0)), WKV6_OK);
    EXPECT(fwd(20, 1, 2, 64, 64, d, P(0) + 3 * b * 2, P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(20, 1, 2, 64, 64, d, P(0) + (20 * b) * 2, P(0)), WKV6_OK);
    const int64_t t = 64, h = 9 * 64, c = 2 * 2 * h;
    int64_t e[12] = {c, t, h, c, t, h, c, t, h, c, t, h};
    EXPECT(fwd(3, 9, 2, 64, 64, e, P(0) + 2 * h * 2, P(0)), WKV6_OK);
    EXPECT(fwd(3, 9, 2, 64, 64, e, P(0) + h * 2, P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(3, 9, 2, 64, 64, e, P(0) + (2 * h + 64) * 2, P(0)), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(3, 9, 2, 64, 64, e, P(0), P(0) + 2 * h * 2), WKV6_OK);
  }
  // the output's rows in one place
  {
    int64_t d[12] = {9 * 128, 128, 64, 9 * 128, 128, 64, 9 * 128, 128, 64, 0, 128, 64};
    EXPECT(fwd(2, 9, 2, 64, 64, d), WKV6_ERR_INVALID_ARG);
    EXPECT(fwd(1, 9, 2, 64, 64, d), WKV6_OK);   // one batch item: its distance does not matter
  }
  // workspace of the caller
  EXPECT(linattn_fwd(1, 2000, 1, 64, 64, P(0), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(5), nullptr, nullptr, 1, 1, ws, 64, nullptr), WKV6_ERR_INVALID_ARG);
  EXPECT(linattn_rms_norm_bwd(4, 64, P(0), P(1), nullptr, F(2), 0.f, P(3), F(4), 1, ws, sizeof(ws), nullptr), WKV6_OK);
  EXPECT(linattn_rms_norm_bwd(4, 64, P(0), P(1), nullptr, F(2), 0.f, P(3), F(4), 1, ws + 8, sizeof(ws) - 8, nullptr), WKV6_ERR_MISALIGNED);
  if (failures) return 1;
  std::puts("all argument checks hold");
  return 0;
}
