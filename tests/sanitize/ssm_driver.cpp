// Drives the argument checks of ssm.h under AddressSanitizer and
// UndefinedBehaviorSanitizer (host code only): sizes and strides near the
// int64 limits must neither overflow nor reach the (stub) kernel side.  Exits 0
// when every check holds.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>

#include "ssm.h"

extern int g_ssm_enqueued;

namespace {

int failures = 0;

void expect(bool ok, const char* what, int line) {
  if (!ok) {
    std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, wkv6_last_error());
    ++failures;
  }
}

char* P(int i) { return reinterpret_cast<char*>(uintptr_t(0x1000000000ull) * (i + 1)); }
float* F(int i) { return reinterpret_cast<float*>(P(i)); }
char ws[4096] __attribute__((aligned(16)));

int conv(int64_t B, int64_t T, int64_t D, int64_t W, const int64_t* s = nullptr) {
  return ssm_conv_fwd(B, T, D, W, P(0), F(1), F(2), 1, nullptr, P(3), P(4), P(5), s, 1, nullptr);
}
int conv_bwd(int64_t B, int64_t T, int64_t D, int64_t W, const int64_t* s = nullptr) {
  return ssm_conv_bwd(B, T, D, W, P(0), F(1), F(2), 1, nullptr, P(3), P(4), P(5), P(6), F(7), F(8), P(9), s, 1, ws,
                      sizeof(ws), nullptr);
}
int scan(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const int64_t* s = nullptr) {
  return ssm_scan_fwd(B, T, D, N, G, P(0), P(1), F(2), P(3), P(4), F(5), P(6), F(7), 1, nullptr, F(8), P(9), F(10), s, 1,
                      nullptr);
}
int scan_bwd(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const int64_t* s = nullptr) {
  return ssm_scan_bwd(B, T, D, N, G, P(0), P(1), F(2), P(3), P(4), F(5), P(6), F(7), 1, nullptr, F(8), P(9), F(10), P(11),
                      P(12), F(13), P(14), P(15), F(16), P(17), F(18), F(19), s, 1, ws, sizeof(ws), nullptr);
}
int norm(int64_t rows, int64_t C, int64_t per) {
  return ssm_block_norm(rows, C, P(0), P(1), P(2), per, F(3), F(4), 1.f, 1, 0.f, P(5), P(6), 1, nullptr);
}
int norm_bwd(int64_t rows, int64_t C, int64_t per) {
  return ssm_block_norm_bwd(rows, C, P(0), P(1), P(2), per, F(3), F(4), 1.f, 1, 0.f, P(5), P(6), P(7), P(8), P(9), F(10),
                            F(11), 1, ws, sizeof(ws), nullptr);
}

}  // namespace

int main() {
  const int64_t big = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
  const int before = g_ssm_enqueued;
  expect(conv(2, 9, 64, 4) == WKV6_OK, "conv", __LINE__);
  expect(conv_bwd(2, 9, 64, 4) == WKV6_OK, "conv_bwd", __LINE__);
  expect(scan(2, 9, 64, 16, 2) == WKV6_OK, "scan", __LINE__);
  expect(scan_bwd(2, 9, 64, 16, 2) == WKV6_OK, "scan_bwd", __LINE__);
  expect(norm(8, 64, 4) == WKV6_OK, "norm", __LINE__);
  expect(norm_bwd(8, 64, 4) == WKV6_OK, "norm_bwd", __LINE__);
  expect(g_ssm_enqueued - before == 6, "calls enqueued", __LINE__);
  const int64_t odd[] = {0, 1, 3, 8, 64, 129, big, low, -1, big - 7, int64_t(1) << 25, int64_t(1) << 32, int64_t(1) << 62};
  for (int64_t a : odd)
    for (int64_t b : odd)
      for (int64_t c : odd) {
        const int64_t strides[33] = {a, b, c, c, a, b, b, c, a, a, a, a, b, b, b, c, c, c, a, b, c,
                                     a, b, c, a, b, c, a, b, c, a, b, c};
        const int enqueued = g_ssm_enqueued;
        const int st[] = {conv(a, b, c, 4), conv(1, a, 8, b), conv_bwd(a, b, c, 3), conv(3, 5, 64, 4, strides),
                          conv_bwd(3, 5, 64, 4, strides), scan(a, b, c, 16, 1), scan(1, a, 64, b, c), scan_bwd(a, b, c, 8, 1),
                          scan_bwd(1, a, 64, b, c), scan(3, 5, 64, 16, 2, strides), scan_bwd(3, 5, 64, 16, 2, strides),
                          norm(a, b, c), norm_bwd(a, b, c)};
        int good = 0;
        for (int s : st) {
          expect(s >= 0 && s <= 3, "a documented status", __LINE__);
          good += s == WKV6_OK;
        }
        expect(g_ssm_enqueued - enqueued <= good, "refused calls enqueue nothing", __LINE__);
        ssm_conv_bwd_workspace_bytes(a, b, c, 4, 1);
        ssm_scan_bwd_workspace_bytes(a, b, 64, 16, c, 1);
        ssm_block_norm_bwd_workspace_bytes(a, b, c, 1, 1, 1, 1);
      }
  if (failures) return 1;
  std::puts("all argument checks hold");
  return 0;
}
