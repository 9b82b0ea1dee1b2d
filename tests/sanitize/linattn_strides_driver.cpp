// Distances between tokens (linattn.h): as far apart as the kernels reach, and
// refused beyond, in bytes of the tensor's own type; single tokens and rotary
// positions at any distance; log_decay and positions at any element of a table.
// Built with the host sanitizers; the kernel side is stubs.  Exits 0 when all
// of it holds.
#include <cstdint>
#include <cstdio>

#include "linattn.h"

namespace {

int failures = 0;
void expect(bool ok, const char* what, int line) {
  if (ok) return;
  std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, wkv6_last_error());
  ++failures;
}
#define EXPECT(x) expect((x), #x, __LINE__)

char* P(int i) { return reinterpret_cast<char*>(uintptr_t(0x1000000000000ull) * (i + 1)); }
float* F(int i) { return reinterpret_cast<float*>(P(i)); }
char ws[1 << 16] __attribute__((aligned(16)));

int fwd(int64_t T, int64_t H, int dtype, int out, const int64_t* s, const float* decay = F(3)) {
  return linattn_fwd(1, T, H, 64, 64, P(0), P(1), P(2), decay, 1.f, nullptr, nullptr, P(4), nullptr, s, dtype, out, ws,
                     sizeof(ws), nullptr);
}
int bwd(int64_t T, int dtype, int grad, const int64_t* s) {
  return linattn_bwd(1, T, 1, 64, 64, P(0), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(4), nullptr, P(5), P(6), P(7),
                     nullptr, s, dtype, grad, ws, sizeof(ws), nullptr);
}
int rope(int64_t T, int64_t H, int dtype, const int64_t* s, const int32_t* positions = nullptr) {
  return linattn_rope(1, T, H, 64, 64, P(0), nullptr, P(1), nullptr, positions, 0, reinterpret_cast<double*>(P(4)), 0, 0, s,
                      dtype, nullptr);
}

}  // namespace

int main() {
  const int64_t most = 33554288;   // bytes: 64 rows within 2^31 - 8192
  for (int dtype = 0; dtype < 2; ++dtype) {
    const int z = dtype ? 2 : 4;
    for (int which = 0; which < 4; ++which) {   // q, k, v, o
      int64_t s[12] = {0, 64, 64, 0, 64, 64, 0, 64, 64, 0, 64, 64};
      s[3 * which + 1] = most / z;
      EXPECT(fwd(9, 1, dtype, dtype, s) == WKV6_OK && fwd(8, 1, dtype, dtype, s) == WKV6_OK);
      s[3 * which + 1] = (most + 16) / z;
      EXPECT(fwd(9, 1, dtype, dtype, s) == WKV6_ERR_UNSUPPORTED);
      EXPECT(fwd(8, 1, dtype, dtype, s) == WKV6_OK && fwd(1, 1, dtype, dtype, s) == WKV6_OK);
    }
    for (int which = 0; which < 7; ++which) {   // q, k, v, d_o, dq, dk, dv
      int64_t s[21];
      for (int i = 0; i < 21; ++i) s[i] = i % 3 ? 64 : 0;
      s[3 * which + 1] = most / z;
      EXPECT(bwd(2, dtype, dtype, s) == WKV6_OK);
      s[3 * which + 1] = (most + 16) / z;
      EXPECT(bwd(2, dtype, dtype, s) == WKV6_ERR_UNSUPPORTED && bwd(1, dtype, dtype, s) == WKV6_OK);
    }
    // contiguous tensors of many heads
    EXPECT(fwd(9, most / z / 64, dtype, dtype, nullptr) == WKV6_OK && fwd(9, most / z / 64 + 1, dtype, dtype, nullptr) == WKV6_ERR_UNSUPPORTED);
    EXPECT(rope(9, 1 << 20, dtype, nullptr) == WKV6_OK);
    const int64_t far[12] = {0, int64_t(1) << 33, 64, 0, 0, 0, 0, int64_t(1) << 33, 64, 0, 0, 0};
    EXPECT(rope(9, 1, dtype, far) == WKV6_OK);
  }
  // an out_dtype of its own: o's distance counts in its own bytes
  int64_t s[12] = {0, 64, 64, 0, 64, 64, 0, 64, 64, 0, most / 4 + 4, 64};
  EXPECT(fwd(9, 1, 1, 1, s) == WKV6_OK && fwd(9, 1, 1, 0, s) == WKV6_ERR_UNSUPPORTED);
  // one layer's row of a table, one sequence's of the positions
  for (int i = 1; i < 4; ++i) {
    EXPECT(fwd(9, 3, 1, 1, nullptr, F(3) + i) == WKV6_OK);
    EXPECT(rope(3, 1, 1, nullptr, reinterpret_cast<int32_t*>(P(6)) + i) == WKV6_OK);
    EXPECT(fwd(9, 3, 1, 1, nullptr, reinterpret_cast<float*>(P(3) + i)) == WKV6_ERR_MISALIGNED);
    EXPECT(rope(3, 1, 1, nullptr, reinterpret_cast<int32_t*>(P(6) + i)) == WKV6_ERR_MISALIGNED);
  }
  if (failures) return 1;
  std::puts("all distances hold");
  return 0;
}
