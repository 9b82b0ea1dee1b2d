// Outputs beside inputs and one another in one buffer (linattn.h's strides):
// slices that lie side by side are accepted whatever their head sizes, and
// nothing that shares a byte is.  Built with the host sanitizers; the kernel
// side is stubs.  Exits 0 when all of it holds.
#include <cstdint>
#include <cstdio>
#include <random>
#include <set>

#include "linattn.h"

extern int g_linattn_enqueued;

namespace {

int failures = 0;
void expect(bool ok, const char* what, int line) {
  if (ok) return;
  std::fprintf(stderr, "FAILED line %d: %s (last error: %s)\n", line, what, wkv6_last_error());
  ++failures;
}
#define EXPECT(x) expect((x), #x, __LINE__)

char* P(int i) { return reinterpret_cast<char*>(uintptr_t(0x1000000000ull) * (i + 1)); }
float* F(int i) { return reinterpret_cast<float*>(P(i)); }
char ws[1 << 16] __attribute__((aligned(16)));

// dq, dk and dv as slices [.., D] of rows of `row` elements of bfloat16, at element offsets
int bwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int64_t row, int64_t oq, int64_t ok, int64_t ov) {
  const int64_t b = T * row;
  const int64_t s[21] = {T * H * K, H * K, K, T * H * K, H * K, K, T * H * V, H * V, V, T * H * V, H * V, V,
                         b, row, K, b, row, K, b, row, V};
  char* const g = P(9);
  return linattn_bwd(B, T, H, K, V, P(0), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(4), nullptr, g + 2 * oq, g + 2 * ok,
                     g + 2 * ov, nullptr, s, 1, 1, ws, sizeof(ws), nullptr);
}

// q at P(4), o `d` bytes after it, with distances in elements
int fwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, const int64_t* sq, const int64_t* so, int64_t d, int dtype, int out) {
  int64_t s[12] = {T * H * K, H * K, K, T * H * K, H * K, K, T * H * V, H * V, V, T * H * V, H * V, V};
  for (int i = 0; i < 3; ++i) s[i] = sq[i], s[9 + i] = so[i];
  return linattn_fwd(B, T, H, K, V, P(4), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(4) + d, nullptr, s, dtype, out, ws,
                     sizeof(ws), nullptr);
}

std::set<int64_t> places(int64_t B, int64_t T, int64_t H, int64_t D, const int64_t* s, int z, int64_t at) {
  std::set<int64_t> p;   // 16-byte places
  for (int64_t b = 0; b < B; ++b)
    for (int64_t t = 0; t < T; ++t)
      for (int64_t h = 0; h < H; ++h)
        for (int64_t c = 0; c < D * z; c += 16) p.insert((at + (b * s[0] + t * s[1] + h * s[2]) * z + c) / 16);
  return p;
}

}  // namespace

int main() {
  // [B, T, H (2 K + V)]: all queries' gradients of a token, then all keys', then all values'
  for (int64_t B : {1, 3})
    for (int64_t T : {1, 9, 70})
      for (int64_t H : {1, 2, 5})
        for (int64_t K : {8, 64, 128})
          for (int64_t V : {8, 64, 128}) {
            const int64_t row = H * (2 * K + V);
            EXPECT(bwd(B, T, H, K, V, row, 0, H * K, 2 * H * K) == WKV6_OK);
            EXPECT(bwd(B, T, H, K, V, row, H * V, H * (V + K), 0) == WKV6_OK);
            EXPECT(bwd(B, T, H, K, V, row + 40, 8, H * K + 16, 2 * H * K + 24) == WKV6_OK);
            if (T > 1 || B > 1) {
              EXPECT(bwd(B, T, H, K, V, row, 0, H * K, 2 * H * K - 8) == WKV6_ERR_INVALID_ARG);
              EXPECT(bwd(B, T, H, K, V, row, 0, H * K, 2 * H * K + 8) == WKV6_ERR_INVALID_ARG);   // reaches the next token's dq
              EXPECT(bwd(B, T, H, K, V, row - 8, 0, H * K, 2 * H * K) == WKV6_ERR_INVALID_ARG);
            }
          }
  // whatever is accepted shares nothing
  std::mt19937 r(7);
  const auto pick = [&](int64_t n) { return (int64_t)(r() % n); };
  int accepted = 0, close = 0;
  for (int i = 0; i < 60000; ++i) {
    const int64_t B = 1 + pick(3), T = 1 + pick(3), H = 1 + pick(3), K = 8 * (1 + pick(3)), V = 8 * (1 + pick(3));
    const int dtype = (int)pick(2), out = dtype ? (int)pick(2) : 0;
    int64_t sq[3], so[3];
    const int64_t h = 8 * pick(6), t = 8 * pick(18), b = 8 * pick(50);
    for (int64_t* s : {sq, so}) {   // often the same distances
      s[2] = pick(3) ? h : 8 * pick(6);
      s[1] = pick(4) ? t : 8 * pick(18);
      s[0] = pick(4) ? b : 8 * pick(50);
    }
    const int64_t d = 16 * (pick(400) - 200);
    const int st = fwd(B, T, H, K, V, sq, so, d, dtype, out);
    EXPECT(st == WKV6_OK || st == WKV6_ERR_INVALID_ARG);
    if (st != WKV6_OK) continue;
    ++accepted;
    const auto q = places(B, T, H, K, sq, dtype ? 2 : 4, 1 << 20), o = places(B, T, H, V, so, out ? 2 : 4, (1 << 20) + d);
    bool shared = false;
    for (int64_t x : o) shared = shared || q.count(x);
    EXPECT(!shared);
    EXPECT((int64_t)o.size() == B * T * H * V * (out ? 2 : 4) / 16);   // and its rows are places of their own
    close += *o.begin() <= *q.rbegin() && *q.begin() <= *o.rbegin();
  }
  EXPECT(accepted > 1000 && close > 50);   // some of them within one another
  if (failures) return 1;
  std::printf("all slices hold (%d accepted, %d within one another)\n", accepted, close);
  return 0;
}
