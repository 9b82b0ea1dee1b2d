// The launches and workspaces of the attention calls (linattn_plan.h) over
// sizes up to the limits: no launch of an accepted call holds 2^32 work-items,
// segments cover every token, and the workspace holds every segment's state.
// Built with the host sanitizers; the kernel side is stubs.  Exits 0 when all
// of it holds.
#include <cstdint>
#include <cstdio>
#include <cstring>

#include "linattn.h"
#include "linattn_plan.h"

extern int g_linattn_enqueued;

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

int fwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int out) {
  return linattn_fwd(B, T, H, K, V, P(0), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(4), nullptr, nullptr, dtype, out,
                     P(5), ~size_t(0), nullptr);
}
int bwd(int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, int dtype, int grad) {
  return linattn_bwd(B, T, H, K, V, P(0), P(1), P(2), F(3), 1.f, nullptr, nullptr, P(4), nullptr, P(5), P(6), P(7),
                     nullptr, nullptr, dtype, grad, P(8), ~size_t(0), nullptr);
}

linattn::Sweep sweep(int64_t B, int64_t T, int64_t H, int K, int V, bool bf16, bool transposed, const int32_t* lengths) {
  linattn::Sweep a = {};
  a.B = B;
  a.T = T;
  a.H = H;
  a.K = K;
  a.V = V;
  a.bf16 = bf16;
  a.s_transposed = transposed;
  a.lengths = lengths;
  return a;
}

// One launch's plan against what it has to hold.
void check_plan(const linattn::Sweep* a, int n, size_t bytes) {
  using namespace linattn;
  const SweepPlan p = plan(a, n);
  int blocks = 0;
  for (int i = 0; i < n; ++i) blocks += (a[i].V + 63) / 64;
  EXPECT(p.blocks == blocks && p.pairs == a->B * a->H && p.items == p.pairs * p.segments);
  EXPECT(p.seg_tokens % 64 == 0 && p.segments >= 1);
  EXPECT((int64_t)p.segments * p.seg_tokens >= a->T && (int64_t)(p.segments - 1) * p.seg_tokens < a->T);
  // every item and block of values has a workgroup
  EXPECT(sweep_groups(p, p.items) >= p.items * blocks && sweep_groups(p, p.items) < (p.items + 8) * blocks);
  const int KP = widest(a, n) <= 64 ? 64 : 128;
  if (p.segments > 1) {
    // the last place that the kernels address
    const int64_t state = KP * 64 * p.vblocks, last = (((n - 1) * p.pairs + p.pairs - 1) * p.segments + p.segments - 1) * state;
    EXPECT((size_t)(last + state) * 4 <= bytes);
  }
}

void check_call(const linattn::Sweep* a, int n) {
  using namespace linattn;
  const size_t bytes = planned_workspace_bytes(a, n);
  if (steps(a, n)) {
    EXPECT(bytes == 0);
    return;
  }
  if (const Split s = split(a, n); s.n[0]) {
    EXPECT(s.n[0] + s.n[1] == n && s.n[1] >= 1);
    for (int g = 0; g < 2; ++g) check_plan(s.a[g], s.n[g], bytes);
    return;
  }
  check_plan(a, n, bytes);
}

}  // namespace

int main() {
  const int64_t tokens[] = {1, 8, 9, 64, 65, 127, 129, 448, 449, 512, 777, 1023, 4096, 16384, 1000003, 2147483583};
  const int64_t pairs[] = {1, 2, 3, 8, 12, 24, 79, 80, 127, 128, 159, 160, 161, 255, 257, 400, 5000, 70000, 1398096, 1398097, 2097152};
  const int sizes[] = {8, 64, 72, 128};
  const int32_t some = 0;
  for (int64_t T : tokens)
    for (int64_t n : pairs)
      for (int K : sizes)
        for (int V : sizes)
          for (int bf = 0; bf < 2; ++bf) {
            size_t had = 0;
            for (int padded = 0; padded < 2; ++padded) {
              const int32_t* const lengths = padded ? &some : nullptr;
              const linattn::Sweep f = sweep(n, T, 1, K, V, bf, false, lengths);
              check_call(&f, 1);
              const linattn::Sweep w[3] = {sweep(n, T, 1, V, K, bf, true, lengths), sweep(n, T, 1, V, K, bf, true, lengths),
                                           sweep(n, T, 1, K, V, bf, false, lengths)};
              check_call(w, 3);
              // the workspace functions answer for calls with lengths: those take as much as others or more
              const size_t takes = linattn::planned_workspace_bytes(&f, 1) + linattn::planned_workspace_bytes(w, 3);
              EXPECT(takes >= had);
              had = takes;
              // refused exactly where a launch would hold 2^32 work-items
              if (T == 1 || T == 9) {
                const int before = g_linattn_enqueued;
                const int64_t most = linattn::largest_launch(w, 3);
                const int st = bwd(n, T, 1, K, V, bf, bf);
                EXPECT(st == (most < (int64_t(1) << 32) ? WKV6_OK : WKV6_ERR_UNSUPPORTED));
                EXPECT(g_linattn_enqueued - before == (st == WKV6_OK));
                EXPECT(linattn::largest_launch(&f, 1) < (int64_t(1) << 32) && fwd(n, T, 1, K, V, bf, bf) == WKV6_OK);
              }
            }
          }
  // the limit itself: 6 workgroups of 512 for each pair
  EXPECT(bwd(1398096, 1, 1, 128, 128, 0, 0) == WKV6_OK);
  EXPECT(bwd(1398097, 1, 1, 128, 128, 0, 0) == WKV6_ERR_UNSUPPORTED && std::strstr(wkv6_last_error(), "launch"));
  EXPECT(bwd(1 << 21, 1, 1, 72, 72, 0, 0) == WKV6_ERR_UNSUPPORTED);
  EXPECT(bwd(1 << 21, 1, 1, 128, 128, 1, 0) == WKV6_OK && bwd(1 << 21, 1, 1, 128, 64, 0, 0) == WKV6_OK &&
         bwd(1 << 21, 1, 1, 64, 128, 0, 0) == WKV6_OK && fwd(1 << 21, 9, 1, 128, 128, 0, 0) == WKV6_OK);
  if (failures) return 1;
  std::puts("all plans hold");
  return 0;
}
