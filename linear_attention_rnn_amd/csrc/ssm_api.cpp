// C ABI of the selective state space layer's operators: argument checks,
// workspace, launch.  The declarations and their contract live in include/ssm.h.
#include "ssm.h"

#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>
#include <string>

#include "api_checks.h"
#include "ssm_internal.h"

namespace {

// Sizes that the convolution and the scan have in common.  A launch holds fewer
// than 2^32 work-items: the scan's at most 512 for each 8 channels.
int check_sizes(int64_t B, int64_t T, int64_t D, int dtype) {
  if (B < 0 || T < 0 || D < 1) return invalid("sizes must be B, T >= 0 and D >= 1");
  const int st = known_dtype(dtype);
  if (st != WKV6_OK) return st;
  if (D % 8 || D > (1 << 20)) return unsupported("D must be a multiple of 8 up to 2^20");
  if (B > (1 << 25) / D) return unsupported("B * D exceeds the supported range (2^25)");
  if (T > INT_MAX - 4096) return unsupported("T exceeds the supported range");
  return WKV6_OK;
}

// Work-items of a call's largest launch over tokens.
int check_items(int64_t B, int64_t T, int64_t per_token) {
  if (B > 0 && T > 0 && T > ((int64_t(1) << 32) - 1) / per_token / B)
    return unsupported("B * T exceeds the work-items of a launch");
  return WKV6_OK;
}

// ---------------------------------------------------------------- convolution
int conv_sizes(int64_t B, int64_t T, int64_t D, int64_t W, int dtype) {
  int st = check_sizes(B, T, D, dtype);
  if (st != WKV6_OK) return st;
  if (W < 2 || W > SSM_MAX_WINDOW) return unsupported("W must be from 2 to 4");
  // 2 channels and a run of at least 16 tokens for each thread; workgroups hold
  // up to 256 runs, and up to twice the channels there are
  return check_items(B, T / 16 + 258, D + 2);
}

ssm::Conv conv_args(int64_t B, int64_t T, int64_t D, int64_t W, const float* weight, const float* bias, int act,
                    const int32_t* lengths, const void* s_in, int dtype) {
  ssm::Conv a = {};
  a.B = B;
  a.T = T;
  a.D = (int)D;
  a.W = (int)W;
  a.weight = weight;
  a.bias = bias;
  a.lengths = lengths;
  a.s_in = s_in;
  a.silu = act == SSM_ACT_SILU;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return a;
}

// A [B, T, D] tensor of a call with (batch, token) distances.
int rows(const char* name, const void* p, const int64_t* d, int64_t B, int64_t T, int64_t D, int dtype, bool out,
         Tensor* t, Span* s) {
  if (T == 0) {   // nothing of it is touched
    *s = flat(name, nullptr, 0, out);
    return WKV6_OK;
  }
  const int64_t three[3] = {d ? d[0] : T * D, d ? d[1] : D, 0};
  return place(name, p, three, B, T, 1, D, dtype, out, t, s);
}

// ---------------------------------------------------------------- scan
int scan_sizes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int dtype) {
  int st = check_sizes(B, T, D, dtype);
  if (st != WKV6_OK) return st;
  if (G < 1) return invalid("G must be at least 1");
  if (D % G || D / G % 8) return unsupported("D must be a multiple of 8 G");
  if (N < 8 || N > SSM_MAX_STATES || N % 8) return unsupported("N must be a multiple of 8 from 8 to 64");
  return WKV6_OK;
}

ssm::Scan scan_args(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int dtype) {
  ssm::Scan a = {};
  a.B = B;
  a.T = T;
  a.D = (int)D;
  a.N = (int)N;
  a.G = (int)G;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return a;
}

// Tensor i of a scan: of the channels, or of the groups' states.
int scan_tensor(const char* name, const void* p, const int64_t* strides, int i, const ssm::Scan& a, bool groups,
                bool out, Tensor* t, Span* s) {
  const int64_t* d = strides ? strides + 3 * i : nullptr;
  const int dtype = a.bf16 ? WKV6_DTYPE_BF16 : WKV6_DTYPE_F32;
  if (groups && a.T) return place(name, p, d, a.B, a.T, a.G, a.N, dtype, out, t, s);
  return rows(name, p, d, a.B, a.T, a.D, dtype, out, t, s);
}

}  // namespace

extern "C" {

int ssm_abi_version(void) { return SSM_ABI_VERSION; }

int ssm_conv_fwd(int64_t B, int64_t T, int64_t D, int64_t W, const void* x, const float* weight, const float* bias,
                 int act, const int32_t* lengths, const void* s_in, void* y, void* s_out, const int64_t* strides,
                 int dtype, void* stream) try {
  set_error(WKV6_OK, "");
  int st = conv_sizes(B, T, D, W, dtype);
  if (st != WKV6_OK) return st;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return invalid("unknown activation");
  if (B == 0 || (T == 0 && !s_out)) return WKV6_OK;
  ssm::Conv a = conv_args(B, T, D, W, weight, bias, act, lengths, s_in, dtype);
  a.s_out = s_out;
  const int64_t sbytes = B * (W - 1) * D * size_of(dtype);
  Span s[7];
  if ((st = rows("x", x, strides, B, T, D, dtype, false, &a.x, &s[0])) != WKV6_OK ||
      (st = rows("y", y, strides ? strides + 2 : nullptr, B, T, D, dtype, true, &a.y, &s[1])) != WKV6_OK ||
      (st = present("weight", weight)) != WKV6_OK || (st = optional("bias", bias)) != WKV6_OK ||
      (st = optional("lengths", lengths)) != WKV6_OK || (st = optional("s_in", s_in)) != WKV6_OK ||
      (st = optional("s_out", s_out)) != WKV6_OK)
    return st;
  s[2] = flat("weight", weight, D * W * 4, false);
  s[3] = flat("bias", bias, D * 4, false);
  s[4] = flat("lengths", lengths, B * 4, false);
  s[5] = flat("s_in", s_in, sbytes, false);
  s[6] = flat("s_out", s_out, sbytes, true);
  const int allowed[1][2] = {{6, 5}};
  if ((st = check_overlaps(s, 7, allowed, 1)) != WKV6_OK) return st;
  return finished(ssm::enqueue_conv(a, static_cast<hipStream_t>(stream)));
} catch (...) {
  return no_memory();
}

size_t ssm_conv_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t W, int dtype) try {
  set_error(WKV6_OK, "");
  if (conv_sizes(B, T, D, W, dtype) != WKV6_OK) return 0;
  return ssm::conv_bwd_workspace_bytes(conv_args(B, T, D, W, nullptr, nullptr, 0, nullptr, nullptr, dtype));
} catch (...) {
  return 0;
}

int ssm_conv_bwd(int64_t B, int64_t T, int64_t D, int64_t W, const void* x, const float* weight, const float* bias,
                 int act, const int32_t* lengths, const void* s_in, const void* dy, const void* ds_out, void* dx,
                 float* dweight, float* dbias, void* ds_in, const int64_t* strides, int dtype, void* workspace,
                 size_t workspace_bytes, void* stream) try {
  set_error(WKV6_OK, "");
  int st = conv_sizes(B, T, D, W, dtype);
  if (st != WKV6_OK) return st;
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU) return invalid("unknown activation");
  ssm::Conv a = conv_args(B, T, D, W, weight, bias, act, lengths, s_in, dtype);
  a.ds_out = ds_out;
  a.ds_in = ds_in;
  a.dweight = dweight;
  a.dbias = dbias;
  const int64_t sbytes = B * (W - 1) * D * size_of(dtype), tokens = B ? T : 0;
  Span s[11];
  if ((st = rows("x", x, strides, B, tokens, D, dtype, false, &a.x, &s[0])) != WKV6_OK ||
      (st = rows("dy", dy, strides ? strides + 2 : nullptr, B, tokens, D, dtype, false, &a.dy, &s[1])) != WKV6_OK ||
      (st = rows("dx", dx, strides ? strides + 4 : nullptr, B, tokens, D, dtype, true, &a.y, &s[2])) != WKV6_OK ||
      (st = present("weight", weight)) != WKV6_OK || (st = optional("bias", bias)) != WKV6_OK ||
      (st = present("dweight", dweight)) != WKV6_OK || (st = optional("dbias", dbias)) != WKV6_OK)
    return st;
  if (B && ((st = optional("lengths", lengths)) != WKV6_OK || (st = optional("s_in", s_in)) != WKV6_OK ||
            (st = optional("ds_out", ds_out)) != WKV6_OK || (st = optional("ds_in", ds_in)) != WKV6_OK))
    return st;
  s[3] = flat("weight", weight, D * W * 4, false);
  s[4] = flat("bias", bias, D * 4, false);
  s[5] = flat("lengths", B ? lengths : nullptr, B * 4, false);
  s[6] = flat("s_in", B ? s_in : nullptr, sbytes, false);
  s[7] = flat("ds_out", B ? ds_out : nullptr, sbytes, false);
  s[8] = flat("ds_in", B ? ds_in : nullptr, sbytes, true);
  s[9] = flat("dweight", dweight, D * W * 4, true);
  s[10] = flat("dbias", dbias, D * 4, true);
  if ((st = check_overlaps(s, 11, nullptr, 0)) != WKV6_OK) return st;
  Workspace ws(static_cast<hipStream_t>(stream));
  if ((st = ws.take(workspace, workspace_bytes, ssm::conv_bwd_workspace_bytes(a))) != WKV6_OK) return st;
  return ws.done(ssm::enqueue_conv_bwd(a, ws.p, ws.stream));
} catch (...) {
  return no_memory();
}

int ssm_scan_fwd(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* x, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias, int softplus,
                 const int32_t* lengths, const float* s_in, void* y, float* s_out, const int64_t* strides, int dtype,
                 void* stream) try {
  set_error(WKV6_OK, "");
  int st = scan_sizes(B, T, D, N, G, dtype);
  if (st != WKV6_OK || B == 0 || (T == 0 && !s_out)) return st;
  ssm::Scan a = scan_args(B, T, D, N, G, dtype);
  const int64_t sbytes = B * D * N * 4;
  Span s[12];
  if ((st = scan_tensor("x", x, strides, 0, a, false, false, &a.x, &s[0])) != WKV6_OK ||
      (st = scan_tensor("dt", dt, strides, 1, a, false, false, &a.dt, &s[1])) != WKV6_OK ||
      (st = scan_tensor("Bm", Bm, strides, 2, a, true, false, &a.b, &s[2])) != WKV6_OK ||
      (st = scan_tensor("Cm", Cm, strides, 3, a, true, false, &a.c, &s[3])) != WKV6_OK)
    return st;
  s[4] = flat("z", nullptr, 0, false);
  if (z && (st = scan_tensor("z", z, strides, 4, a, false, false, &a.z, &s[4])) != WKV6_OK) return st;
  if ((st = scan_tensor("y", y, strides, 5, a, false, true, &a.y, &s[5])) != WKV6_OK ||
      (st = present("A", A)) != WKV6_OK || (st = optional("skip", skip)) != WKV6_OK ||
      (st = optional("dt_bias", dt_bias)) != WKV6_OK || (st = optional("lengths", lengths)) != WKV6_OK ||
      (st = optional("s_in", s_in)) != WKV6_OK || (st = optional("s_out", s_out)) != WKV6_OK)
    return st;
  s[6] = flat("A", A, D * N * 4, false);
  s[7] = flat("skip", skip, D * 4, false);
  s[8] = flat("dt_bias", dt_bias, D * 4, false);
  s[9] = flat("lengths", lengths, B * 4, false);
  s[10] = flat("s_in", s_in, sbytes, false);
  s[11] = flat("s_out", s_out, sbytes, true);
  const int allowed[1][2] = {{11, 10}};
  if ((st = check_overlaps(s, 12, allowed, 1)) != WKV6_OK) return st;
  a.A = A;
  a.skip = skip;
  a.bias = dt_bias;
  a.softplus = softplus != 0;
  a.lengths = lengths;
  a.s_in = s_in;
  a.s_out = s_out;
  return finished(ssm::enqueue_scan(a, static_cast<hipStream_t>(stream)));
} catch (...) {
  return no_memory();
}

size_t ssm_scan_bwd_workspace_bytes(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, int dtype) try {
  set_error(WKV6_OK, "");
  if (scan_sizes(B, T, D, N, G, dtype) != WKV6_OK) return 0;
  return ssm::scan_bwd_workspace_bytes(scan_args(B, T, D, N, G, dtype));
} catch (...) {
  return 0;
}

int ssm_scan_bwd(int64_t B, int64_t T, int64_t D, int64_t N, int64_t G, const void* x, const void* dt, const float* A,
                 const void* Bm, const void* Cm, const float* skip, const void* z, const float* dt_bias, int softplus,
                 const int32_t* lengths, const float* s_in, const void* dy, const float* ds_out, void* dx, void* ddt,
                 float* dA, void* dB, void* dC, float* dskip, void* dz, float* ddt_bias, float* ds_in,
                 const int64_t* strides, int dtype, void* workspace, size_t workspace_bytes, void* stream) try {
  set_error(WKV6_OK, "");
  int st = scan_sizes(B, T, D, N, G, dtype);
  if (st != WKV6_OK) return st;
  if ((z == nullptr) != (dz == nullptr)) return invalid("z and dz are both given or both null");
  ssm::Scan a = scan_args(B, T, D, N, G, dtype);
  if (B == 0) a.T = 0;
  const int64_t sbytes = B * D * N * 4;
  Span s[21];
  struct {
    const char* name;
    const void* p;
    bool groups, out;
    Tensor* to;
  } const t[11] = {{"x", x, false, false, &a.x},    {"dt", dt, false, false, &a.dt},   {"Bm", Bm, true, false, &a.b},
                   {"Cm", Cm, true, false, &a.c},   {"z", z, false, false, &a.z},      {"dy", dy, false, false, &a.dy},
                   {"dx", dx, false, true, &a.dx},  {"ddt", ddt, false, true, &a.ddt}, {"dB", dB, true, true, &a.db},
                   {"dC", dC, true, true, &a.dc},   {"dz", dz, false, true, &a.dz}};
  for (int i = 0; i < 11; ++i) {
    s[i] = flat(t[i].name, nullptr, 0, t[i].out);
    if (!z && (i == 4 || i == 10)) continue;
    if ((st = scan_tensor(t[i].name, t[i].p, strides, i, a, t[i].groups, t[i].out, t[i].to, &s[i])) != WKV6_OK) return st;
  }
  if ((st = present("A", A)) != WKV6_OK || (st = optional("skip", skip)) != WKV6_OK ||
      (st = optional("dt_bias", dt_bias)) != WKV6_OK || (st = present("dA", dA)) != WKV6_OK ||
      (st = optional("dskip", dskip)) != WKV6_OK || (st = optional("ddt_bias", ddt_bias)) != WKV6_OK)
    return st;
  if (B && ((st = optional("lengths", lengths)) != WKV6_OK || (st = optional("s_in", s_in)) != WKV6_OK ||
            (st = optional("ds_out", ds_out)) != WKV6_OK || (st = optional("ds_in", ds_in)) != WKV6_OK))
    return st;
  s[11] = flat("A", A, D * N * 4, false);
  s[12] = flat("skip", skip, D * 4, false);
  s[13] = flat("dt_bias", dt_bias, D * 4, false);
  s[14] = flat("lengths", B ? lengths : nullptr, B * 4, false);
  s[15] = flat("s_in", B ? s_in : nullptr, sbytes, false);
  s[16] = flat("ds_out", B ? ds_out : nullptr, sbytes, false);
  s[17] = flat("ds_in", B ? ds_in : nullptr, sbytes, true);
  s[18] = flat("dA", dA, D * N * 4, true);
  s[19] = flat("dskip", dskip, D * 4, true);
  s[20] = flat("ddt_bias", ddt_bias, D * 4, true);
  const int allowed[1][2] = {{17, 16}};
  if ((st = check_overlaps(s, 21, allowed, 1)) != WKV6_OK) return st;
  a.A = A;
  a.skip = skip;
  a.bias = dt_bias;
  a.softplus = softplus != 0;
  a.lengths = lengths;
  a.s_in = s_in;
  a.ds_out = ds_out;
  a.ds_in = ds_in;
  a.dA = dA;
  a.dskip = dskip;
  a.dbias = ddt_bias;
  Workspace ws(static_cast<hipStream_t>(stream));
  if ((st = ws.take(workspace, workspace_bytes, ssm::scan_bwd_workspace_bytes(a))) != WKV6_OK) return st;
  return ws.done(ssm::enqueue_scan_bwd(a, ws.p, ws.stream));
} catch (...) {
  return no_memory();
}

}  // extern "C"

namespace {

// ---------------------------------------------------------------- norms between blocks
int norm_sizes(int64_t rows, int64_t C, int64_t gate_rows, bool gate, float scale, int act, float eps, int dtype) {
  if (rows < 0 || C < 1) return invalid("sizes must be rows >= 0 and C >= 1");
  const int st = known_dtype(dtype);
  if (st != WKV6_OK) return st;
  if (!std::isfinite(scale)) return invalid("scale must be finite");
  if (!(std::isfinite(eps) && eps >= 0.f)) return invalid("eps must be finite and >= 0");
  if (act != SSM_ACT_NONE && act != SSM_ACT_SILU && act != SSM_ACT_SIGMOID) return invalid("unknown activation");
  if (!gate && rows > 0 && act != SSM_ACT_NONE) return invalid("an activation without a gate");
  if (gate && (gate_rows < 1 || rows % gate_rows)) return invalid("gate_rows must divide rows");
  if (C % 8 || C > SSM_MAX_COLUMNS) return unsupported("C must be a multiple of 8 up to 16384");
  // a launch holds fewer than 2^32 work-items: 64 at most for each row of up to
  // 512 columns, else up to 1024
  if (rows > (C <= 512 ? 1 << 25 : 1 << 21))
    return unsupported("rows exceed the supported number (2^25, or 2^21 of more than 512 columns)");
  // (the gradients take up to 512 for each gate that rows share)
  if (gate && gate_rows > 1 && rows / gate_rows > (1 << 22)) return unsupported("more than 2^22 gates that rows share");
  return WKV6_OK;
}

ssm::BlockNorm norm_args(int64_t rows, int64_t C, const void* x, const void* gate, int64_t gate_rows, const float* post,
                         const float* pre, float scale, int act, float eps, int dtype) {
  ssm::BlockNorm a = {};
  a.rows = rows;
  a.C = C;
  a.x = x;
  a.gate = gate;
  a.gate_rows = gate ? gate_rows : 1;
  a.post = post;
  a.pre = pre;
  a.scale = scale;
  a.eps = eps;
  a.act = act == SSM_ACT_SILU ? ssm::kSilu : act == SSM_ACT_SIGMOID ? ssm::kSigmoid : ssm::kNone;
  a.bf16 = dtype == WKV6_DTYPE_BF16;
  return a;
}

}  // namespace

extern "C" {

int ssm_block_norm(int64_t rows, int64_t C, const void* x, const void* residual, const void* gate, int64_t gate_rows,
                   const float* post, const float* pre, float scale, int act, float eps, void* h, void* y, int dtype,
                   void* stream) try {
  set_error(WKV6_OK, "");
  int st = norm_sizes(rows, C, gate_rows, gate != nullptr, scale, act, eps, dtype);
  if (st != WKV6_OK || rows == 0) return st;
  if ((pre == nullptr) != (y == nullptr)) return invalid("pre and y are both given or both null");
  if ((st = present("x", x)) != WKV6_OK || (st = optional("residual", residual)) != WKV6_OK ||
      (st = optional("gate", gate)) != WKV6_OK || (st = optional("post", post)) != WKV6_OK ||
      (st = optional("pre", pre)) != WKV6_OK || (st = present("h", h)) != WKV6_OK || (st = optional("y", y)) != WKV6_OK)
    return st;
  const int64_t bytes = rows * C * size_of(dtype);
  const Span s[7] = {flat("x", x, bytes, false),
                     flat("residual", residual, bytes, false),
                     flat("gate", gate, gate ? bytes / gate_rows : 0, false),
                     flat("post", post, C * 4, false),
                     flat("pre", pre, C * 4, false),
                     flat("h", h, bytes, true),
                     flat("y", y, bytes, true)};
  const int allowed[2][2] = {{5, 0}, {5, 1}};
  if ((st = check_overlaps(s, 7, allowed, 2)) != WKV6_OK) return st;
  ssm::BlockNorm a = norm_args(rows, C, x, gate, gate_rows, post, pre, scale, act, eps, dtype);
  a.residual = residual;
  a.h = h;
  a.y = y;
  return finished(ssm::enqueue_block_norm(a, static_cast<hipStream_t>(stream)));
} catch (...) {
  return no_memory();
}

size_t ssm_block_norm_bwd_workspace_bytes(int64_t rows, int64_t C, int64_t gate_rows, int post, int gate, int pre,
                                          int dtype) try {
  set_error(WKV6_OK, "");
  if (norm_sizes(rows, C, gate_rows, gate != 0, 1.f, SSM_ACT_NONE, 0.f, dtype) != WKV6_OK) return 0;
  const float some = 0.f;
  return ssm::block_norm_bwd_workspace_bytes(norm_args(rows, C, nullptr, gate ? &some : nullptr, gate_rows,
                                                       post ? &some : nullptr, pre ? &some : nullptr, 1.f, SSM_ACT_NONE,
                                                       0.f, dtype));
} catch (...) {
  return 0;
}

int ssm_block_norm_bwd(int64_t rows, int64_t C, const void* x, const void* h, const void* gate, int64_t gate_rows,
                       const float* post, const float* pre, float scale, int act, float eps, const void* dy,
                       const void* dh, void* dx, void* dresidual, void* dgate, float* dpost, float* dpre, int dtype,
                       void* workspace, size_t workspace_bytes, void* stream) try {
  set_error(WKV6_OK, "");
  int st = norm_sizes(rows, C, gate_rows, gate != nullptr, scale, act, eps, dtype);
  if (st != WKV6_OK) return st;
  if ((post == nullptr) != (dpost == nullptr)) return invalid("post and dpost are both given or both null");
  if ((pre == nullptr) != (dpre == nullptr)) return invalid("pre and dpre are both given or both null");
  if ((st = optional("post", post)) != WKV6_OK || (st = optional("pre", pre)) != WKV6_OK ||
      (st = optional("dpost", dpost)) != WKV6_OK || (st = optional("dpre", dpre)) != WKV6_OK)
    return st;
  if (rows > 0) {
    if ((pre == nullptr) != (dy == nullptr)) return invalid("pre and dy are both given or both null");
    if ((gate == nullptr) != (dgate == nullptr)) return invalid("gate and dgate are both given or both null");
    if ((st = present("x", x)) != WKV6_OK || (pre && (st = present("h", h)) != WKV6_OK) ||
        (st = optional("gate", gate)) != WKV6_OK || (st = optional("dy", dy)) != WKV6_OK ||
        (st = optional("dh", dh)) != WKV6_OK || (st = present("dx", dx)) != WKV6_OK ||
        (st = optional("dresidual", dresidual)) != WKV6_OK || (st = optional("dgate", dgate)) != WKV6_OK)
      return st;
  }
  const int64_t bytes = rows * C * size_of(dtype), gbytes = gate ? bytes / gate_rows : 0;
  const auto some = [&](const void* p) { return rows > 0 ? p : nullptr; };
  const Span s[12] = {flat("x", some(x), bytes, false),
                      flat("h", some(pre ? h : nullptr), bytes, false),
                      flat("gate", some(gate), gbytes, false),
                      flat("post", post, C * 4, false),
                      flat("pre", pre, C * 4, false),
                      flat("dy", some(dy), bytes, false),
                      flat("dh", some(dh), bytes, false),
                      flat("dx", some(dx), bytes, true),
                      flat("dresidual", some(dresidual), bytes, true),
                      flat("dgate", some(dgate), gbytes, true),
                      flat("dpost", dpost, C * 4, true),
                      flat("dpre", dpre, C * 4, true)};
  const int allowed[2][2] = {{7, 5}, {8, 6}};
  if ((st = check_overlaps(s, 12, allowed, 2)) != WKV6_OK) return st;
  ssm::BlockNorm a = norm_args(rows, C, x, some(gate), gate_rows, post, pre, scale, act, eps, dtype);
  a.h = const_cast<void*>(h);
  a.dy = dy;
  a.dh = dh;
  a.dx = dx;
  a.dresidual = dresidual;
  a.dgate = dgate;
  a.dpost = dpost;
  a.dpre = dpre;
  Workspace ws(static_cast<hipStream_t>(stream));
  if ((st = ws.take(workspace, workspace_bytes, ssm::block_norm_bwd_workspace_bytes(a))) != WKV6_OK) return st;
  return ws.done(ssm::enqueue_block_norm_bwd(a, ws.p, ws.stream));
} catch (...) {
  return no_memory();
}

}  // extern "C"
