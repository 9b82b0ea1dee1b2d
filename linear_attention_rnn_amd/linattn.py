"""ctypes binding of the linear-attention operators (C ABI in
include/linattn.h, in libwkv6.so).

Argument marshalling only, as in ``linear_attention_rnn_amd.wkv6``: every
computation runs in the library's HIP kernels, PyTorch provides device memory
and the current HIP stream, and there is no fallback.  Calls run on the
inputs' GPU whichever device is current.

Calls on torch's current stream take their workspace from torch's allocator
(a call of the library's pool costs the host 11 us, torch's 1.3) and can be
captured in a HIP graph (``torch.cuda.graph``).  Calls with a ``stream`` of
their own take it from the library's pool; to be recorded there they are given
a ``workspace``, a uint8 tensor of at least ``fwd_workspace_bytes`` /
``bwd_workspace_bytes`` bytes.  New outputs always come from torch's allocator
on its current stream: with a ``stream`` of their own, callers order the two
streams.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import wkv6
from .wkv6 import DTYPE_BF16, DTYPE_F32, OK, _stream_handle

MAX_HEAD = 128          # LINATTN_MAX_HEAD
MAX_COLUMNS = 16384     # LINATTN_MAX_COLUMNS
_LAYOUTS = {"half": 0, "interleaved": 1}
_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}

_fns = None


class LinattnError(wkv6.WKV6Error):
    def __init__(self, name: str, status: int):
        RuntimeError.__init__(self, f"{name} failed with status {status}: {wkv6.status_str(status)}: "
                                    f"{wkv6.last_error()}")
        self.status = status


def lib() -> ctypes.CDLL:
    """The library, with the argument types of linattn.h set (once)."""
    global _fns
    L = wkv6.lib()
    if _fns is not L:
        i64, vp, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        tail = [vp, sz, vp]   # workspace, its bytes, stream
        L.linattn_fwd.argtypes = [i64] * 5 + [vp] * 4 + [f32] + [vp] * 5 + [i32, i32] + tail
        L.linattn_bwd.argtypes = [i64] * 5 + [vp] * 4 + [f32] + [vp] * 9 + [i32, i32] + tail
        L.linattn_rope.argtypes = [i64] * 5 + [vp] * 5 + [i64, vp, i32, i32, vp, i32, vp]
        L.linattn_rms_norm.argtypes = [i64, i64, vp, vp, vp, f32, vp, vp, i32, vp]
        L.linattn_rms_norm_q8.argtypes = [i64, i64, vp, vp, vp, f32, vp, vp, vp, i32, i32, vp]
        L.linattn_rms_norm_bwd.argtypes = [i64, i64, vp, vp, vp, vp, f32, vp, vp, i32] + tail
        for f in (L.linattn_fwd, L.linattn_bwd, L.linattn_rope, L.linattn_rms_norm, L.linattn_rms_norm_q8,
                  L.linattn_rms_norm_bwd, L.linattn_abi_version):
            f.restype = i32
        L.linattn_abi_version.argtypes = []
        for f in (L.linattn_fwd_workspace_bytes, L.linattn_bwd_workspace_bytes):
            f.argtypes, f.restype = [i64] * 5 + [i32] * 3, sz
        L.linattn_rms_norm_bwd_workspace_bytes.argtypes = [i64, i64, i32]
        L.linattn_rms_norm_bwd_workspace_bytes.restype = sz
        _fns = L
    return L


def abi_version() -> int:
    return lib().linattn_abi_version()


def fwd_workspace_bytes(B, T, H, K, V, dtype=torch.bfloat16, out_dtype=None, state_out=False) -> int:
    """Workspace bytes of a fwd call of these sizes (host arithmetic)."""
    return lib().linattn_fwd_workspace_bytes(B, T, H, K, V, _DTYPES[dtype], _DTYPES[out_dtype or dtype], state_out)


def bwd_workspace_bytes(B, T, H, K, V, dtype=torch.bfloat16, grad_dtype=torch.float32, state_grad=False) -> int:
    """Workspace bytes of a bwd call of these sizes (host arithmetic)."""
    return lib().linattn_bwd_workspace_bytes(B, T, H, K, V, _DTYPES[dtype], _DTYPES[grad_dtype], state_grad)


# ---------------------------------------------------------------- checks
# These run before every call and are most of what a call costs the host next
# to the launch itself (3 us of 6.5 for a single-token step), hence few and
# plain expressions, and none for tensors made here.
def _dtype(t, name):
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return d


def _tensor(t, name, shape, dtype, device):
    """A [B, T, H, D] tensor with adjacent channels on the call's GPU; returns
    its address."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on the GPU of the first tensor, {device}")
    if not t.is_contiguous() and t.stride(3) != 1 and shape[3] > 1:
        raise ValueError(f"the channels of {name} must be adjacent")
    return t.data_ptr()


def _flat(t, name, shape, dtype, device):
    """A contiguous tensor of one shape and type on the call's GPU; returns its
    address, 0 for None."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


def _strides(*tensors):
    """(batch, token, head) distances of each, or None if all are contiguous."""
    for t in tensors:
        if t is not None and not t.is_contiguous():
            break
    else:
        return None
    out = []
    for t in tensors:
        out += t.stride()[:3] if t is not None else (0, 0, 0)
    return (ctypes.c_int64 * len(out))(*out)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(name, f, device, stream, *args):
    """The library call, with the inputs' GPU current and on `stream` or torch's
    current one."""
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = _stream_handle(stream, device)
    if _current_device() == device.index:
        status = f(*args, handle)
    else:
        with torch.cuda.device(device):
            status = f(*args, handle)
    if status != OK:
        raise LinattnError(name, status)


def _workspace(given, need, device, stream):
    """(address, bytes, tensor kept alive) of a call's workspace; need() gives
    its bytes.  Nothing where the library's pool serves (a stream of the
    caller's) or none is needed."""
    if given is not None:
        if given.dtype != torch.uint8 or given.device != device or not given.is_contiguous():
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
        return given.data_ptr(), given.numel(), given
    if stream is None:
        n = need()
        if n:
            t = torch.empty(n, dtype=torch.uint8, device=device)
            return t.data_ptr(), n, t
    return _NO_WORKSPACE


_NO_WORKSPACE = (0, 0, None)
_STEP_TOKENS = 8   # fwd calls of at most so many tokens take no workspace


def _attention(q, k, v, log_decay, lengths):
    """Sizes, type, GPU and addresses of what fwd and bwd have in common."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k, v must be [B, T, H, channels]")
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    shape, t, dev = q.shape, q.dtype, q.device
    B, T, H, K = shape
    V = v.shape[3]
    dtype = _dtype(q, "q, k, v")
    return (B, T, H, K, V, dtype, dev, _tensor(q, "q", shape, t, dev), _tensor(k, "k", shape, t, dev),
            _tensor(v, "v", (B, T, H, V), t, dev), _flat(log_decay, "log_decay", (H,), torch.float32, dev),
            _flat(lengths, "lengths", (B,), torch.int32, dev))


# ---------------------------------------------------------------- attention
def fwd(q, k, v, log_decay, scale: float = 1.0, lengths=None, s_in=None, want_state: bool = False, out=None,
        s_out=None, out_dtype=None, workspace=None, stream=None):
    """Linear attention with one decay for each head: (o, s_out).

    Per sequence and head, with a = exp(log_decay[h]):
    S_t = a S_{t-1} + k_t^T v_t from s_in (or zero), o_t = scale * q_t S_t.

    q, k: [B, T, H, K], v: [B, T, H, V], float32 or bfloat16, any distances
    between batch items, tokens and heads (channels adjacent; an expanded
    tensor repeats its rows); log_decay: float32 [H]; lengths: None or int32
    [B] (padded batch: rows behind a sequence are not read, their outputs are
    zero); s_in: None or float32 [B, H, K, V].  o is `out`, or a new
    [B, T, H, V] tensor of `out_dtype` (default: q's type; float32 for float32
    inputs).  The state after the last token goes to `s_out` (which may be
    s_in), or to a new tensor if `want_state`; otherwise None is returned for
    it.
    """
    B, T, H, K, V, dtype, dev, pq, pk, pv, pg, pl = _attention(q, k, v, log_decay, lengths)
    if out is None:
        out = torch.empty((B, T, H, V), dtype=out_dtype or q.dtype, device=dev)
        py = out.data_ptr()
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise ValueError("out must have out_dtype")
        py = _tensor(out, "out", (B, T, H, V), out.dtype, dev)
    odt = _dtype(out, "out")
    ps = _flat(s_in, "s_in", (B, H, K, V), torch.float32, dev)
    if s_out is not None:
        po = ps if s_out is s_in else _flat(s_out, "s_out", (B, H, K, V), torch.float32, dev)
    elif want_state:
        s_out = torch.empty((B, H, K, V), dtype=torch.float32, device=dev)
        po = s_out.data_ptr()
    else:
        po = 0
    L = lib()
    pw, nw, keep = _NO_WORKSPACE if T <= _STEP_TOKENS else _workspace(
        workspace, lambda: L.linattn_fwd_workspace_bytes(B, T, H, K, V, dtype, odt, po != 0), dev, stream)
    _call("linattn_fwd", L.linattn_fwd, dev, stream, B, T, H, K, V, pq, pk, pv, pg, scale, pl, ps, py, po,
          _strides(q, k, v, out), dtype, odt, pw, nw)
    return out, s_out


def bwd(q, k, v, log_decay, do, scale: float = 1.0, lengths=None, s_in=None, ds_out=None, want_ds_in: bool = False,
        grad_dtype=torch.float32, out=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(o * do) + sum(s_out * ds_out) for (o, s_out) = fwd(...).

    do: [B, T, H, V] of q's type; ds_out: None or float32 [B, H, K, V].
    Returns {"q", "k", "v"} of `grad_dtype` (float32, or bfloat16 for bfloat16
    inputs), and "s_in" (float32) if `want_ds_in`.  `out`: a dict of tensors to
    write "q", "k", "v" and "s_in" to instead of new ones (slices of one buffer
    are fine).  Expanded inputs get the gradient of every place they are used
    at: the caller sums them.
    """
    B, T, H, K, V, dtype, dev, pq, pk, pv, pg, pl = _attention(q, k, v, log_decay, lengths)
    pdo = _tensor(do, "do", (B, T, H, V), q.dtype, dev)
    ps = _flat(s_in, "s_in", (B, H, K, V), torch.float32, dev)
    pd = _flat(ds_out, "ds_out", (B, H, K, V), torch.float32, dev)
    g = dict(out) if out else {}
    for name, D in (("q", K), ("k", K), ("v", V)):
        if name not in g:
            g[name] = torch.empty((B, T, H, D), dtype=grad_dtype, device=dev)
        _tensor(g[name], "d" + name, (B, T, H, D), g["q"].dtype, dev)
    gdt = _dtype(g["q"], "gradients")
    if want_ds_in and "s_in" not in g:
        g["s_in"] = torch.empty((B, H, K, V), dtype=torch.float32, device=dev)
    pi = _flat(g.get("s_in"), "ds_in", (B, H, K, V), torch.float32, dev)
    L = lib()
    pw, nw, keep = _workspace(
        workspace, lambda: L.linattn_bwd_workspace_bytes(B, T, H, K, V, dtype, gdt, pi != 0), dev, stream)
    _call("linattn_bwd", L.linattn_bwd, dev, stream, B, T, H, K, V, pq, pk, pv, pg, scale, pl, ps, pdo, pd,
          g["q"].data_ptr(), g["k"].data_ptr(), g["v"].data_ptr(), pi,
          _strides(q, k, v, do, g["q"], g["k"], g["v"]), dtype, gdt, pw, nw)
    return g


# ---------------------------------------------------------------- rotary positions
def rope_freqs(R: int, base: float = 10000.0, scaling=None, factor: float = 1.0, original: int = 4096,
               slow_turns: float = 1.0, fast_turns: float = 32.0, device="cuda"):
    """Angles per position of R / 2 pairs, float64: base^(-2i/R), for

    scaling None: as they are;
    "linear":  all divided by `factor` (positions interpolated);
    "base":    base multiplied by factor^(R / (R - 2)), which leaves the first
               pair alone and divides the last by `factor`;
    "bands":   divided by `factor` for pairs with at most `slow_turns` turns
               over the `original` context, as they are from `fast_turns` on,
               blended linearly in their turns between.
    """
    if R < 2 or R % 2:
        raise ValueError("R must be even and positive")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'bands'")
    if scaling is not None and not factor > 0:
        raise ValueError("factor must be positive")
    if scaling == "base":
        if R < 4:
            raise ValueError("scaling by the base needs two pairs")
        base = base * factor ** (R / (R - 2))
    f = base ** (-2.0 * torch.arange(R // 2, dtype=torch.float64) / R)
    if scaling == "linear":
        f = f / factor
    elif scaling == "bands":
        if not fast_turns > slow_turns:
            raise ValueError("fast_turns must be above slow_turns")
        keep = ((original * f / (2.0 * math.pi) - slow_turns) / (fast_turns - slow_turns)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f.to(device)


def rope(q, k, freqs, positions=None, start: int = 0, layout: str = "half", inverse: bool = False, q_out=None,
         k_out=None, stream=None):
    """Rotary positions of q and k ([B, T, H, D]; k may be None): (q_out, k_out).

    Pair i of the first R = 2 * len(freqs) channels, (i, i + R/2) for layout
    "half" or (2i, 2i + 1) for "interleaved", turns by position * freqs[i];
    the other channels are copied.  The position of token t is start + t, or
    start + positions[b, t] (int32 [B, T]).  `inverse` turns back: applied to
    gradients of the outputs it gives those of the inputs.  q_out may be q and
    k_out k (in place).
    """
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}")
    if q.dim() != 4:
        raise ValueError("q must be [B, T, H, D]")
    if not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    shape, t, dev = q.shape, q.dtype, q.device
    B, T, H, D = shape
    dtype = _dtype(q, "q and k")
    pq = _tensor(q, "q", shape, t, dev)
    if freqs is None or freqs.dim() != 1:
        raise ValueError("freqs must be a float64 vector of R / 2 values")
    pf = _flat(freqs, "freqs", freqs.shape, torch.float64, dev)
    pp = _flat(positions, "positions", (B, T), torch.int32, dev)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        pqo = q_out.data_ptr()
    else:
        pqo = pq if q_out is q else _tensor(q_out, "q_out", shape, t, dev)
    pk = pko = 0
    if k is not None:
        pk = _tensor(k, "k", shape, t, dev)
        if k_out is None:
            k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
            pko = k_out.data_ptr()
        else:
            pko = pk if k_out is k else _tensor(k_out, "k_out", shape, t, dev)
    elif k_out is not None:
        raise ValueError("k_out without k")
    _call("linattn_rope", lib().linattn_rope, dev, stream, B, T, H, D, 2 * freqs.shape[0], pq, pk, pqo, pko, pp, start,
          pf, _LAYOUTS[layout], inverse, _strides(q, k, q_out, k_out), dtype)
    return q_out, k_out


def _turned(q, k, freqs, positions, start, layout, stream):
    """Turned copies of q and k that live for one call on `stream`: torch's
    allocator must not hand them out on its own stream before that has run."""
    q, k = rope(q, k, freqs, positions, start, layout, stream=stream)
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), q.device)
        q.record_stream(s)
        k.record_stream(s)
    return q, k


def retention(q, k, v, log_decay, freqs, positions=None, start: int = 0, layout: str = "half", **fwd_arguments):
    """fwd of q and k turned by their positions: a state whose decay is complex,
    exp(log_decay[h] + i freqs).  Returns (o, s_out) of fwd, whose other
    arguments it takes; s_in and s_out are states of turned keys, so a next
    piece of the sequence goes on with the next positions."""
    q, k = _turned(q, k, freqs, positions, start, layout, fwd_arguments.get("stream"))
    return fwd(q, k, v, log_decay, **fwd_arguments)


def retention_bwd(q, k, v, log_decay, do, freqs, positions=None, start: int = 0, layout: str = "half",
                  **bwd_arguments) -> dict:
    """Gradients of retention(...): those of bwd at the turned q and k, turned
    back.  Other arguments as bwd.  bfloat16 gradients of q and k are rounded
    before they are turned and again after (float32 ones, the default, once
    each at 2^-24); keys that heads share are turned for each of them."""
    stream = bwd_arguments.get("stream")
    q, k = _turned(q, k, freqs, positions, start, layout, stream)
    g = bwd(q, k, v, log_decay, do, **bwd_arguments)
    rope(g["q"], g["k"], freqs, positions, start, layout, inverse=True, q_out=g["q"], k_out=g["k"], stream=stream)
    return g


# ---------------------------------------------------------------- norm
def _rows(x, weight):
    if x.dim() < 1 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor [..., C]")
    C = x.shape[-1]
    rows = x.shape[0] if x.dim() == 2 else x.numel() // C if C else 0
    return rows, C, _dtype(x, "x"), x.device, _flat(weight, "weight", (C,), torch.float32, x.device)


def _residual(x, residual, h):
    if residual is None:
        if h is not None:
            raise ValueError("h without a residual")
        return x, 0, 0
    pr = _flat(residual, "residual", x.shape, x.dtype, x.device)
    if h is None:
        h = torch.empty_like(x)
        return h, pr, h.data_ptr()
    return h, pr, _flat(h, "h", x.shape, x.dtype, x.device)


def rms_norm(x, weight, eps: float = 1e-6, residual=None, h=None, out=None, stream=None):
    """(y, h): h = x + residual (rounded to x's type; x itself without one),
    y = h / sqrt(mean(h^2) + eps) * weight over the last dimension.

    x, residual: [..., C] float32 or bfloat16, contiguous; weight: float32 [C].
    `h` may be x or residual (in place)."""
    rows, C, dtype, dev, pw = _rows(x, weight)
    h, pr, ph = _residual(x, residual, h)
    if out is None:
        out = torch.empty_like(x)
        py = out.data_ptr()
    else:
        py = _flat(out, "out", x.shape, x.dtype, dev)
    _call("linattn_rms_norm", lib().linattn_rms_norm, dev, stream, rows, C, x.data_ptr(), pr, pw, eps, ph, py, dtype)
    return out, h


def rms_norm_q8(x, weight, eps: float = 1e-6, residual=None, group: int = 128, h=None, codes=None, scales=None,
                stream=None):
    """(codes, scales, h): rms_norm with y as float8_e4m3fn codes times float32
    scales, one scale for each 128 columns (group 128: scales [..., ceil(C /
    128)]) or for the row (group 0: scales [..., 1])."""
    rows, C, dtype, dev, pw = _rows(x, weight)
    if group not in (0, 128):
        raise ValueError("group must be 0 or 128")
    h, pr, ph = _residual(x, residual, h)
    if codes is None:
        codes = torch.empty_like(x, dtype=torch.float8_e4m3fn)
        pc = codes.data_ptr()
    else:
        pc = _flat(codes, "codes", x.shape, torch.float8_e4m3fn, dev)
    shape = (*x.shape[:-1], (C + 127) // 128 if group else 1)
    if scales is None:
        scales = torch.empty(shape, dtype=torch.float32, device=dev)
        ps = scales.data_ptr()
    else:
        ps = _flat(scales, "scales", shape, torch.float32, dev)
    _call("linattn_rms_norm_q8", lib().linattn_rms_norm_q8, dev, stream, rows, C, x.data_ptr(), pr, pw, eps, ph, pc, ps,
          group, dtype)
    return codes, scales, h


def rms_norm_bwd(dy, h, weight, eps: float = 1e-6, dh=None, out=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(y * dy) + sum(h * dh) for (y, h) = rms_norm(...):
    {"x": with respect to h, and so to x and residual alike, "weight": [C]}.
    `out`: where "x" goes (dy or dh itself is fine)."""
    rows, C, dtype, dev, pw = _rows(h, weight)
    pdy = _flat(dy, "dy", h.shape, h.dtype, dev)
    pdh = _flat(dh, "dh", h.shape, h.dtype, dev)
    if dy is None:
        raise ValueError("dy is missing")
    if out is None:
        out = torch.empty_like(h)
        px = out.data_ptr()
    else:
        px = _flat(out, "out", h.shape, h.dtype, dev)
    dweight = torch.empty((C,), dtype=torch.float32, device=dev)
    L = lib()
    pws, nws, keep = _workspace(workspace, lambda: L.linattn_rms_norm_bwd_workspace_bytes(rows, C, dtype), dev, stream)
    _call("linattn_rms_norm_bwd", L.linattn_rms_norm_bwd, dev, stream, rows, C, pdy, h.data_ptr(), pdh, pw, eps, px,
          dweight.data_ptr(), dtype, pws, nws)
    return {"x": out, "weight": dweight}
