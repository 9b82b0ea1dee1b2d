"""ctypes binding of the selective state space layer's operators (C ABI in
include/ssm.h, in libwkv6.so).

Argument marshalling only, as in ``linear_attention_rnn_amd.linattn``: every
computation runs in the library's HIP kernels, PyTorch provides device memory
and the current HIP stream, and there is no fallback.  Calls run on the inputs'
GPU whichever device is current.  Workspaces, streams and graphs are as in
``linattn``: gradients on torch's current stream take their workspace from torch's
allocator and can be captured; calls with a ``stream`` of their own take it
from the library's pool, or are given a ``workspace``, a uint8 tensor of at
least ``*_workspace_bytes`` bytes, to be recorded.
"""
from __future__ import annotations

import ctypes

import torch

from . import linattn, wkv6
from .linattn import _DTYPES, _call, _dtype, _flat, _workspace

MAX_STATES = 64         # SSM_MAX_STATES
MAX_WINDOW = 4          # SSM_MAX_WINDOW
MAX_COLUMNS = 16384     # SSM_MAX_COLUMNS
_ACTIVATIONS = {None: 0, "silu": 1, "sigmoid": 2}

SsmError = linattn.LinattnError   # a call's name, status and the library's text

_fns = None


def lib() -> ctypes.CDLL:
    """The library, with the argument types of ssm.h set (once)."""
    global _fns
    L = wkv6.lib()
    if _fns is not L:
        i64, vp, i32, f32, sz = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        tail = [vp, sz, vp]   # workspace, its bytes, stream
        L.ssm_conv_fwd.argtypes = [i64] * 4 + [vp] * 3 + [i32] + [vp] * 5 + [i32, vp]
        L.ssm_conv_bwd.argtypes = [i64] * 4 + [vp] * 3 + [i32] + [vp] * 9 + [i32] + tail
        L.ssm_scan_fwd.argtypes = [i64] * 5 + [vp] * 8 + [i32] + [vp] * 5 + [i32, vp]
        L.ssm_scan_bwd.argtypes = [i64] * 5 + [vp] * 8 + [i32] + [vp] * 14 + [i32] + tail
        L.ssm_block_norm.argtypes = [i64, i64, vp, vp, vp, i64, vp, vp, f32, i32, f32, vp, vp, i32, vp]
        L.ssm_block_norm_bwd.argtypes = [i64, i64, vp, vp, vp, i64, vp, vp, f32, i32, f32] + [vp] * 7 + [i32] + tail
        L.ssm_abi_version.argtypes = []
        for f in (L.ssm_conv_fwd, L.ssm_conv_bwd, L.ssm_scan_fwd, L.ssm_scan_bwd, L.ssm_block_norm,
                  L.ssm_block_norm_bwd, L.ssm_abi_version):
            f.restype = i32
        L.ssm_conv_bwd_workspace_bytes.argtypes = [i64] * 4 + [i32]
        L.ssm_scan_bwd_workspace_bytes.argtypes = [i64] * 5 + [i32]
        L.ssm_block_norm_bwd_workspace_bytes.argtypes = [i64] * 3 + [i32] * 4
        for f in (L.ssm_conv_bwd_workspace_bytes, L.ssm_scan_bwd_workspace_bytes, L.ssm_block_norm_bwd_workspace_bytes):
            f.restype = sz
        _fns = L
    return L


def abi_version() -> int:
    return lib().ssm_abi_version()


def conv_bwd_workspace_bytes(B, T, D, W, dtype=torch.bfloat16) -> int:
    """Workspace bytes of a conv_bwd call of these sizes (host arithmetic)."""
    return lib().ssm_conv_bwd_workspace_bytes(B, T, D, W, _DTYPES[dtype])


def scan_bwd_workspace_bytes(B, T, D, N, G=1, dtype=torch.bfloat16) -> int:
    """Workspace bytes of a scan_bwd call of these sizes (host arithmetic)."""
    return lib().ssm_scan_bwd_workspace_bytes(B, T, D, N, G, _DTYPES[dtype])


def block_norm_bwd_workspace_bytes(rows, C, gate_rows=1, post=True, gate=True, pre=True, dtype=torch.bfloat16) -> int:
    """Workspace bytes of a block_norm_bwd call of these sizes (host arithmetic)."""
    return lib().ssm_block_norm_bwd_workspace_bytes(rows, C, gate_rows, post, gate, pre, _DTYPES[dtype])


# ---------------------------------------------------------------- checks
def _first(x):
    """Shape, type and GPU of a call's first tensor, [B, T, D]."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, D]")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    return x.shape, x.dtype, x.device, _dtype(x, "x")


def _rows(t, name, shape, dtype, device):
    """A tensor with adjacent last places on the call's GPU; returns its address."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on the GPU of x, {device}")
    if not t.is_contiguous() and t.stride(-1) != 1 and shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be adjacent")
    return t.data_ptr()


def _table(t, name, shape, device):
    return _flat(t, name, shape, torch.float32, device)


def _strides(n, *tensors):
    """The first n distances of each (0 for those it lacks), or None if all are
    contiguous."""
    for t in tensors:
        if t is not None and not t.is_contiguous():
            break
    else:
        return None
    out = []
    for t in tensors:
        s = t.stride()[:-1] if t is not None else ()
        out += s + (0,) * (n - len(s))
    return (ctypes.c_int64 * len(out))(*out)


def _new(t, name, shape, dtype, device):
    """(t, its address), a new tensor for None."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        return t, t.data_ptr()
    return t, _rows(t, name, shape, dtype, device)


def _state_out(s_out, s_in, ps, want, shape, dtype, device):
    if s_out is not None:
        return s_out, ps if s_out is s_in else _flat(s_out, "s_out", shape, dtype, device)
    if want:
        s_out = torch.empty(shape, dtype=dtype, device=device)
        return s_out, s_out.data_ptr()
    return None, 0


def _activation(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {list(allowed)}")
    return _ACTIVATIONS[name]


def _lengths(lengths, B, device):
    return _flat(lengths, "lengths", (B,), torch.int32, device)


# ---------------------------------------------------------------- convolution
def _window(weight, bias, D, device):
    if weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    return W, _table(weight, "weight", (D, W), device), _table(bias, "bias", (D,), device)


def conv(x, weight, bias=None, activation="silu", lengths=None, s_in=None, want_state: bool = False, out=None,
         s_out=None, stream=None):
    """Short causal convolution of each channel: (y, s_out).

    y_t[d] = act(bias[d] + sum_j weight[d, j] x_{t-W+1+j}[d]), act "silu" or None.

    x: [B, T, D], float32 or bfloat16, any distances between batch items and
    tokens (channels adjacent); weight: float32 [D, W], W from 2 to 4; bias: None
    or float32 [D]; lengths: None or int32 [B] (padded batch: rows behind a
    sequence are not read, their outputs are zero); s_in: None (zero) or [B, W - 1,
    D] of x's type, the rows before the first token.  y is `out`, or a new tensor.
    The last W - 1 rows go to `s_out` (which may be s_in), or to a new tensor if
    `want_state`; otherwise None is returned for them.
    """
    (B, T, D), t, dev, dtype = _first(x)
    act = _activation(activation, (None, "silu"))
    px, pl = _rows(x, "x", x.shape, t, dev), _lengths(lengths, B, dev)
    W, pw, pb = _window(weight, bias, D, dev)
    out, py = _new(out, "out", x.shape, t, dev)
    state = (B, W - 1, D)
    ps = _flat(s_in, "s_in", state, t, dev)
    s_out, po = _state_out(s_out, s_in, ps, want_state, state, t, dev)
    L = lib()
    _call("ssm_conv_fwd", L.ssm_conv_fwd, dev, stream, B, T, D, W, px, pw, pb, act, pl, ps, py, po,
          _strides(2, x, out), dtype)
    return out, s_out


def conv_bwd(x, weight, dy, bias=None, activation="silu", lengths=None, s_in=None, ds_out=None,
             want_ds_in: bool = False, out=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(y * dy) + sum(s_out * ds_out) for (y, s_out) = conv(...).

    dy: [B, T, D] of x's type; ds_out: None or [B, W - 1, D] of it.  Returns {"x",
    "weight", "bias" (with a bias)}, and "s_in" if `want_ds_in`; "x" is written
    to `out` if that is given.
    """
    (B, T, D), t, dev, dtype = _first(x)
    act = _activation(activation, (None, "silu"))
    px, pdy, pl = _rows(x, "x", x.shape, t, dev), _rows(dy, "dy", x.shape, t, dev), _lengths(lengths, B, dev)
    W, pw, pb = _window(weight, bias, D, dev)
    state = (B, W - 1, D)
    ps, pd = _flat(s_in, "s_in", state, t, dev), _flat(ds_out, "ds_out", state, t, dev)
    g = {}
    g["x"], pdx = _new(out, "out", x.shape, t, dev)
    g["weight"] = torch.empty((D, W), dtype=torch.float32, device=dev)
    pdb = pdi = 0
    if bias is not None:
        g["bias"] = torch.empty((D,), dtype=torch.float32, device=dev)
        pdb = g["bias"].data_ptr()
    if want_ds_in:
        g["s_in"] = torch.empty(state, dtype=t, device=dev)
        pdi = g["s_in"].data_ptr()
    L = lib()
    pws, nws, keep = _workspace(workspace, lambda: L.ssm_conv_bwd_workspace_bytes(B, T, D, W, dtype), dev, stream)
    _call("ssm_conv_bwd", L.ssm_conv_bwd, dev, stream, B, T, D, W, px, pw, pb, act, pl, ps, pdy, pd, pdx,
          g["weight"].data_ptr(), pdb, pdi, _strides(2, x, dy, g["x"]), dtype, pws, nws)
    return g


# ---------------------------------------------------------------- scan
def _scan(x, dt, A, B, C, D, z, dt_bias, lengths):
    """Sizes, type, GPU and addresses of what scan and scan_bwd have in common."""
    (b, T, d), t, dev, dtype = _first(x)
    if B.dim() != 4 or A.dim() != 2:
        raise ValueError("B and C must be [B, T, G, N] and A [D, N]")
    G, N = B.shape[2:]
    groups = (b, T, G, N)
    return ((b, T, d, N, G), groups, t, dev, dtype,
            (_rows(x, "x", x.shape, t, dev), _rows(dt, "dt", x.shape, t, dev), _table(A, "A", (d, N), dev),
             _rows(B, "B", groups, t, dev), _rows(C, "C", groups, t, dev), _table(D, "D", (d,), dev),
             0 if z is None else _rows(z, "z", x.shape, t, dev), _table(dt_bias, "dt_bias", (d,), dev)),
            _lengths(lengths, b, dev))


def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, lengths=None, s_in=None,
         want_state: bool = False, out=None, s_out=None, stream=None):
    """Selective scan of each channel d over N states: (y, s_out).

    delta_t = softplus(dt_t + dt_bias)  (or the sum itself),
    h_t[n] = exp(delta_t A[d, n]) h_{t-1}[n] + delta_t x_t B_t[g, n] from s_in (or zero),
    y_t = (sum_n C_t[g, n] h_t[n] + D[d] x_t) * silu(z_t), with d's group g = d // (channels / G).

    x, dt, z: [B, T, channels], float32 or bfloat16, any distances between batch
    items and tokens; B, C: [B, T, G, N] of x's type, any distances but between
    states; A: float32 [channels, N], negative; D, dt_bias: None or float32
    [channels]; z: None (no gate); lengths: None or int32 [B] (padded batch: rows
    behind a sequence are not read, their outputs are zero); s_in: None or float32
    [B, channels, N].  channels / G and N are multiples of 8, N up to 64.  y is
    `out`, or a new tensor.  The state after the last token goes to `s_out` (which
    may be s_in), or to a new tensor if `want_state`; otherwise None is returned
    for it.
    """
    (b, T, d, N, G), _, t, dev, dtype, p, pl = _scan(x, dt, A, B, C, D, z, dt_bias, lengths)
    out, py = _new(out, "out", x.shape, t, dev)
    ps = _table(s_in, "s_in", (b, d, N), dev)
    s_out, po = _state_out(s_out, s_in, ps, want_state, (b, d, N), torch.float32, dev)
    L = lib()
    _call("ssm_scan_fwd", L.ssm_scan_fwd, dev, stream, b, T, d, N, G, *p, softplus, pl, ps, py, po,
          _strides(3, x, dt, B, C, z, out), dtype)
    return out, s_out


def scan_bwd(x, dt, A, B, C, dy, D=None, z=None, dt_bias=None, softplus: bool = True, lengths=None, s_in=None,
             ds_out=None, want_ds_in: bool = False, out=None, workspace=None, stream=None) -> dict:
    """Gradients of sum(y * dy) + sum(s_out * ds_out) for (y, s_out) = scan(...).

    dy: [B, T, channels] of x's type; ds_out: None or float32 [B, channels, N].
    Returns {"x", "dt", "A", "B", "C"}, "D", "z" and "dt_bias" where those are
    given, and "s_in" if `want_ds_in`.  `out`: a dict of tensors to write "x",
    "dt", "B", "C", "z" and "s_in" to instead of new ones (None: a new one; slices
    of one buffer are fine; "s_in" may be ds_out).  Expanded inputs get the gradient of every
    place they are used at: the caller sums them.
    """
    (b, T, d, N, G), groups, t, dev, dtype, p, pl = _scan(x, dt, A, B, C, D, z, dt_bias, lengths)
    pdy = _rows(dy, "dy", x.shape, t, dev)
    state = (b, d, N)
    ps, pd = _table(s_in, "s_in", state, dev), _table(ds_out, "ds_out", state, dev)
    g, q = {n: t for n, t in out.items() if t is not None} if out else {}, {}
    for name, shape in (("x", x.shape), ("dt", x.shape), ("B", groups), ("C", groups), ("z", x.shape)):
        if name == "z" and z is None:
            if "z" in g:
                raise ValueError("an output for the gradient of z without z")
            q[name] = 0
        else:
            g[name], q[name] = _new(g.get(name), "d" + name, shape, t, dev)
    if out and not out.keys() <= {"x", "dt", "B", "C", "z", "s_in", "A", "D", "dt_bias"}:
        raise ValueError("an output of a name that no gradient has")
    for name, shape, given in (("A", (d, N), True), ("D", (d,), D is not None), ("dt_bias", (d,), dt_bias is not None)):
        if name in g:
            raise ValueError(f"the gradient of {name} is a new tensor")
        q[name] = 0
        if given:
            g[name] = torch.empty(shape, dtype=torch.float32, device=dev)
            q[name] = g[name].data_ptr()
    if want_ds_in and "s_in" not in g:
        g["s_in"] = torch.empty(state, dtype=torch.float32, device=dev)
    pi = _table(g.get("s_in"), "ds_in", state, dev)
    L = lib()
    pws, nws, keep = _workspace(workspace, lambda: L.ssm_scan_bwd_workspace_bytes(b, T, d, N, G, dtype), dev, stream)
    _call("ssm_scan_bwd", L.ssm_scan_bwd, dev, stream, b, T, d, N, G, *p, softplus, pl, ps, pdy, pd, q["x"], q["dt"],
          q["A"], q["B"], q["C"], q["D"], q["z"], q["dt_bias"], pi,
          _strides(3, x, dt, B, C, z, dy, g["x"], g["dt"], g["B"], g["C"], g.get("z")), dtype, pws, nws)
    return g


# ---------------------------------------------------------------- norms between blocks
def _leading(gate, x, rows):
    """Refuses a gate that broadcasting would repeat over other rows of x than those
    that follow each other: leading dimensions of x, then ones, or as many rows in a row."""
    for i in range(len(x) + 1):
        if gate == x[:i] + (1,) * (len(x) - i) if len(gate) == len(x) else rows == x[:i].numel():
            return
    raise ValueError("gate must have leading dimensions of x, and ones behind them")


def _block(x, gate, post_weight, pre_weight, activation):
    """Sizes, type, GPU and addresses of what block_norm and its gradients have in
    common; also how many rows share a gate."""
    if x.dim() < 1 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous GPU tensor [..., C]")
    C, dev, dtype = x.shape[-1], x.device, _dtype(x, "x")
    rows = x.numel() // C if C else 0
    act = _activation(activation, tuple(_ACTIVATIONS))
    pg, per = 0, 1
    if gate is not None:
        if gate.dim() < 1 or gate.shape[-1] != C:
            raise ValueError("gate must be [..., C]")
        pg = _flat(gate, "gate", gate.shape, x.dtype, dev)
        gates = gate.numel() // C if C else 0
        if gates:
            per, left = divmod(rows, gates)
            if left or (rows and not per):
                raise ValueError("the rows of gate must divide those of x")
            per = max(per, 1)
            if x.dim() > 2 and gate.shape != x.shape:
                _leading(gate.shape[:-1], x.shape[:-1], gates)
        elif rows:
            raise ValueError("gate has no rows")
    elif act:
        raise ValueError("an activation without a gate")
    return (rows, C, per, act, dtype, dev, pg, _flat(post_weight, "post_weight", (C,), torch.float32, dev),
            _flat(pre_weight, "pre_weight", (C,), torch.float32, dev))


def block_norm(x, residual=None, gate=None, post_weight=None, pre_weight=None, scale: float = 1.0, activation=None,
               eps: float = 1e-6, h=None, out=None, stream=None):
    """(y, h): what happens between two blocks, with n = x / sqrt(mean(x^2) + eps)
    * post_weight (x itself without one) over the last dimension,

    h = residual + scale * act(gate) * n  (rounded to x's type; a missing residual is 0, a missing gate 1),
    y = h / sqrt(mean(h^2) + eps) * pre_weight  (None without pre_weight).

    x, residual: [..., C] float32 or bfloat16, contiguous; gate: [..., C] of x's
    type, contiguous: one row for each row of x, or for each so many rows of x
    that follow each other ([B, 1, C] or [B, C] for x of [B, T, C]), or for all;
    activation: None, "silu" or "sigmoid", of the gate; post_weight, pre_weight:
    None or float32 [C].  `h` may be x or residual (in place).
    """
    rows, C, per, act, dtype, dev, pg, pp, pq = _block(x, gate, post_weight, pre_weight, activation)
    pr = _flat(residual, "residual", x.shape, x.dtype, dev)
    if h is None:
        h = torch.empty_like(x)
    ph, py = _flat(h, "h", x.shape, x.dtype, dev), 0
    if pre_weight is not None:
        if out is None:
            out = torch.empty_like(x)
        py = _flat(out, "out", x.shape, x.dtype, dev)
    elif out is not None:
        raise ValueError("out without pre_weight")
    _call("ssm_block_norm", lib().ssm_block_norm, dev, stream, rows, C, x.data_ptr(), pr, pg, per, pp, pq, scale, act,
          eps, ph, py, dtype)
    return out, h


def block_norm_bwd(x, h, dy=None, dh=None, gate=None, post_weight=None, pre_weight=None, scale: float = 1.0,
                   activation=None, eps: float = 1e-6, want_residual: bool = True, out=None, residual_out=None,
                   workspace=None, stream=None) -> dict:
    """Gradients of sum(y * dy) + sum(h * dh) for (y, h) = block_norm(...): {"x"},
    "residual" unless `want_residual` is false, and "gate", "post_weight" and
    "pre_weight" where those are given.

    h: of the forward call (None without pre_weight); dy: given exactly where
    pre_weight is.  `out`: where "x" goes (dy itself is fine), `residual_out`:
    where "residual" goes (dh itself is fine).  Gates and weights that no row uses
    have gradients of zero.
    """
    rows, C, per, act, dtype, dev, pg, pp, pq = _block(x, gate, post_weight, pre_weight, activation)
    if (dy is None) != (pre_weight is None):
        raise ValueError("dy and pre_weight are both given or both None")
    if h is None and pre_weight is not None:
        raise ValueError("h is missing")
    ph, pdy, pdh = (_flat(t, n, x.shape, x.dtype, dev) for t, n in ((h, "h"), (dy, "dy"), (dh, "dh")))
    g = {"x": torch.empty_like(x) if out is None else out}
    if residual_out is not None or want_residual:
        g["residual"] = torch.empty_like(x) if residual_out is None else residual_out
    if gate is not None:
        # (no rows: no kernel writes it)
        g["gate"] = torch.empty_like(gate) if rows else torch.zeros_like(gate)
    for name, w in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if w is not None:
            g[name] = torch.empty((C,), dtype=torch.float32, device=dev)
    at = {n: t.data_ptr() for n, t in g.items()}
    _flat(g["x"], "out", x.shape, x.dtype, dev)
    _flat(g.get("residual"), "residual_out", x.shape, x.dtype, dev)
    L = lib()
    pws, nws, keep = _workspace(workspace, lambda: L.ssm_block_norm_bwd_workspace_bytes(
        rows, C, per, pp != 0, pg != 0, pq != 0, dtype), dev, stream)
    _call("ssm_block_norm_bwd", L.ssm_block_norm_bwd, dev, stream, rows, C, x.data_ptr(), ph, pg, per, pp, pq, scale, act,
          eps, pdy, pdh, at["x"], at.get("residual", 0), at.get("gate", 0), at.get("post_weight", 0),
          at.get("pre_weight", 0), dtype, pws, nws)
    return g
