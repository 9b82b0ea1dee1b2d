"""float64 CPU reference of the selective state space layer's operators: the
short causal convolution, the selective scan (token by token, and as explicit
sums), the norms between blocks, and their gradients.  Plain numpy; shares
nothing with the GPU path."""
from __future__ import annotations

import numpy as np


def _f64(*xs):
    return [None if x is None else np.asarray(x, np.float64) for x in xs]


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1.0, e) / (1.0 + e)


def act(name, v):
    """Activation None, "silu" or "sigmoid" of v, and its derivative."""
    s = sigmoid(v)
    if name is None:
        return v, np.ones_like(v)
    if name == "sigmoid":
        return s, s * (1 - s)
    return v * s, s * (1 + v * (1 - s))


# ---------------------------------------------------------------- convolution
def _conv_rows(x, s_in, W, n):
    """The state followed by the n tokens that count, [W - 1 + n, D]."""
    first = np.zeros((W - 1, x.shape[1])) if s_in is None else s_in
    return np.concatenate((first, x[:n]))


def conv_ref(x, weight, bias=None, activation="silu", lengths=None, s_in=None):
    """(y, s_out): y_t = act(bias + sum_j weight[:, j] x_{t-W+1+j})."""
    x, w, bias, s_in = _f64(x, weight, bias, s_in)
    (B, T, D), W = x.shape, w.shape[1]
    y, s_out = np.zeros((B, T, D)), np.zeros((B, W - 1, D))
    for b, n in enumerate(_lengths(lengths, B, T)):
        r = _conv_rows(x[b], None if s_in is None else s_in[b], W, n)
        for t in range(n):
            p = (w * r[t:t + W].T).sum(1) + (0 if bias is None else bias)
            y[b, t] = act(activation, p)[0]
        s_out[b] = r[n:]
    return y, s_out


def conv_ref_backward(x, weight, dy, bias=None, activation="silu", lengths=None, s_in=None, ds_out=None):
    """Gradients of sum(y dy) + sum(s_out ds_out): {"x", "weight", "bias", "s_in"}."""
    x, w, dy, bias, s_in, ds_out = _f64(x, weight, dy, bias, s_in, ds_out)
    (B, T, D), W = x.shape, w.shape[1]
    g = {"x": np.zeros((B, T, D)), "weight": np.zeros((D, W)), "bias": np.zeros(D), "s_in": np.zeros((B, W - 1, D))}
    for b, n in enumerate(_lengths(lengths, B, T)):
        r = _conv_rows(x[b], None if s_in is None else s_in[b], W, n)
        dr = np.zeros_like(r)
        if ds_out is not None:
            dr[n:] += ds_out[b]
        for t in range(n):
            p = (w * r[t:t + W].T).sum(1) + (0 if bias is None else bias)
            dp = dy[b, t] * act(activation, p)[1]
            dr[t:t + W] += w.T * dp
            g["weight"] += dp[:, None] * r[t:t + W].T
            g["bias"] += dp
        g["s_in"][b], g["x"][b, :n] = dr[:W - 1], dr[W - 1:]
    return g


# ---------------------------------------------------------------- scan
def step_sizes(dt, dt_bias=None, softplus=True):
    v = np.asarray(dt, np.float64) + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v))) if softplus else v


def _per_channel(m, D):
    """[..., G, N] for each channel: [..., D, N]."""
    return np.repeat(m, D // m.shape[-2], axis=-2)


def scan_states(delta, ux, A, Bm, n, s_in=None):
    """States after 0 to n tokens of one sequence, [n + 1, D, N]: h_t = exp(delta_t A) h_{t-1} + ux_t B_t."""
    D, N = A.shape
    h = np.zeros((n + 1, D, N))
    if s_in is not None:
        h[0] = s_in
    for t in range(n):
        h[t + 1] = np.exp(delta[t, :, None] * A) * h[t] + ux[t, :, None] * _per_channel(Bm[t], D)
    return h


def scan_ref(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, lengths=None, s_in=None):
    """(y, s_out) of the selective scan."""
    x, A, Bm, Cm, D, z, s_in = _f64(x, A, Bm, Cm, D, z, s_in)
    B, T, C = x.shape
    delta = step_sizes(dt, dt_bias, softplus)
    y, s_out = np.zeros((B, T, C)), np.zeros((B, *A.shape))
    for b, n in enumerate(_lengths(lengths, B, T)):
        h = scan_states(delta[b], delta[b] * x[b], A, Bm[b], n, None if s_in is None else s_in[b])
        y[b, :n] = (h[1:] * _per_channel(Cm[b, :n], C)).sum(2)
        if D is not None:
            y[b, :n] += D * x[b, :n]
        if z is not None:
            y[b, :n] *= act("silu", z[b, :n])[0]
        s_out[b] = h[n]
    return y, s_out


def scan_bruteforce(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=True, lengths=None, s_in=None):
    """The same outputs as explicit sums over pairs of tokens."""
    x, A, Bm, Cm, D, z, s_in = _f64(x, A, Bm, Cm, D, z, s_in)
    B, T, C = x.shape
    delta = step_sizes(dt, dt_bias, softplus)
    y = np.zeros((B, T, C))
    for b, n in enumerate(_lengths(lengths, B, T)):
        for d in range(C):
            g = d // (C // Bm.shape[2])
            for t in range(n):
                for i in range(t + 1):
                    w = np.exp(A[d] * delta[b, i + 1:t + 1, d].sum())
                    y[b, t, d] += delta[b, i, d] * x[b, i, d] * float((w * Bm[b, i, g] * Cm[b, t, g]).sum())
                if s_in is not None:
                    y[b, t, d] += float((np.exp(A[d] * delta[b, :t + 1, d].sum()) * s_in[b, d] * Cm[b, t, g]).sum())
                y[b, t, d] += 0 if D is None else D[d] * x[b, t, d]
                if z is not None:
                    y[b, t, d] *= z[b, t, d] / (1 + np.exp(-z[b, t, d]))
    return y


def scan_adjoint(delta, ux, A, rates, Bm, Cm, dm, n, s_in=None, ds_out=None):
    """The adjoint of one sequence's states: sums {"B", "C" (of the groups), "ux" = sum_n g B, "step" = sum_n rates q,
    "A" = sum_t delta q, "s_in", "m" = sum_n C h}, q_t = exp(delta_t A) g_t h_{t-1}."""
    (C, N), G = A.shape, Bm.shape[1]
    h = scan_states(delta, ux, A, Bm, n, s_in)
    T = delta.shape[0]
    o = {"B": np.zeros((T, G, N)), "C": np.zeros((T, G, N)), "ux": np.zeros((T, C)), "step": np.zeros((T, C)),
         "A": np.zeros((C, N)), "m": np.zeros((T, C))}
    g = np.zeros((C, N)) if ds_out is None else np.array(ds_out, np.float64)
    for t in range(n - 1, -1, -1):
        Bt, Ct = _per_channel(Bm[t], C), _per_channel(Cm[t], C)
        g = g + Ct * dm[t, :, None]
        o["m"][t] = (Ct * h[t + 1]).sum(1)
        o["C"][t] = (h[t + 1] * dm[t, :, None]).reshape(G, C // G, N).sum(1)
        o["B"][t] = (g * ux[t, :, None]).reshape(G, C // G, N).sum(1)
        o["ux"][t] = (g * Bt).sum(1)
        g = np.exp(delta[t, :, None] * A) * g
        q = g * h[t]
        o["step"][t] = (q * rates).sum(1)
        o["A"] += q * delta[t, :, None]
    o["s_in"] = g
    return o


def scan_ref_backward(x, dt, A, Bm, Cm, dy, D=None, z=None, dt_bias=None, softplus=True, lengths=None, s_in=None,
                      ds_out=None):
    """Gradients of sum(y dy) + sum(s_out ds_out): {"x", "dt", "A", "B", "C", "D", "z", "dt_bias", "s_in"}."""
    x, A, Bm, Cm, dy, D, z, s_in, ds_out = _f64(x, A, Bm, Cm, dy, D, z, s_in, ds_out)
    B, T, C = x.shape
    v = np.asarray(dt, np.float64) + (0 if dt_bias is None else np.asarray(dt_bias, np.float64))
    delta = step_sizes(dt, dt_bias, softplus)
    skip = np.zeros(C) if D is None else D
    g = {"x": np.zeros_like(x), "dt": np.zeros_like(x), "z": np.zeros_like(x), "B": np.zeros_like(Bm),
         "C": np.zeros_like(Cm), "A": np.zeros_like(A), "D": np.zeros(C), "s_in": np.zeros((B, *A.shape))}
    for b, n in enumerate(_lengths(lengths, B, T)):
        s, ds = act("silu", z[b]) if z is not None else (np.ones((T, C)), np.zeros((T, C)))
        dm = dy[b] * s
        o = scan_adjoint(delta[b], delta[b] * x[b], A, A, Bm[b], Cm[b], dm, n, None if s_in is None else s_in[b],
                         None if ds_out is None else ds_out[b])
        g["z"][b, :n] = (dy[b] * (o["m"] + skip * x[b]) * ds)[:n]
        g["x"][b, :n] = (delta[b] * o["ux"] + skip * dm)[:n]
        ddt = x[b] * o["ux"] + o["step"]
        g["dt"][b, :n] = (ddt * sigmoid(v[b]) if softplus else ddt)[:n]
        g["D"] += (dm * x[b])[:n].sum(0)
        g["B"][b], g["C"][b], g["s_in"][b] = o["B"], o["C"], o["s_in"]
        g["A"] += o["A"]
    g["dt_bias"] = g["dt"].sum((0, 1))
    return g


# ---------------------------------------------------------------- norms between blocks
def unit(x, eps):
    """x / rms(x), and 1 / rms(x)."""
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return x * r, r


def _rows_of(gate, rows):
    return np.repeat(gate, rows // gate.shape[0], axis=0)


def block_h_ref(x, residual=None, gate=None, post=None, scale=1.0, activation=None, eps=1e-6):
    """h before it is rounded, [rows, C]; gate: [gates, C]."""
    x, residual, gate, post = _f64(x, residual, gate, post)
    h = x if post is None else unit(x, eps)[0] * post
    if gate is not None:
        h = h * _rows_of(act(activation, gate)[0], x.shape[0])
    h = scale * h
    return h if residual is None else residual + h


def block_norm_ref(h, pre, eps=1e-6):
    h, pre = _f64(h, pre)
    return unit(h, eps)[0] * pre


def _unit_back(d, x, eps):
    """The gradient through x -> x / rms(x)."""
    n, r = unit(x, eps)
    return r * (d - n * np.mean(d * n, -1, keepdims=True))


def block_norm_ref_backward(x, h, dy=None, dh=None, gate=None, post=None, pre=None, scale=1.0, activation=None, eps=1e-6):
    """{"x", "residual", "gate", "post_weight", "pre_weight"}; rows are the first dimension's."""
    x, h, dy, dh, gate, post, pre = _f64(x, h, dy, dh, gate, post, pre)
    g = {}
    total = np.zeros_like(x) if dh is None else dh.copy()
    if pre is not None:
        g["pre_weight"] = (dy * unit(h, eps)[0]).sum(0)
        total = total + _unit_back(dy * pre, h, eps)
    g["residual"] = total
    n = x if post is None else unit(x, eps)[0] * post
    d = scale * total
    if gate is not None:
        a, s = act(activation, gate)
        rows = x.shape[0] // gate.shape[0]
        g["gate"] = (d * n).reshape(gate.shape[0], rows, -1).sum(1) * s
        d = d * _rows_of(a, x.shape[0])
    if post is not None:
        g["post_weight"] = (d * unit(x, eps)[0]).sum(0)
        d = _unit_back(d * post, x, eps)
    g["x"] = d
    return g
