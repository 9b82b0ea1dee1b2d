"""float64 CPU reference of the linear-attention layer's operators: attention
with one decay per head (token by token, and as explicit sums), its gradients,
rotary positions, and the root-mean-square norm with its 8-bit output and
gradients.  Plain numpy; shares nothing with the GPU path."""
from __future__ import annotations

import numpy as np


def _lengths(lengths, B, T):
    return [T] * B if lengths is None else [min(max(int(n), 0), T) for n in lengths]


def linattn_ref(q, k, v, log_decay, scale=1.0, lengths=None, s_in=None):
    """(o, s_out): S_t = a S_{t-1} + k_t^T v_t, o_t = scale q_t S_t, [B, T, H, *]."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, T, H, K = q.shape
    V = v.shape[3]
    a = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    o = np.zeros((B, T, H, V))
    S = np.zeros((B, H, K, V)) if s_in is None else np.array(s_in, np.float64)
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            S[b] = a * S[b] + k[b, t, :, :, None] * v[b, t, :, None, :]
            o[b, t] = scale * np.matmul(q[b, t, :, None, :], S[b])[:, 0]
    return o, S


def linattn_bruteforce(q, k, v, log_decay, scale=1.0, lengths=None, s_in=None):
    """The same outputs as explicit sums over pairs of tokens."""
    B, T, H, K = q.shape
    o = np.zeros((B, T, H, v.shape[3]))
    for b, n in enumerate(_lengths(lengths, B, T)):
        for h in range(H):
            for t in range(n):
                for i in range(t + 1):
                    w = float(log_decay[h]) * (t - i) if t > i else 0.0
                    o[b, t, h] += scale * np.exp(w) * float(np.dot(q[b, t, h], k[b, i, h])) * v[b, i, h]
                if s_in is not None:
                    o[b, t, h] += scale * np.exp(float(log_decay[h]) * (t + 1)) * (q[b, t, h] @ s_in[b, h])
    return o


def linattn_ref_backward(q, k, v, log_decay, do, scale=1.0, lengths=None, s_in=None, ds_out=None):
    """Gradients of sum(o do) + sum(s_out ds_out): {"q", "k", "v", "s_in"}."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    B, T, H, K = q.shape
    V = v.shape[3]
    a = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    g = {"q": np.zeros_like(q), "k": np.zeros_like(k), "v": np.zeros_like(v),
         "s_in": np.zeros((B, H, K, V)) if ds_out is None else np.array(ds_out, np.float64)}
    S = np.zeros((B, H, K, V)) if s_in is None else np.array(s_in, np.float64)
    for b, n in enumerate(_lengths(lengths, B, T)):
        for t in range(n):
            S[b] = a * S[b] + k[b, t, :, :, None] * v[b, t, :, None, :]
            g["q"][b, t] = scale * np.matmul(S[b], do[b, t, :, :, None])[..., 0]
        D = g["s_in"][b]
        for t in range(n - 1, -1, -1):
            D = D + scale * q[b, t, :, :, None] * do[b, t, :, None, :]
            g["k"][b, t] = np.matmul(D, v[b, t, :, :, None])[..., 0]
            g["v"][b, t] = np.matmul(k[b, t, :, None, :], D)[:, 0]
            D = a * D
        g["s_in"][b] = D
    return g


# 1 / (2 pi) in units of 2^-256, from the first hundred decimals of pi
_INVERSE_TURN = (10 ** 100 << 256) // (2 * int(
    "3" "1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679"))


def rope_angles(positions, freqs):
    """positions x freqs, less whole turns: radians in [0, 2 pi), [*, R / 2].  Products of whole positions and float64
    frequencies are whole numbers of some 2^-n, multiplied by 1 / (2 pi) as such: exact to 2^-48 at any position."""
    m, e = np.frexp(np.asarray(freqs, np.float64))
    whole = np.ldexp(m, 53).astype(np.int64).astype(object)
    turns = np.asarray(positions).astype(np.int64).astype(object)[..., None] * (whole * _INVERSE_TURN)
    part = np.mod(turns >> (256 - 64 + 53 - e.astype(np.int64)).astype(object), 1 << 64)
    return part.astype(np.float64) * (2 * np.pi / 2.0 ** 64)


def rope_ref(x, positions, freqs, layout="half", inverse=False):
    """x: [B, T, H, D]; positions: [B, T] whole numbers; freqs: [R / 2].  Far
    positions are exact."""
    x = np.array(x, np.float64)
    R = 2 * len(freqs)
    angle = rope_angles(positions, freqs)
    c, s = np.cos(angle)[:, :, None], np.sin(angle)[:, :, None]
    if inverse:
        s = -s
    i, j = (slice(0, R, 2), slice(1, R, 2)) if layout == "interleaved" else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = a * c - b * s, a * s + b * c
    return x


def rms_norm_ref(h, weight, eps):
    h = np.asarray(h, np.float64)
    return h / np.sqrt(np.mean(h * h, -1, keepdims=True) + eps) * np.asarray(weight, np.float64)


def rms_norm_ref_backward(dy, h, weight, eps, dh=None):
    """{"x", "weight"}: rows are the last dimension's."""
    dy, h, w = (np.asarray(x, np.float64) for x in (dy, h, weight))
    rms = np.sqrt(np.mean(h * h, -1, keepdims=True) + eps)
    n, dn = h / rms, dy * w
    dx = (dn - n * np.mean(dn * n, -1, keepdims=True)) / rms
    return {"x": dx if dh is None else dx + np.asarray(dh, np.float64),
            "weight": (dy * n).reshape(-1, h.shape[-1]).sum(0)}


# The values of the e4m3 format without infinities: 4 exponent bits of bias 7,
# 3 fraction bits, largest 448.
E4M3 = np.array(sorted({(1 + f / 8) * 2.0 ** (e - 7) for e in range(1, 16) for f in range(8) if (e, f) != (15, 7)}
                       | {f / 8 * 2.0 ** -6 for f in range(8)}))


def e4m3_nearest(x):
    """Each |x| <= 448 rounded to the nearest e4m3 value, ties to the even code."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 1, len(E4M3) - 1)
    lo = hi - 1
    up = (E4M3[hi] - a < a - E4M3[lo]) | ((E4M3[hi] - a == a - E4M3[lo]) & (hi % 2 == 0))
    return np.copysign(np.where(up, E4M3[hi], E4M3[lo]), x)


def scales_ref(y, group):
    """Scales of 8-bit rows: max|y| / 448 over `group` columns (0: the row), at least 2^-126; 1 where all are 0."""
    y = np.asarray(y, np.float64)
    w = group or y.shape[-1]
    tops = [np.abs(y[..., c:c + w]).max(-1) for c in range(0, y.shape[-1], w)]
    s = np.stack(tops, -1) / 448.0
    return np.where(s > 0, np.maximum(s, 2.0 ** -126), 1.0)
