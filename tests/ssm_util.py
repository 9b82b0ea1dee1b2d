"""Inputs and bounds shared by the GPU tests of the selective state space
layer.

How far a result may be from the oracle's, derived from the arithmetic; u =
2^-24 is half a step of float32, b = 2^-8 of bfloat16, and a "size" is the same
result computed from absolute values, what the magnitudes of all terms add up to.

* A step delta is off by at most 18 u of itself: e^-|v| 6 u (product, its
  remainder, exp2 of one unit, fma), the quotient 4 u (sum, reciprocal of one
  unit, product), the series 6 u and two sums.  SiLU and sigmoid: 12 u.
* A decay from token i to t is a product of factors exp(delta A) over at most 8
  tokens of a lane, four doubling steps and one factor for each block of at
  least 32 tokens: (2 (8 + 4 + T / 32) + 8) u of the weight for the factors' own roundings and
  the products, and the exponent X carries (18 + 2) u of itself: X e^-X <= (2 /
  e) e^(-X / 2), so 20 u of 0.74 e^(-X / 2).  Sizes are therefore computed
  with half the rates, where the two are below (44 + T / 16) u of them.
* The state's sums: one addition each in the lane (8), in the steps (4) and for
  each block (T / 32), of 2 u with the input's product; the input is off by 18 +
  2 u.  Sum over states: N u.  All of it: K = 100 + T / 8 + N units of the
  size, doubled for the gradients, which run the same chain back.
* Sums over channels (dB, dC) add chains of at most 8 channels and 8 waves and
  then 64 bits: 16 u more.  Sums over tokens (dA, dD, dt_bias): chains of at most T / 4 + 16.
* A bfloat16 result is rounded once: b of it.
* These are worst cases; roundings are independent, so the 2-norm of the error
  over that of the result stays under 2e-6 for float32 (the square root of some
  hundred roundings of 0.6 u is 4e-7, results of sums with signs are down to a
  fifth of their sizes), and under b for bfloat16.
"""
import numpy as np
import torch

from oracle import ssm_oracle as R
from tests.linattn_util import BF, TYPES, U, bits, f64, generator, normal, say  # noqa: F401


def inputs(seed, B, T, D, N, G, dtype, gate=True, state=True, slow=False):
    """Rates 1 to N and steps of a thousandth to a tenth at rest, as a layer starts with (`slow`: a hundredth of them)."""
    g, t = generator(seed), TYPES[dtype]
    p = {"x": normal(g, B, T, D, dtype=t), "dt": normal(g, B, T, D, std=1.0, dtype=t),
         "A": -(torch.arange(1, N + 1).float() * torch.exp(0.2 * torch.randn(D, N, generator=g))),
         "B": normal(g, B, T, G, N, std=1.0, dtype=t), "C": normal(g, B, T, G, N, std=1.0, dtype=t),
         "D": 1.0 + normal(g, D, std=0.2), "z": normal(g, B, T, D, std=1.0, dtype=t) if gate else None}
    rest = torch.exp(torch.rand(D, generator=g) * 4.6 - 6.9) * (0.01 if slow else 1.0)
    p["dt_bias"] = rest + torch.log(-torch.expm1(-rest))
    p["s_in"] = normal(g, B, D, N, std=1.0) if state else None
    return p


def cuda(p):
    return {n: None if v is None else v.cuda() for n, v in p.items()}


def oracle_args(p):
    q = {n: None if v is None else f64(v) for n, v in p.items()}
    q["Bm"], q["Cm"] = q.pop("B"), q.pop("C")
    return q


def within(name, got, ref, size, units, bf16, rel=2e-6):
    x = f64(got)
    assert x.shape == ref.shape and np.isfinite(x).all(), name
    err = np.abs(x - ref)
    bound = units * U * size + (BF * np.abs(ref) * (1 + units * U) if bf16 else 0) + 1e-37
    worst = float(np.max(err / bound)) if err.size else 0.0
    norm = float(np.linalg.norm(ref))
    e = float(np.linalg.norm(err)) / norm if norm else float(np.linalg.norm(err))
    say(f"[ssm] {name}: {worst:.3g} of the bound, rel {e:.3g}")
    assert worst <= 1.0, f"{name}: error {worst:.3g} times the bound"
    assert e <= (BF if bf16 else rel), f"{name}: relative error {e:.3g}"


def absolute(q):
    """The oracle's inputs for sizes: absolute values, steps as they are, half the rates."""
    return {n: v if v is None or n in ("dt", "dt_bias") else v / 2 if n == "A" else np.abs(v) for n, v in q.items()}


def check_scan(name, p, y, s_out, lengths=None, softplus=True):
    """p: the tensors of a call."""
    q = oracle_args(p)
    y_ref, s_ref = R.scan_ref(**q, softplus=softplus, lengths=lengths)
    a = absolute(q)
    z = a.pop("z")
    y_size, s_size = R.scan_ref(**a, softplus=softplus, lengths=lengths)
    if z is not None:
        y_size = y_size * np.abs(R.act("silu", q["z"])[0])
    K = 100 + y.shape[1] / 8 + q["A"].shape[1]
    bf16 = y.dtype == torch.bfloat16
    within(name + " y", y, y_ref, y_size, K, bf16)
    if s_out is not None:
        within(name + " state", s_out, s_ref, s_size, K, False)


def check_scan_bwd(name, p, g, dy, ds_out=None, lengths=None, softplus=True):
    q = oracle_args(p)
    ref = R.scan_ref_backward(**q, dy=f64(dy), ds_out=None if ds_out is None else f64(ds_out), softplus=softplus,
                              lengths=lengths)
    B, T, C = q["x"].shape
    N = q["A"].shape[1]
    a = absolute(q)
    delta = R.step_sizes(q["dt"], q["dt_bias"], softplus)
    skip = np.zeros(C) if q["D"] is None else a["D"]
    size = {n: np.zeros_like(v) for n, v in ref.items()}
    for b in range(B):
        n = T if lengths is None else min(max(int(lengths[b]), 0), T)
        s, ds = R.act("silu", q["z"][b]) if q["z"] is not None else (np.ones((T, C)), np.zeros((T, C)))
        dm = np.abs(f64(dy)[b] * s)
        o = R.scan_adjoint(delta[b], delta[b] * a["x"][b], a["A"], np.abs(q["A"]), a["Bm"][b], a["Cm"][b],
                           dm, n, None if a["s_in"] is None else a["s_in"][b],
                           None if ds_out is None else np.abs(f64(ds_out)[b]))
        # (1 - s that is nearly 0 is off by u of 1: the derivative by u (1 + |z|))
        size["z"][b, :n] = (np.abs(f64(dy)[b]) * (o["m"] + skip * a["x"][b]) * (np.abs(ds) + 1))[:n]
        size["x"][b, :n] = (delta[b] * o["ux"] + skip * dm)[:n]
        size["dt"][b, :n] = (a["x"][b] * o["ux"] + o["step"])[:n]
        size["D"] += (dm * a["x"][b])[:n].sum(0)
        size["B"][b], size["C"][b], size["s_in"][b] = o["B"], o["C"], o["s_in"]
        size["A"] += o["A"]
    size["dt_bias"] = size["dt"].sum((0, 1))
    bf16 = dy.dtype == torch.bfloat16
    K = 2 * (100 + T / 8 + N) + 32
    for n, v in g.items():
        tokens = n in ("x", "dt", "z", "B", "C")
        within(f"{name} d{n}", v, ref[n], size[n], K + (0 if tokens else T / 4 + 16), bf16 and tokens, 4e-6)
