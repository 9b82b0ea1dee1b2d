"""Inputs and bounds shared by the GPU tests of the linear-attention operators.

How far a result may be from the oracle's, derived from the arithmetic.  u =
2^-24 is half a step of float32, b = 2^-8 of bfloat16.  A is the same result
computed from absolute values: what the magnitudes of all terms add up to.

* Every operand carried whole is off by at most u of itself (three bfloat16
  parts of 2^-8 each), the dropped products of low parts by 2 u: 4 u of each
  term.  Each factor exp(g n) has an exponent that is off by 2 u of itself and
  a result by 2 u; a term whose exponent is x weighs e^-x, and x e^-x < 1.
* Sums: a matrix instruction adds 32 products to its accumulator at a time;
  6 part products make up to 6 (K + 64) / 32 such steps for a chunk, and the
  state takes one decay and 12 steps for each chunk of T / 64.  Each step errs
  by at most 2 u of its partial sum <= A (twice, for an instruction that cuts
  off instead of rounding), and its internal additions by at most 5 levels of
  the same.
  steps(T, K) = (6 (K + 64) / 32 + 13 T / 64) * 6, error <= (16 + 2 steps) u A.
* A bfloat16 output rounds once: b |o|; what arises in between is rounded once
  to bfloat16 in either product: b A; the state's update on two parts: b^2 A.
* All of these are worst cases.  Errors of many terms are independent: the
  error's 2-norm over that of the result stays under 1e-6 for float32 (a
  hundred roundings add up to ten of u = 6e-8, with cancellation of up to
  twice), and under sqrt(3) * 2^-8 / sqrt(3) = b for bfloat16, whose single
  roundings have a standard deviation of b / sqrt(3) at most.
"""
import numpy as np
import torch

U, BF = 2.0 ** -24, 2.0 ** -8
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print(*a, flush=True)


def normal(gen, *shape, std=0.5, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


def generator(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def f64(t):
    return t.detach().double().cpu().numpy()


def steps(T, K):
    return (6 * (K + 64) / 32 + 13 * T / 64) * 6


def check(name, got, ref, size, T, K, bf16):
    """got (a tensor) against ref with the bounds above; size: A."""
    x = f64(got)
    assert np.array_equal(np.isfinite(x), np.isfinite(ref)), f"{name}: not finite in other places"
    err = np.abs(x - ref)
    bound = (16 + 2 * steps(T, K)) * U * size + 1e-37
    if bf16:
        bound = bound + BF * np.abs(ref) + (BF + BF * BF) * size
    worst = float(np.max(err / bound)) if err.size else 0.0
    norm = float(np.linalg.norm(ref))
    rel = float(np.linalg.norm(err)) / norm if norm else float(np.linalg.norm(err))
    say(f"[linattn] {name}: {worst:.3g} of the bound, rel {rel:.3g}")
    assert worst <= 1.0, f"{name}: error {worst:.3g} times the bound"
    assert rel <= (BF if bf16 else 1e-6), f"{name}: relative error {rel:.3g}"


def bits(a, b):
    return a.shape == b.shape and torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
