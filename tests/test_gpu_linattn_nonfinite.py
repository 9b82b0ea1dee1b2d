"""A key, query or gradient that is not finite, or whose products overflow,
reaches the tokens that read it and no others: outputs before it (gradients
behind it, in the sweeps from the last token to the first) keep every bit."""
import pytest
import torch

from tests.linattn_util import TYPES, bits, generator, normal
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu

BAD = {"nan": float("nan"), "inf": float("inf"), "huge": 3e38}


def draw(dtype, T, K, V):
    g = generator(T + K)
    return {n: normal(g, 2, T, 2, d, dtype=TYPES[dtype]).cuda() for n, d in (("q", K), ("k", K), ("v", V), ("do", V))}


@pytest.mark.parametrize("T,at", [(130, 70), (130, 0), (130, 129), (40, 17), (1500, 333)])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 40)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("bad", list(BAD))
def test_keys_and_queries(linattn, T, at, K, V, dtype, out, bad):  # noqa: F811
    x = draw(dtype, T, K, V)
    x["q"], x["k"] = 4 * x["q"], 4 * x["k"]
    decay = torch.tensor([-0.01, -0.3], device="cuda")
    call = lambda y: linattn.fwd(y["q"], y["k"], y["v"], decay, out_dtype=TYPES[out])[0]  # noqa: E731
    want = call(x)
    y = dict(x, k=x["k"].clone())
    y["k"][1, at] = BAD[bad]
    o = call(y)
    assert bits(o[0], want[0]) and bits(o[1, :at], want[1, :at])
    assert not torch.isfinite(o[1, at]).any()
    y = dict(x, q=x["q"].clone())
    y["q"][1, at] = float("nan")
    o = call(y)
    assert bits(o[1, :at], want[1, :at]) and bits(o[1, at + 1:], want[1, at + 1:]) and torch.isnan(o[1, at]).all()


@pytest.mark.parametrize("T,at", [(130, 70), (40, 17), (1500, 333)])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 40)])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_gradients(linattn, T, at, K, V, dtype, grad):  # noqa: F811
    """dk reads later d_o, and dv later q, the way outputs read earlier keys."""
    x = draw(dtype, T, K, V)
    decay = torch.tensor([-0.01, -0.3], device="cuda")
    call = lambda y: linattn.bwd(y["q"], y["k"], y["v"], decay, y["do"], grad_dtype=TYPES[grad])  # noqa: E731
    want = call(x)
    for name, grads in (("do", "k"), ("q", "v")):
        y = {**x, name: x[name].clone()}
        y[name][1, at] = float("nan")
        got = call(y)[grads]
        assert bits(got[0], want[grads][0]) and bits(got[1, at + 1:], want[grads][1, at + 1:])
        assert torch.isnan(got[1, at]).all()


@pytest.mark.parametrize("T,at", [(130, 70), (130, 97), (40, 17)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_values(linattn, T, at, dtype, out):  # noqa: F811
    """One in v reaches no token before its 32 tokens of the chunk."""
    x = draw(dtype, T, 64, 64)
    decay = torch.tensor([-0.01, -0.3], device="cuda")
    want, _ = linattn.fwd(x["q"], x["k"], x["v"], decay, out_dtype=TYPES[out])
    x["v"][1, at] = float("nan")
    o, _ = linattn.fwd(x["q"], x["k"], x["v"], decay, out_dtype=TYPES[out])
    assert bits(o[0], want[0]) and bits(o[1, :at // 32 * 32], want[1, :at // 32 * 32])
    assert torch.isnan(o[1, at]).all()
