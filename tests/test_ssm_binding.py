"""Refusals of the ssm binding before any library call: no GPU needed.  The
library loader fails the test if it is reached."""
import pytest
import torch

from linear_attention_rnn_amd import ssm, wkv6
from tests.test_linattn_binding import Gpu


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def fail():
        raise AssertionError("the library was called")

    monkeypatch.setattr(wkv6, "lib", fail)


BF = torch.bfloat16
B, T, D, N, G, W = 2, 5, 16, 8, 2, 4


@pytest.mark.parametrize("kw", [
    dict(x=Gpu(B, T * D)), dict(x=torch.zeros(B, T, D)), dict(x=Gpu(B, T, D, dtype=torch.float16)),
    dict(x=Gpu(B, T, D, strides=(400, 32, 2))), dict(weight=Gpu(D * W)), dict(weight=Gpu(D + 8, W)), dict(weight=Gpu(D, W, dtype=BF)),
    dict(weight=torch.zeros(D, W)), dict(bias=Gpu(D + 1)), dict(activation="tanh"), dict(activation="sigmoid"),
    dict(lengths=Gpu(B)), dict(lengths=Gpu(B + 1, dtype=torch.int32)), dict(s_in=Gpu(B, W, D)), dict(s_in=Gpu(B, W - 1, D, dtype=BF)),
    dict(out=Gpu(B, T, D, dtype=BF)), dict(out=torch.zeros(B, T, D))])
def test_conv_refuses(kw):
    x = dict(x=Gpu(B, T, D), weight=Gpu(D, W), bias=Gpu(D), out=Gpu(B, T, D), s_in=Gpu(B, W - 1, D))
    x.update(kw)
    with pytest.raises(ValueError):
        ssm.conv(s_out=Gpu(B, W - 1, D), **x)
    with pytest.raises(ValueError):
        ssm.conv_bwd(dy=Gpu(B, T, D), **x)


def test_conv_outputs_refused():
    with pytest.raises(ValueError):
        ssm.conv(Gpu(B, T, D), Gpu(D, W), out=Gpu(B, T, D), s_out=Gpu(B, W, D))
    for dy in (Gpu(B, T, D, dtype=BF), Gpu(B, T, D + 8), Gpu(B, T, D, device="cuda:1")):
        with pytest.raises(ValueError):
            ssm.conv_bwd(Gpu(B, T, D), Gpu(D, W), dy)


def scan_inputs(**kw):
    x = dict(x=Gpu(B, T, D), dt=Gpu(B, T, D), A=Gpu(D, N), B=Gpu(B, T, G, N), C=Gpu(B, T, G, N), D=Gpu(D), z=Gpu(B, T, D),
             dt_bias=Gpu(D), s_in=Gpu(B, D, N))
    x.update(kw)
    return x


@pytest.mark.parametrize("kw", [
    dict(x=Gpu(B, T * D)), dict(dt=Gpu(B, T, D + 8)), dict(dt=Gpu(B, T, D, dtype=BF)), dict(A=Gpu(D)), dict(A=Gpu(D, N + 8)),
    dict(A=Gpu(D, N, dtype=BF)), dict(B=Gpu(B, T, N)), dict(C=Gpu(B, T, 1, N)), dict(B=Gpu(B, T, G, N, strides=(200, 32, 1, 2))),
    dict(D=Gpu(N)), dict(z=Gpu(B, T)), dict(z=Gpu(B, T, D, dtype=BF)), dict(dt_bias=Gpu(D, dtype=BF)), dict(s_in=Gpu(B, N, D)),
    dict(s_in=Gpu(B, D, N, strides=(500, 12, 1))), dict(lengths=Gpu(B, 1, dtype=torch.int32)), dict(C=Gpu(B, T, G, N, device="cuda:1"))])
def test_scan_refuses(kw):
    with pytest.raises(ValueError):
        ssm.scan(out=Gpu(B, T, D), **scan_inputs(**kw))
    grads = {n: Gpu(B, T, D) for n in ("x", "dt", "z")} | {n: Gpu(B, T, G, N) for n in ("B", "C")}
    with pytest.raises(ValueError):
        ssm.scan_bwd(dy=Gpu(B, T, D), out=grads, **scan_inputs(**kw))


def test_scan_outputs_refused():
    with pytest.raises(ValueError):
        ssm.scan(out=Gpu(B, T, D + 8), **scan_inputs())
    with pytest.raises(ValueError):
        ssm.scan(out=Gpu(B, T, D), s_out=Gpu(B, D, N, dtype=BF), **scan_inputs())
    full = {n: Gpu(B, T, D) for n in ("x", "dt", "z")} | {n: Gpu(B, T, G, N) for n in ("B", "C")}
    for bad in (dict(x=Gpu(B, T, D, dtype=BF)), dict(B=Gpu(B, T, N)), dict(A=Gpu(D, N))):
        with pytest.raises(ValueError):
            ssm.scan_bwd(dy=Gpu(B, T, D), out={**full, **bad}, **scan_inputs())
    with pytest.raises(ValueError):
        ssm.scan_bwd(dy=Gpu(B, T, D), out=full, **scan_inputs(z=None))
    with pytest.raises(ValueError):
        ssm.scan_bwd(dy=Gpu(B, T, D), out={**full, "y": Gpu(B, T, D)}, **scan_inputs())


@pytest.mark.parametrize("kw", [
    dict(x=torch.zeros(4, 16)), dict(x=Gpu(4, 16, dtype=torch.float16)), dict(x=Gpu(4, 16, strides=(32, 1))), dict(gate=Gpu(3, 16)),
    dict(gate=Gpu(8, 16)), dict(gate=Gpu(4, 8)), dict(gate=Gpu(4, 16, dtype=BF)), dict(gate=Gpu(0, 16)), dict(gate=None),
    dict(activation="tanh"), dict(post_weight=Gpu(8)), dict(pre_weight=Gpu(16, dtype=BF))])
def test_block_norm_refuses(kw):
    x = dict(x=Gpu(4, 16), gate=Gpu(2, 16), post_weight=Gpu(16), pre_weight=Gpu(16), activation="silu")
    x.update(kw)
    with pytest.raises(ValueError):
        ssm.block_norm(h=Gpu(4, 16), out=Gpu(4, 16), **x)
    with pytest.raises(ValueError):
        ssm.block_norm_bwd(h=Gpu(4, 16), dy=Gpu(4, 16), out=Gpu(4, 16), residual_out=Gpu(4, 16), **x)


@pytest.mark.parametrize("shape,gate", [((2, 3, 16), (3, 16)), ((2, 3, 16), (1, 3, 16)), ((3, 3, 16), (1, 3, 16)), ((2, 6, 16), (3, 16)),
                                        ((2, 3, 4, 16), (2, 1, 4, 16)), ((4, 2, 16), (2, 1, 16))])
def test_gates_that_other_rows_would_share_refused(shape, gate):
    """Broadcasting would repeat them over rows that do not follow each other."""
    x = Gpu(*shape)
    with pytest.raises(ValueError):
        ssm.block_norm(x, gate=Gpu(*gate), h=x)
    with pytest.raises(ValueError):
        ssm.block_norm_bwd(x, None, gate=Gpu(*gate), out=Gpu(*shape), residual_out=Gpu(*shape))


def test_block_norm_outputs_refused():
    x = Gpu(4, 16)
    for kw in (dict(h=Gpu(4, 8)), dict(h=Gpu(4, 16), out=Gpu(4, 16)), dict(h=Gpu(4, 16), residual=Gpu(4, 16, dtype=BF))):
        with pytest.raises(ValueError):
            ssm.block_norm(x, **kw)
    w = Gpu(16)
    for kw in (dict(h=None, dy=x, pre_weight=w), dict(h=x, pre_weight=w), dict(h=x, dy=x), dict(h=x, dh=Gpu(4, 8))):
        with pytest.raises(ValueError):
            ssm.block_norm_bwd(x, out=Gpu(4, 16), residual_out=Gpu(4, 16), **kw)


def test_unknown_outputs_refused_as_none_too():
    full = {n: Gpu(B, T, D) for n in ("x", "dt", "z")} | {n: Gpu(B, T, G, N) for n in ("B", "C")}
    with pytest.raises(ValueError):
        ssm.scan_bwd(dy=Gpu(B, T, D), out={**full, "y": None}, **scan_inputs())
