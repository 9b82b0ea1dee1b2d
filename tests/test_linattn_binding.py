"""Refusals of the linattn binding before any library call, and the table of
rotary frequencies: no GPU needed.  The library loader fails the test if it is
reached."""
import math

import pytest
import torch

from linear_attention_rnn_amd import linattn, wkv6


class Gpu:
    """A host tensor that says it lies on a GPU."""

    def __init__(self, *shape, dtype=torch.float32, device="cuda:0", strides=None):
        self.t = torch.zeros(shape, dtype=dtype)
        if strides:
            self.t = torch.as_strided(torch.zeros(1 << 16, dtype=dtype), shape, strides)
        self.device, self.is_cuda, self.shape, self.dtype = torch.device(device), True, self.t.shape, dtype

    def __getattr__(self, name):
        return getattr(self.t, name)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def fail():
        raise AssertionError("the library was called")

    monkeypatch.setattr(wkv6, "lib", fail)


B, T, H, K, V = 2, 5, 3, 16, 24
BF, F32 = torch.bfloat16, torch.float32


def attention(**kw):
    x = {"q": Gpu(B, T, H, K), "k": Gpu(B, T, H, K), "v": Gpu(B, T, H, V), "log_decay": Gpu(H), "out": Gpu(B, T, H, V)}
    x.update(kw)
    return x


BAD = [
    dict(q=Gpu(B, T, H * K)), dict(q=Gpu(B, T, H, K, dtype=torch.float16)), dict(k=Gpu(B, T, H, V)),
    dict(k=Gpu(B, T, H, K, dtype=BF)), dict(v=Gpu(B, T + 1, H, V)), dict(v=torch.zeros(B, T, H, V)),
    dict(k=Gpu(B, T, H, K, device="cuda:1")), dict(q=Gpu(B, T, H, K, strides=(1000, 200, 2, 8))),
    dict(log_decay=Gpu(H + 1)), dict(log_decay=Gpu(H, dtype=torch.float64)), dict(log_decay=torch.zeros(H)),
    dict(lengths=Gpu(B)), dict(lengths=Gpu(B + 1, dtype=torch.int32)), dict(s_in=Gpu(B, H, V, K)),
    dict(s_in=Gpu(B, H, K, V, dtype=BF)), dict(s_in=Gpu(B, H, K, V, strides=(5000, 1000, 30, 1))),
]


@pytest.mark.parametrize("kw", BAD + [
    dict(out=torch.zeros(B, T, H, V)), dict(out=Gpu(B, T, H, V, device="cuda:1")), dict(out=Gpu(B, T, H, K)),
    dict(out_dtype=BF), dict(s_out=torch.zeros(B, H, K, V)), dict(s_out=Gpu(B, H, K, K))])
def test_fwd_refuses(kw):
    with pytest.raises(ValueError):
        linattn.fwd(**attention(**kw))


@pytest.mark.parametrize("kw", BAD + [
    dict(do=Gpu(B, T, H, K)), dict(do=Gpu(B, T, H, V, dtype=BF)), dict(ds_out=Gpu(B, H, K)),
    dict(out={"q": torch.zeros(B, T, H, K)}), dict(out={"q": Gpu(B, T, H, K), "k": Gpu(B, T, H, K, dtype=BF)})])
def test_bwd_refuses(kw):
    x = attention(do=Gpu(B, T, H, V))
    x["out"] = {"q": Gpu(B, T, H, K), "k": Gpu(B, T, H, K), "v": Gpu(B, T, H, V), "s_in": Gpu(B, H, K, V)}
    x.update(kw)
    with pytest.raises((ValueError, RuntimeError, AssertionError)) as e:
        linattn.bwd(**x)
    assert "library was called" not in str(e.value)


@pytest.mark.parametrize("kw", [
    dict(layout="quarter"), dict(q=Gpu(B, T, H)), dict(k=Gpu(B, T, H, V)), dict(freqs=Gpu(8)), dict(freqs=None),
    dict(freqs=Gpu(8, 1, dtype=torch.float64)), dict(positions=Gpu(B, T)), dict(positions=Gpu(B, dtype=torch.int32)),
    dict(q_out=torch.zeros(B, T, H, K)), dict(k=None), dict(k_out=Gpu(B, T, H, K, dtype=BF)),
    dict(q=Gpu(B, T, H, K, dtype=torch.float16))])
def test_rope_refuses(kw):
    x = dict(q=Gpu(B, T, H, K), k=Gpu(B, T, H, K), freqs=Gpu(8, dtype=torch.float64), q_out=Gpu(B, T, H, K),
             k_out=Gpu(B, T, H, K))
    x.update(kw)
    with pytest.raises(ValueError):
        linattn.rope(**x)


@pytest.mark.parametrize("kw", [
    dict(x=torch.zeros(4, 16)), dict(x=Gpu(4, 16, dtype=torch.float16)), dict(x=Gpu(4, 16, strides=(32, 1))),
    dict(weight=Gpu(8)), dict(weight=Gpu(16, dtype=BF)), dict(residual=Gpu(4, 8)), dict(residual=Gpu(4, 16, dtype=BF)),
    dict(residual=None), dict(h=torch.zeros(4, 16)), dict(residual=Gpu(4, 16, device="cuda:1"))])
def test_norm_refuses(kw):
    x = dict(x=Gpu(4, 16), weight=Gpu(16), residual=Gpu(4, 16), h=Gpu(4, 16))
    x.update(kw)
    with pytest.raises(ValueError):
        linattn.rms_norm(out=Gpu(4, 16), **x)
    with pytest.raises(ValueError):
        linattn.rms_norm_q8(codes=Gpu(4, 16), **x)


@pytest.mark.parametrize("kw", [dict(out=torch.zeros(4, 16)), dict(out=Gpu(4, 16, dtype=BF))])
def test_norm_output_refused(kw):
    with pytest.raises(ValueError):
        linattn.rms_norm(Gpu(4, 16), Gpu(16), **kw)


@pytest.mark.parametrize("kw", [dict(group=64), dict(codes=Gpu(4, 16)), dict(codes=Gpu(4, 16, dtype=torch.float8_e4m3fn), scales=Gpu(4, 2))])
def test_q8_refuses(kw):
    with pytest.raises(ValueError):
        linattn.rms_norm_q8(Gpu(4, 16), Gpu(16), **kw)


@pytest.mark.parametrize("kw", [dict(dy=Gpu(4, 8)), dict(dy=None), dict(dh=Gpu(4, 16, dtype=BF)), dict(weight=Gpu(4)),
                                dict(out=torch.zeros(4, 16))])
def test_norm_bwd_refuses(kw):
    x = dict(dy=Gpu(4, 16), h=Gpu(4, 16), weight=Gpu(16), out=Gpu(4, 16))
    x.update(kw)
    with pytest.raises(ValueError):
        linattn.rms_norm_bwd(**x)


def test_frequencies():
    f = linattn.rope_freqs(8, device="cpu")
    assert f.dtype == torch.float64 and f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-15)
    assert linattn.rope_freqs(8, scaling="linear", factor=4.0, device="cpu").tolist() == pytest.approx((f / 4).tolist())
    b = linattn.rope_freqs(8, scaling="base", factor=4.0, device="cpu")
    assert b[0] == 1.0 and b[3].item() == pytest.approx(f[3].item() / 4) and b[1] < f[1]
    # 4096 f / 2 pi turns: 652, 65, 6.5, 0.65
    g = linattn.rope_freqs(8, scaling="bands", factor=4.0, device="cpu")
    t = 4096 * 0.01 / (2 * math.pi)
    keep = (t - 1) / 31
    assert g.tolist() == pytest.approx([1.0, 0.1, 0.01 * (keep + (1 - keep) / 4), 0.001 / 4], rel=1e-12)


@pytest.mark.parametrize("kw", [dict(R=7), dict(R=0), dict(R=8, scaling="magic"), dict(R=8, scaling="linear", factor=0.0),
                                dict(R=2, scaling="base", factor=2.0),
                                dict(R=8, scaling="bands", factor=2.0, slow_turns=4.0, fast_turns=4.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        linattn.rope_freqs(device="cpu", **kw)
