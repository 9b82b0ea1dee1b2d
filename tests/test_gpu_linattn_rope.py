"""linattn.rope against the oracle: both layouts, parts of the head, far
positions, every piece width, strides, in place.

Bounds: the angle is the oracle's float64 product; its reduction keeps an
eighth of a turn to 2^-24 of itself (2^-24 pi/4 < u), sine and cosine are off
by at most 2 u more, the two products and their sum by u each of their terms:
6 u (|x| + |y|) in all, plus half a step of bfloat16 outputs."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import BF, TYPES, U, bits, f64, generator, normal, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def linattn():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import linattn

    return linattn


def check(name, got, x, positions, freqs, layout, inverse, bf16):
    ref = R.rope_ref(f64(x), positions, freqs, layout, inverse)
    R2 = len(freqs)
    size = np.abs(f64(x))
    i, j = (slice(0, 2 * R2, 2), slice(1, 2 * R2, 2)) if layout == "interleaved" else (slice(0, R2), slice(R2, 2 * R2))
    both = size[..., i] + size[..., j]
    bound = np.zeros_like(ref)
    bound[..., i] = bound[..., j] = 6 * U * both
    if bf16:
        bound[..., : 2 * R2] += BF * np.abs(ref[..., : 2 * R2]) + 2 * U * np.abs(ref[..., : 2 * R2])
    err = np.abs(f64(got) - ref)
    worst = float(np.max(err / np.maximum(bound, 1e-37))) if err.size else 0.0
    say(f"[rope] {name}: {worst:.3g} of the bound")
    assert np.all(err <= bound)


@pytest.mark.parametrize("D,Rn", [(64, 64), (64, 32), (80, 40), (80, 80), (128, 128), (128, 6), (8, 2), (72, 24), (40, 20)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matches_oracle(linattn, D, Rn, layout, dtype):
    g = generator(D + Rn)
    B, T, H = 2, 37, 3
    q, k = normal(g, B, T, H, D, dtype=TYPES[dtype]), normal(g, B, T, H, D, dtype=TYPES[dtype])
    freqs = linattn.rope_freqs(Rn)
    pos = torch.randint(-5, 2 ** 31 - 1, (B, T), generator=g, dtype=torch.int32)
    pos[0, 0], pos[0, 1], pos[1, 0] = 0, 2 ** 31 - 1, -(2 ** 31)
    for inverse in (False, True):
        a, b = linattn.rope(q.cuda(), k.cuda(), freqs, positions=pos.cuda(), layout=layout, inverse=inverse)
        torch.cuda.synchronize()
        for name, got, x in (("q", a, q), ("k", b, k)):
            check(f"D={D} R={Rn} {layout} {dtype} {name}", got, x, pos.numpy(), f64(freqs), layout, inverse, dtype == "bf16")


@pytest.mark.parametrize("B,T,H", [(1, 1, 1), (64, 1, 32), (3, 1000, 2), (2, 513, 5), (1, 20000, 1)])
@pytest.mark.parametrize("start", [0, 123456789012])
def test_counted_positions(linattn, B, T, H, start):
    """No positions given: start + t; q alone."""
    q = normal(generator(T), B, T, H, 64)
    freqs = linattn.rope_freqs(64, scaling="bands", factor=8.0)
    a, none = linattn.rope(q.cuda(), None, freqs, start=start)
    assert none is None
    pos = start + np.arange(T)[None].repeat(B, 0)
    check(f"B={B} T={T} H={H} from {start}", a, q, pos, f64(freqs), "half", False, False)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("Rn", [64, 32, 40, 4])
def test_layouts_and_in_place(linattn, layout, Rn):
    """In place, slices of a fused buffer, heads before tokens: the same bits; turning back returns."""
    B, T, H, D = 2, 50, 3, 80
    qkv = normal(generator(1), B, T, 3, H, D, dtype=torch.bfloat16).cuda()
    keep = qkv.clone()
    freqs = linattn.rope_freqs(Rn)
    q, k = (keep[:, :, i].contiguous() for i in range(2))
    want = linattn.rope(q, k, freqs, start=9, layout=layout)
    linattn.rope(qkv[:, :, 0], qkv[:, :, 1], freqs, start=9, layout=layout, q_out=qkv[:, :, 0], k_out=qkv[:, :, 1])
    assert bits(qkv[:, :, 0], want[0]) and bits(qkv[:, :, 1], want[1]) and bits(qkv[:, :, 2], keep[:, :, 2])
    t = q.transpose(1, 2).contiguous().transpose(1, 2)
    out = torch.empty_like(t)
    linattn.rope(t, None, freqs, start=9, layout=layout, q_out=out)
    assert bits(out, want[0])
    x = q.float()
    y, _ = linattn.rope(x, None, freqs, start=9, layout=layout)
    z, _ = linattn.rope(y, None, freqs, start=9, layout=layout, inverse=True)
    assert float((z - x).abs().max()) <= 12 * U * 2 * float(x.abs().max()) * 2


def test_rows_far_apart(linattn):
    wide = torch.empty((1, 70000, 1, 32768), dtype=torch.bfloat16, device="cuda")
    wide[..., :64] = normal(generator(3), 1, 70000, 1, 64, dtype=torch.bfloat16).cuda()
    q, out = wide[..., :64], wide[..., 64:128]
    freqs = linattn.rope_freqs(64)
    linattn.rope(q, None, freqs, q_out=out)
    assert bits(out, linattn.rope(q.contiguous(), None, freqs)[0])


def test_graph_and_stream(linattn):
    q, k = (normal(generator(i), 4, 1, 8, 64, dtype=torch.bfloat16).cuda() for i in range(2))
    pos = torch.tensor([[3], [70000], [0], [9]], dtype=torch.int32, device="cuda")
    freqs = linattn.rope_freqs(64, scaling="linear", factor=4.0)
    linattn.rope(q, k, freqs, positions=pos)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = linattn.rope(q, k, freqs, positions=pos)
    side = torch.cuda.Stream()
    for _ in range(3):
        pos.add_(1)
        torch.cuda.synchronize()
        g.replay()
        want = linattn.rope(q, k, freqs, positions=pos, stream=side)
        torch.cuda.synchronize()
        assert bits(out[0], want[0]) and bits(out[1], want[1])


def test_empty(linattn):
    q = torch.empty((2, 0, 3, 64), device="cuda")
    assert linattn.rope(q, q, linattn.rope_freqs(64))[0].shape == q.shape
