"""Keys and values of different widths as slices of one projection's output:
inputs, outputs and gradients in one buffer each, bit for bit the calls on
tensors of their own; rows between the slices keep what they hold."""
import pytest
import torch

from tests.linattn_util import TYPES, bits, generator, normal
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu


def cut(buffer, H, *widths):
    """[B, T, sum(H * w) + 8] as [B, T, H, w] slices side by side."""
    B, T, _ = buffer.shape
    parts = buffer[..., :H * sum(widths)].split([H * w for w in widths], -1)
    return [p.unflatten(-1, (H, w)) for p, w in zip(parts, widths)]


@pytest.mark.parametrize("B,T", [(2, 1), (3, 7), (2, 100), (1, 1500)])
@pytest.mark.parametrize("K,V", [(64, 128), (128, 40)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_buffer(linattn, B, T, K, V, dtype):  # noqa: F811
    H, t = 3, TYPES[dtype]
    g = generator(T + K)
    decay = torch.tensor([-0.3, -0.02, -0.001], device="cuda")
    x = [normal(g, B, T, H, w, dtype=t).cuda() for w in (K, K, V, V)]
    want, _ = linattn.fwd(*x[:3], decay)
    grads = linattn.bwd(*x[:3], decay, x[3], grad_dtype=t)
    inputs = torch.full((B, T, H * (2 * K + 3 * V) + 8), 7.0, dtype=t, device="cuda")
    *views, o = cut(inputs, H, K, K, V, V, V)
    for a, b in zip(views, x):
        a.copy_(b)
    linattn.fwd(*views[:3], decay, out=o)
    assert bits(o, want) and all(bits(a, b) for a, b in zip(views, x)) and torch.all(inputs[..., -8:] == 7)
    out = torch.full((B, T, H * (2 * K + V) + 8), 7.0, dtype=t, device="cuda")
    dq, dk, dv = cut(out, H, K, K, V)
    got = linattn.bwd(*views[:3], decay, views[3], out={"q": dq, "k": dk, "v": dv})
    assert all(bits(got[n], grads[n]) for n in grads) and torch.all(out[..., -8:] == 7)
    assert got["q"].data_ptr() == out.data_ptr()
