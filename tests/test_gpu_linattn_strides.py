"""Token rows up to 33.5 MB apart, and any distance for single tokens and rotary
positions; one layer's row of a table of decays.  Bit for bit the calls on
packed tensors."""
import pytest
import torch

from tests.linattn_util import TYPES, bits, generator, normal
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu


def far(x, distance, dtype):
    """x [1, T, H, D] with `distance` elements between tokens."""
    _, T, H, D = x.shape
    buffer = torch.empty((T - 1) * distance + H * D, dtype=dtype, device="cuda")
    view = torch.as_strided(buffer, (1, T, H, D), (0, distance, D, 1))
    view.copy_(x)
    return view


@pytest.mark.parametrize("T,dtype,distance", [(70, "bf16", 33554288 // 2), (70, "f32", 33554288 // 4), (8, "bf16", 2 ** 26),
                                              (8, "f32", 2 ** 26)])
def test_tokens_far_apart(linattn, T, dtype, distance):  # noqa: F811
    g, t = generator(T), TYPES[dtype]
    q, k, v = (normal(g, 1, T, 2, 64, dtype=t).cuda() for _ in range(3))
    decay = torch.tensor([-0.01, -0.2], device="cuda")
    want, S = linattn.fwd(q, k, v, decay, want_state=True)
    o, S2 = linattn.fwd(q, far(k, distance, t), v, decay, want_state=True, out=far(torch.zeros_like(v), distance, t))
    assert bits(o, want) and bits(S, S2)
    if T > 8:
        want = linattn.bwd(q, k, v, decay, v, grad_dtype=t)
        got = linattn.bwd(far(q, distance, t), k, v, decay, v, grad_dtype=t,
                          out={"v": far(torch.zeros_like(v), distance, t)})
        assert all(bits(got[n], want[n]) for n in want)


def test_rotary_positions_far_apart(linattn):  # noqa: F811
    q = normal(generator(1), 1, 3, 2, 64, dtype=torch.bfloat16).cuda()
    freqs = linattn.rope_freqs(64)
    x = far(q, 2 ** 31, torch.bfloat16)
    want, _ = linattn.rope(q, None, freqs, start=5)
    linattn.rope(x, None, freqs, start=5, q_out=x)
    assert bits(x, want)


def test_rows_of_tables(linattn):  # noqa: F811
    g = generator(2)
    H = 3
    decays = -0.1 * torch.arange(1, 13, dtype=torch.float32, device="cuda").view(4, H)
    for T in (1, 100):
        q, k, v = (normal(g, 4, T, H, 64, dtype=torch.bfloat16).cuda() for _ in range(3))
        positions = torch.randint(0, 9999, (4, T), generator=g, dtype=torch.int32).cuda()
        freqs = linattn.rope_freqs(64)
        for i in range(4):
            assert bits(linattn.fwd(q, k, v, decays[i])[0], linattn.fwd(q, k, v, decays[i].clone())[0])
            assert bits(linattn.rope(q[i:], None, freqs, positions[i:])[0], linattn.rope(q, None, freqs, positions)[0][i:])
