"""ssm.scan and conv on tensors whose tokens and batch items pass 2^32 bytes and
2^31 elements: bit for bit the calls on contiguous ones."""
import pytest
import torch

from tests import ssm_util as S
from tests.ssm_util import bits, generator, normal

pytestmark = pytest.mark.gpu

B, D, N = 2, 24, 16


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


@pytest.fixture(scope="module")
def room():
    """8 GiB, of which the tests use a few rows."""
    buffer = torch.empty(2 ** 32, dtype=torch.bfloat16, device="cuda")
    yield buffer
    del buffer
    torch.cuda.empty_cache()


def far(room, shape, slot, T):
    """A tensor of the room: the second batch item 2^31 elements behind the first, tokens spread over the rest."""
    batch, token = 2 ** 31, (2 ** 31 - 2 ** 16) // T // 8 * 8
    inner = (token, shape[-1], 1) if len(shape) == 4 else (token, 1)
    t = room.as_strided(shape, (batch, *inner), slot * 256)
    assert slot * 256 + (shape[1] - 1) * token + 256 <= batch
    return t


@pytest.mark.parametrize("T", [5, 150])
def test_scan(ssm, room, T):
    p = S.cuda(S.inputs(T, B, T, D, N, 1, "bf16"))
    dy = normal(generator(1), B, T, D, std=1.0, dtype=torch.bfloat16).cuda()
    want, want_s = ssm.scan(**p, want_state=True)
    want_g = ssm.scan_bwd(**p, dy=dy)
    q = dict(p)
    for i, n in enumerate(("x", "dt", "B", "C", "z")):
        q[n] = far(room, p[n].shape, i, T)
        q[n].copy_(p[n])
    d = far(room, dy.shape, 5, T)
    d.copy_(dy)
    y = far(room, dy.shape, 6, T)
    y, s = ssm.scan(**q, want_state=True, out=y)
    out = {n: far(room, p[n].shape, 7 + i, T) for i, n in enumerate(("x", "dt", "B", "C", "z"))}
    g = ssm.scan_bwd(**q, dy=d, out=out)
    torch.cuda.synchronize()
    assert bits(y.contiguous(), want) and bits(s, want_s)
    for n in want_g:
        assert bits(g[n].contiguous(), want_g[n]), n


@pytest.mark.parametrize("T", [5, 150])
def test_conv(ssm, room, T):
    g = generator(T)
    x, dy = (normal(g, B, T, D, std=1.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    w, b = normal(g, D, 4, std=0.5).cuda(), normal(g, D, std=0.1).cuda()
    want, want_s = ssm.conv(x, w, b, want_state=True)
    want_g = ssm.conv_bwd(x, w, dy, bias=b)
    fx, fd = far(room, x.shape, 0, T), far(room, x.shape, 1, T)
    fx.copy_(x)
    fd.copy_(dy)
    y, s = ssm.conv(fx, w, b, want_state=True, out=far(room, x.shape, 2, T))
    got = ssm.conv_bwd(fx, w, fd, bias=b, out=far(room, x.shape, 3, T))
    torch.cuda.synchronize()
    assert bits(y.contiguous(), want) and bits(s, want_s)
    for n in want_g:
        assert bits(got[n].contiguous(), want_g[n]), n
