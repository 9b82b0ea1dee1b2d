"""The largest numbers of sequences and rows that ssm.h allows, on the fewest
channels: both ends and places between them, bit for bit the calls on those alone."""
import pytest
import torch

from tests import ssm_util as S
from tests.ssm_util import bits, generator, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    yield ssm
    torch.cuda.empty_cache()


def over(t, count):
    """Rows of t over and over, `count` in all."""
    return t.repeat(-(-count // t.shape[0]), *[1] * (t.dim() - 1))[:count]


@pytest.mark.parametrize("T", [1, 10])
def test_sequences_of_a_scan(ssm, T):
    """2^22 sequences of 8 channels."""
    B, few = 2 ** 22, 96
    p = S.cuda(S.inputs(T, few, T, 8, 8, 1, "bf16"))
    dy = normal(generator(1), few, T, 8, std=1.0, dtype=torch.bfloat16).cuda()
    shared = ("A", "D", "dt_bias")
    many = {n: t if n in shared else over(t, B) for n, t in p.items()}
    y, s = ssm.scan(**many, want_state=True)
    want_y, want_s = ssm.scan(**p, want_state=True)
    torch.cuda.synchronize()
    places = [a // few * few for a in (0, B // 2, 3 * B // 4, B - few)]
    for a in places:
        assert bits(y[a:a + few], want_y) and bits(s[a:a + few], want_s), a
    if T == 1:   # (the sums of dA over so many sequences are long chains of one thread)
        return
    B = 2 ** 18
    many = {n: t if n in shared else over(t, B) for n, t in p.items()}
    got, want = ssm.scan_bwd(**many, dy=over(dy, B)), ssm.scan_bwd(**p, dy=dy)
    torch.cuda.synchronize()
    for a in (0, B // 2 // few * few, (B - few) // few * few):
        for n in ("x", "dt", "B", "C", "z"):
            assert bits(got[n][a:a + few], want[n]), (n, a)


def test_sequences_of_a_convolution(ssm):
    """2^20 sequences of 8 channels: 258 x 10 x 2^20 work-items, below 2^32."""
    B, few = 2 ** 20, 64
    g = generator(4)
    x, w, s_in = normal(g, few, 3, 8).cuda(), normal(g, 8, 4).cuda(), normal(g, few, 3, 8).cuda()
    y, s = ssm.conv(over(x, B), w, s_in=over(s_in, B), want_state=True)
    want_y, want_s = ssm.conv(x, w, s_in=s_in, want_state=True)
    got, want = ssm.conv_bwd(over(x, B), w, over(x, B)), ssm.conv_bwd(x, w, x)
    torch.cuda.synchronize()
    for a in (0, B // 2, B - few):
        assert bits(y[a:a + few], want_y) and bits(s[a:a + few], want_s) and bits(got["x"][a:a + few], want["x"]), a


@pytest.mark.parametrize("C,rows,per", [(8, 2 ** 25, 8), (520, 2 ** 21, 1), (520, 2 ** 21, 2 ** 21)])
def test_rows_of_a_norm(ssm, C, rows, per):
    """2^25 rows with 2^22 gates, each of 8 of them, and the most rows of more than 512 columns."""
    few = 64
    g = generator(C)
    x, dh = (normal(g, few, C, std=1.0, dtype=torch.bfloat16).cuda() for _ in range(2))
    one = normal(g, max(1, few // per), C, std=1.0, dtype=torch.bfloat16).cuda()
    w = (1 + normal(g, C, std=0.2)).cuda()
    gates = over(one, rows // per)
    y, h = ssm.block_norm(over(x, rows), gate=gates, post_weight=w, pre_weight=w, activation="silu")
    want_y, want_h = ssm.block_norm(x, gate=one, post_weight=w, pre_weight=w, activation="silu")
    torch.cuda.synchronize()
    places = (0, rows // 2, rows - few)
    for a in places:
        assert bits(y[a:a + few], want_y) and bits(h[a:a + few], want_h), a
    del y, want_y
    kw = dict(post_weight=w, pre_weight=w, activation="silu")
    got = ssm.block_norm_bwd(over(x, rows), h, dy=over(dh, rows), dh=over(dh, rows), gate=gates, **kw)
    want = ssm.block_norm_bwd(x, want_h, dy=dh, dh=dh, gate=one, **kw)
    torch.cuda.synchronize()
    for a in places:
        assert bits(got["x"][a:a + few], want["x"]) and bits(got["residual"][a:a + few], want["residual"]), a
        if per == 8:
            assert bits(got["gate"][a // 8:a // 8 + 8], want["gate"]), a
