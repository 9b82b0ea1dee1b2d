"""The ends of the selective state space layer's calls: batches without rows,
what is not finite in the last token, gradients that it must not reach, rows of
zeros with the smallest eps."""
import numpy as np
import pytest
import torch

from oracle import ssm_oracle as R
from tests import ssm_util as S
from tests.ssm_util import TYPES, U, bits, f64, generator, normal

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


def poison():
    """NaN in what torch's allocator hands out next."""
    torch.cuda.synchronize()
    junk = [torch.full((n,), NAN, device="cuda") for n in (16, 64, 128, 512, 1024, 4096) for _ in range(16)]
    torch.cuda.synchronize()
    del junk


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,gate", [((0, 64), (64,)), ((0, 64), (1, 64)), ((3, 0, 64), (3, 1, 64)), ((3, 0, 64), (3, 64)),
                                        ((0, 5, 64), (1, 1, 64)), ((0, 64), (0, 64)), ((2, 0, 64), (2, 0, 64))])
@pytest.mark.parametrize("weights", [True, False])
def test_gates_of_no_rows(ssm, shape, gate, weights, dtype):
    """The gradient of a gate that no row uses is zero."""
    t = TYPES[dtype]
    x, g = torch.ones(shape, dtype=t, device="cuda"), torch.ones(gate, dtype=t, device="cuda")
    w = torch.ones(64, device="cuda") if weights else None
    kw = dict(gate=g, post_weight=w, pre_weight=w, activation="silu")
    y, h = ssm.block_norm(x, **kw)
    poison()
    got = ssm.block_norm_bwd(x, h, dy=y, **kw)
    torch.cuda.synchronize()
    assert got["x"].shape == x.shape and got["gate"].shape == g.shape and got["gate"].dtype is t
    for n in set(got) - {"x", "residual"}:
        assert torch.equal(got[n], torch.zeros_like(got[n])), n


def changed(name, got, clean, ref, ref_clean, nan):
    """Places whose reference does not change keep their bits; with a NaN, those that it reaches are not finite."""
    for n in got:
        same = ref[n] == ref_clean[n]
        a, b = (f64(t) for t in (got[n], clean[n]))
        assert np.array_equal(a[same], b[same]), f"{name}: d{n}"
        if nan:
            assert not np.isfinite(a[~np.isfinite(ref[n])]).any(), f"{name}: d{n}"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [None, [200, 151]])
@pytest.mark.parametrize("T,N", [(200, 16), (200, 40), (256, 16), (20, 8)])
@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "z", "dy"])
def test_scan_gradients_that_nan_reaches(ssm, name, T, N, lengths, dtype):
    """A NaN in the middle and in the last token of one sequence reaches what the formulas say and nothing else."""
    D, G = 32, 2
    lengths = None if lengths is None else [n * T // 200 for n in lengths]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    p = S.inputs(2, 2, T, D, N, G, dtype)
    p["dy"] = normal(generator(1), 2, T, D, std=1.0, dtype=p["x"].dtype)
    ds = normal(generator(2), 2, D, N)

    def both(p):
        q = S.oracle_args({k: v for k, v in p.items() if k != "dy"})
        with np.errstate(all="ignore"):
            ref = R.scan_ref_backward(**q, dy=f64(p["dy"]), ds_out=f64(ds), lengths=lengths)
        g = ssm.scan_bwd(**S.cuda(p), ds_out=ds.cuda(), lengths=n, want_ds_in=True)
        torch.cuda.synchronize()
        return g, ref

    clean, ref_clean = both(p)
    for at in (T // 2 + 3, (lengths or [T, T])[1] - 1):
        bad = {k: None if v is None else v.clone() for k, v in p.items()}
        bad[name][1, at].view(-1)[:2] = NAN
        got, ref = both(bad)
        changed(f"{name} at {at}", got, clean, ref, ref_clean, True)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("activation", ["silu", None])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("name", ["x", "dy"])
def test_conv_gradients_that_nan_reaches(ssm, name, W, activation, bad):
    """The same for the convolution, padded: the tokens behind the last one have no gradients that could meet it."""
    B, T, D = 2, 60, 16
    lengths = [60, 37]
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    g = generator(W)
    p = {"x": normal(g, B, T, D, std=1.0), "weight": normal(g, D, W), "bias": normal(g, D), "s_in": normal(g, B, W - 1, D),
         "dy": normal(g, B, T, D)}

    def both(p):
        q = {k: f64(v) for k, v in p.items()}
        with np.errstate(all="ignore"):
            ref = R.conv_ref_backward(**q, activation=activation, lengths=lengths)
        got = ssm.conv_bwd(**S.cuda(p), activation=activation, lengths=n, want_ds_in=True)
        torch.cuda.synchronize()
        return got, ref

    clean, ref_clean = both(p)
    for at in (20, 36):
        spoiled = {k: v.clone() for k, v in p.items()}
        spoiled[name][1, at, 5] = bad
        got, ref = both(spoiled)
        changed(f"{name} at {at}", got, clean, ref, ref_clean, bad != bad)


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_behind_a_sequence_are_zero(ssm, dtype, bad):
    """Also with weights, biases and states that are not finite."""
    B, T, D, W = 3, 70, 16, 4
    lengths = [0, 33, 68]
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    g, t = generator(5), TYPES[dtype]
    x, dy = (normal(g, B, T, D, std=1.0, dtype=t).cuda() for _ in range(2))
    w, b, s = normal(g, D, W).cuda(), normal(g, D).cuda(), normal(g, B, W - 1, D, dtype=t).cuda()
    p = S.cuda(S.inputs(3, B, T, D, 16, 1, dtype))
    for place in ((w, (3, 1)), (b, (5,)), (s, (1, 0, 7)), (p["s_in"], (1, 2, 3)), (p["D"], (4,)), (p["A"], (6, 2))):
        place[0][place[1]] = bad
    outs = [ssm.conv(x, w, b, lengths=n, s_in=s)[0]]
    for act in ("silu", None):
        outs.append(ssm.conv_bwd(x, w, dy, bias=b, activation=act, lengths=n, s_in=s)["x"])
    outs.append(ssm.scan(**p, lengths=n)[0])
    grads = ssm.scan_bwd(**p, dy=dy, lengths=n)
    torch.cuda.synchronize()
    for i, o in enumerate(outs + [grads[m] for m in ("x", "dt", "B", "C", "z")]):
        for k, length in enumerate(lengths):
            assert not o[k, length:].any(), (i, k)


@pytest.mark.parametrize("C", [64, 1024, 2048, 16384])
def test_zero_rows_with_the_smallest_eps(ssm, C):
    """A row of zeros, whose root is sqrt(eps): 1 / rms is 2^64 at most, its square no float32.  dx = scale post pre dy / eps
    would pass the range as well, so each norm is looked at by itself: dx = weight dy / sqrt(eps), roundings as in the norm tests."""
    eps = 2.0 ** -128
    g = generator(C)
    x, w, dy = torch.zeros(3, C), 1.0 + normal(g, C, std=0.3), normal(g, 3, C, std=1.0)
    x[1] = normal(g, C, std=1.0)
    xs, ws, dys = x.cuda(), w.cuda(), dy.cuda()
    y, h = ssm.block_norm(xs, pre_weight=ws, eps=eps)
    pre = ssm.block_norm_bwd(xs, h, dy=dys, pre_weight=ws, eps=eps)
    post = ssm.block_norm_bwd(xs, None, dh=dys, post_weight=ws, eps=eps)
    torch.cuda.synchronize()
    q = [f64(v) for v in (x, x, dy, None)[:3]]
    ref = R.block_norm_ref_backward(q[0], q[1], q[2], pre=f64(w), eps=eps)
    assert np.array_equal(f64(y)[[0, 2]], np.zeros((2, C)))
    for got in (pre["x"], post["x"]):
        size = np.abs(ref["x"]) + R.unit(q[0], eps)[1] * np.abs(f64(w) * q[2])
        assert np.isfinite(f64(got)).all() and (np.abs(f64(got) - ref["x"]) <= 160 * U * size).all()


def test_outputs_given_as_none(ssm):
    """An output given as None is a new tensor, the state's gradient among them."""
    p = S.cuda(S.inputs(4, 2, 20, 16, 16, 1, "f32"))
    dy = torch.ones_like(p["x"])
    want = ssm.scan_bwd(**p, dy=dy, want_ds_in=True)
    got = ssm.scan_bwd(**p, dy=dy, want_ds_in=True, out={n: None for n in ("x", "dt", "B", "C", "z", "s_in")})
    plain = ssm.scan_bwd(**p, dy=dy, out={"s_in": None})
    torch.cuda.synchronize()
    assert set(got) == set(want) and all(bits(got[n], want[n]) for n in want)
    assert set(plain) == set(want) - {"s_in"}
