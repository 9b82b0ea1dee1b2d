"""ssm.block_norm and block_norm_bwd against the oracle.

Bounds (u = 2^-24): a mean over C squares errs by 41 u (32 columns a thread, 9
levels of lanes and waves), its root by half, root, quotient and products by u
each, an activation by 12 u: 48 u of each term of h covers it, 30 u |y| y.
Gradients: two such means and their products, 160 u of the absolute terms; sums
over rows are chains of at most 32 rows and 64 bits: 32 u more.  bfloat16 adds half a
step, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import ssm_oracle as R
from tests.ssm_util import BF, TYPES, U, bits, f64, generator, normal, within

pytestmark = pytest.mark.gpu

# rows, C, rows that share a gate
SHAPES = [(1, 8, 1), (6, 64, 3), (70, 72, 1), (40, 136, 20), (65, 264, 13), (7, 520, 7), (300, 1032, 1), (96, 2048, 48), (1200, 512, 1200),
          (9, 4104, 3), (5, 8200, 1), (4, 16384, 2), (3000, 64, 2)]
ALL = ("residual", "gate", "post", "pre")


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


def draw(rows, C, per, dtype, parts=ALL):
    g, t = generator(rows + C), TYPES[dtype]
    p = {"x": normal(g, rows, C, std=1.0, dtype=t), "residual": normal(g, rows, C, std=2.0, dtype=t),
         "gate": normal(g, rows // per, C, std=1.0, dtype=t), "post": 1.0 + normal(g, C, std=0.3),
         "pre": 1.0 + normal(g, C, std=0.3)}
    return {n: v if n == "x" or n in parts else None for n, v in p.items()}


def call(p, scale=0.5, activation="silu", eps=1e-5):
    c = {n: None if v is None else v.cuda() for n, v in p.items()}
    return dict(x=c["x"], gate=c["gate"], post_weight=c["post"], pre_weight=c["pre"], scale=scale,
                activation=activation if p["gate"] is not None else None, eps=eps), c["residual"]


def check(ssm, p, scale=0.5, activation="silu", eps=1e-5):
    kw, residual = call(p, scale, activation, eps)
    activation = kw["activation"]
    y, h = ssm.block_norm(residual=residual, **kw)
    torch.cuda.synchronize()
    bf16 = p["x"].dtype == torch.bfloat16
    q = {n: None if v is None else f64(v) for n, v in p.items()}
    ref = R.block_h_ref(q["x"], q["residual"], q["gate"], q["post"], scale, activation, eps)
    term = R.block_h_ref(q["x"], None, q["gate"], q["post"], scale, activation, eps)
    within("h", h, ref, np.abs(term) + np.abs(ref), 48, bf16)
    if y is not None:
        ref = R.block_norm_ref(f64(h), q["pre"], eps)
        within("y", y, ref, np.abs(ref), 30, bf16)
    else:
        assert q["pre"] is None
    g, t = generator(9), p["x"].dtype
    dy = None if p["pre"] is None else normal(g, *p["x"].shape, std=1.0, dtype=t)
    dh = normal(g, *p["x"].shape, std=1.0, dtype=t)
    got = ssm.block_norm_bwd(h=h, dy=None if dy is None else dy.cuda(), dh=dh.cuda(), **kw)
    torch.cuda.synchronize()
    names = {"x", "residual"} | {n for n, v in (("gate", p["gate"]), ("post_weight", p["post"]), ("pre_weight", p["pre"])) if v is not None}
    assert set(got) == names
    a = (q["x"], f64(h), None if dy is None else f64(dy), f64(dh), q["gate"], q["post"], q["pre"], scale, activation, eps)
    ref, size = R.block_norm_ref_backward(*a), sizes(*a)
    for n in names:
        rows = n in ("x", "residual", "gate")
        within("d" + n, got[n], ref[n], size[n], 160 + (0 if n in ("x", "residual") else 32), bf16 and rows)


def sizes(x, h, dy, dh, gate, post, pre, scale, activation, eps):
    """The gradients' terms added up by their absolute values."""
    s = {"residual": np.abs(dh)}
    back = lambda d, v: R.unit(v, eps)[1] * (d + np.abs(R.unit(v, eps)[0]) * np.mean(d * np.abs(R.unit(v, eps)[0]), -1, keepdims=True))  # noqa: E731
    if pre is not None:
        s["pre_weight"] = np.abs(dy * R.unit(h, eps)[0]).sum(0)
        s["residual"] = s["residual"] + back(np.abs(dy * pre), h)
    n = np.abs(x) if post is None else np.abs(R.unit(x, eps)[0] * post)
    d = scale * s["residual"]
    if gate is not None:
        a, slope = R.act(activation, gate)
        per = x.shape[0] // gate.shape[0]
        s["gate"] = (d * n).reshape(gate.shape[0], per, -1).sum(1) * (np.abs(slope) + (0.1 if activation else 0))
        d = d * np.repeat(np.abs(a), per, 0)
    if post is not None:
        s["post_weight"] = (d * np.abs(R.unit(x, eps)[0])).sum(0)
        d = back(d * np.abs(post), x)
    s["x"] = d
    return s


@pytest.mark.parametrize("rows,C,per", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("activation", [None, "silu", "sigmoid"])
def test_block_norm(ssm, rows, C, per, activation, dtype):
    check(ssm, draw(rows, C, per, dtype), activation=activation)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("parts", [(), ("pre",), ("post",), ("residual", "pre"), ("gate",), ("gate", "post"), ("residual", "post"),
                                   ("residual", "gate", "pre")])
@pytest.mark.parametrize("per", [1, 10])
def test_parts(ssm, parts, per, dtype):
    check(ssm, draw(40, 264, per, dtype, parts), scale=0.25)


def test_gradients_are_differences(ssm):
    """As for the scan: 1e-4 of the size."""
    p = draw(20, 64, 5, "f32")
    kw, residual = call(p)
    t = dict(kw, residual=residual)
    dy, dh = (normal(generator(i), 20, 64).cuda() for i in (1, 2))
    h = ssm.block_norm(**t)[1]
    g = ssm.block_norm_bwd(h=h, dy=dy, dh=dh, **kw)
    for i, n in enumerate(("x", "residual", "gate", "post_weight", "pre_weight")):
        d = normal(generator(20 + i), *t[n].shape, std=0.1).cuda()
        slopes = []
        for step in (2.0 ** -5, 2.0 ** -6):
            loss = []
            for k in (1.0, -1.0):
                y, h = ssm.block_norm(**{**t, n: t[n] + k * step * d})
                loss.append(float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum()))
            slopes.append((loss[0] - loss[1]) / (2 * step))
        slope, want = (4 * slopes[1] - slopes[0]) / 3, float((g[n].double() * d.double()).sum())
        assert abs(slope - want) <= 1e-4 * float(y.double().norm() * dy.double().norm() + h.double().norm() * dh.double().norm()), n


def test_gate_shapes(ssm):
    """A gate for every token, each sequence, or all: broadcast over [B, T, C]."""
    B, T, C = 3, 10, 64
    g = generator(4)
    x, gate = normal(g, B, T, C, std=1.0).cuda(), normal(g, B, T, C, std=1.0).cuda()
    for small in (gate, gate[:, :1].contiguous(), gate[0, :1].contiguous(), gate[0, 0].contiguous()):
        full = small.expand(B, T, C).contiguous()
        a, b = ssm.block_norm(x, gate=small, activation="silu")[1], ssm.block_norm(x, gate=full, activation="silu")[1]
        ga = ssm.block_norm_bwd(x, None, dh=x, gate=small, activation="silu")
        gb = ssm.block_norm_bwd(x, None, dh=x, gate=full, activation="silu")
        torch.cuda.synchronize()
        assert bits(a, b) and bits(ga["x"], gb["x"]) and ga["gate"].shape == small.shape
        want = gb["gate"].double().sum_to_size(small.shape if small.dim() == 3 else (1, 1, C)).reshape(small.shape)
        # chains of up to 30 float32 terms, each off by 16 u
        assert torch.all((ga["gate"] - want).abs() <= 48 * U * gb["gate"].abs().double().sum((0, 1)).max())


def test_in_place(ssm):
    for dtype in ("f32", "bf16"):
        kw, residual = call(draw(40, 2048, 1, dtype))
        y, h = ssm.block_norm(residual=residual, **kw)
        for name in ("x", "residual"):
            x, r = kw["x"].clone(), residual.clone()
            to = x if name == "x" else r
            y2, h2 = ssm.block_norm(**dict(kw, x=x), residual=r, h=to)
            assert h2 is to and bits(y, y2) and bits(h, h2)
        want = ssm.block_norm_bwd(h=h, dy=y, dh=residual, **kw)
        dy, dh = y.clone(), residual.clone()
        got = ssm.block_norm_bwd(h=h, dy=dy, dh=dh, out=dy, residual_out=dh, **kw)
        torch.cuda.synchronize()
        assert got["x"] is dy and got["residual"] is dh and all(bits(got[n], want[n]) for n in want)
        assert "residual" not in ssm.block_norm_bwd(h=h, dy=y, dh=residual, want_residual=False, **kw)


def test_rows_of_their_own(ssm):
    """What is not finite stays in its row; rows of zeros stay finite."""
    p = draw(6, 256, 1, "f32")
    p["x"][2, 7], p["residual"][4, 9], p["x"][5], p["residual"][5] = float("nan"), float("inf"), 0, 0
    kw, residual = call(p)
    y, h = ssm.block_norm(residual=residual, **kw)
    torch.cuda.synchronize()
    good = [0, 1, 3, 5]
    assert torch.isfinite(y[good]).all() and torch.isnan(y[2]).all() and torch.isnan(y[4, 9])
    assert not y[5].any()


def test_empty(ssm):
    kw, residual = call(draw(4, 64, 1, "f32"))
    e = dict(kw, x=kw["x"][:0], gate=kw["gate"][:0])
    y, h = ssm.block_norm(residual=residual[:0], **e)
    g = ssm.block_norm_bwd(h=h, dy=y, **e)
    torch.cuda.synchronize()
    assert y.shape == (0, 64) and g["gate"].shape == (0, 64) and not g["post_weight"].any() and not g["pre_weight"].any()


def test_many_rows(ssm):
    """More rows than a launch of one workgroup each could hold in 2^24: both ends and the middle."""
    rows = 2 ** 22 + 4
    x = normal(generator(3), 64, 64, std=1.0, dtype=torch.bfloat16).cuda()
    big = x.repeat(rows // 64 + 1, 1)[:rows]
    w = torch.ones(64, device="cuda")
    y, h = ssm.block_norm(big, residual=big, post_weight=w, pre_weight=w)
    want, _ = ssm.block_norm(x, residual=x, post_weight=w, pre_weight=w)
    torch.cuda.synchronize()
    for at in (0, 2 ** 21, 2 ** 22 - 64):
        assert bits(y[at:at + 64], want)
    g = ssm.block_norm_bwd(big, h, dy=y, gate=x[:1], post_weight=w, pre_weight=w)
    torch.cuda.synchronize()
    assert torch.isfinite(g["post_weight"]).all() and bits(g["x"][:64], g["x"][2 ** 22 - 64:2 ** 22])


def test_graph_and_streams(ssm):
    kw, residual = call(draw(60, 520, 20, "bf16"))

    def run(**s):
        y, h = ssm.block_norm(residual=residual, **kw, **s)
        g = ssm.block_norm_bwd(h=residual, dy=residual, dh=residual, **kw, **s)
        return [y, h, *(g[n] for n in sorted(g))]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    side = torch.cuda.Stream()
    for _ in range(3):
        kw["x"].mul_(-0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, other = run(), run(stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, other):
            assert bits(a, b) and bits(a, c)


def test_gates_of_leading_dimensions(ssm):
    """Rows counted by leading dimensions of x, with and without ones behind them: bit for bit the gate of every row."""
    g = generator(3)
    x = normal(g, 2, 3, 4, 64, std=1.0).cuda()
    gate = normal(g, 2, 3, 1, 64, std=1.0).cuda()
    want = ssm.block_norm(x, gate=gate.expand(2, 3, 4, 64).contiguous(), activation="silu")[1]
    for small in (gate, gate[:, :, 0], gate.view(6, 64)):
        assert bits(ssm.block_norm(x, gate=small, activation="silu")[1], want)
    one = gate[:, :1]
    want = ssm.block_norm(x, gate=one.expand(2, 3, 4, 64).contiguous(), activation="sigmoid")[1]
    for small in (one.contiguous(), one[:, 0, 0].contiguous(), one[:, 0].contiguous()):
        assert bits(ssm.block_norm(x, gate=small, activation="sigmoid")[1], want)
