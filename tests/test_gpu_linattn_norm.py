"""linattn.rms_norm, rms_norm_q8 and rms_norm_bwd against the oracle.

Bounds (u = 2^-24): a sum of C squares is added up by each thread (up to 32
columns), then over at most 9 levels of lanes and waves: 41 u of itself; the
root halves that, and mean, root, quotient and the two products add u each:
30 u |y| covers y.  bfloat16 adds half a step, 2^-8 |y|.  h is one rounding of
an exact sum: equal to torch's bit for bit.  Codes may differ from those of
the exact y only where y / scale is within 60 u of a tie; scales are off by
32 u.  Gradients: the mean of dy w h adds 41 u of its absolute terms; dweight
adds up to rows / groups, 16 + log terms one after another: (rows / 32 + 64) u."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import BF, TYPES, U, bits, f64, generator, normal, say

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8), (3, 64), (33, 72), (100, 128), (19, 136), (65, 256), (35, 264), (5, 504), (7, 520), (300, 2048), (2500, 2048), (2500, 1032), (4, 4104), (9, 8192), (2, 8200),
          (3, 16384), (2100, 512)]


@pytest.fixture(scope="module")
def linattn():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import linattn

    return linattn


def within(name, err, bound):
    worst = float(np.max(err / np.maximum(bound, 1e-37))) if err.size else 0.0
    say(f"[norm] {name}: {worst:.3g} of the bound")
    assert worst <= 1.0, name


def draw(rows, C, dtype, residual=True):
    g = generator(rows * 7 + C)
    return (normal(g, rows, C, std=1.0, dtype=TYPES[dtype]), 1.0 + normal(g, C, std=0.3),
            normal(g, rows, C, std=2.0, dtype=TYPES[dtype]) if residual else None)


@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("residual", [True, False])
def test_norm(linattn, rows, C, dtype, residual):
    x, w, r = draw(rows, C, dtype, residual)
    y, h = linattn.rms_norm(x.cuda(), w.cuda(), 1e-5, residual=None if r is None else r.cuda())
    torch.cuda.synchronize()
    want_h = x if r is None else (x.float() + r.float()).to(x.dtype)
    assert bits(h.cpu(), want_h)
    ref = R.rms_norm_ref(f64(want_h), f64(w), 1e-5)
    within(f"{rows}x{C} {dtype}", np.abs(f64(y) - ref), (30 * U + (BF if dtype == "bf16" else 0)) * np.abs(ref))


@pytest.mark.parametrize("rows,C", SHAPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_q8(linattn, rows, C, group, dtype):
    x, w, r = draw(rows, C, dtype)
    x[0], r[0] = 0, 0      # a row of zeros
    codes, scales, h = linattn.rms_norm_q8(x.cuda(), w.cuda(), 1e-5, residual=r.cuda(), group=group)
    torch.cuda.synchronize()
    want_h = (x.float() + r.float()).to(x.dtype)
    assert bits(h.cpu(), want_h)
    y = R.rms_norm_ref(f64(want_h), f64(w), 1e-5)
    s = R.scales_ref(y, group)
    within(f"scales {rows}x{C}", np.abs(f64(scales) - s), 32 * U * s)
    z = y / np.repeat(s, group or C, -1)[:, :C]
    got = f64(codes)
    low, high = R.e4m3_nearest(np.clip(z * (1 - 60 * U), -448, 448)), R.e4m3_nearest(np.clip(z * (1 + 60 * U), -448, 448))
    assert np.all((got == low) | (got == high))
    say(f"[norm] codes {rows}x{C}: {np.mean(low != high):.2g} next to a tie")
    assert np.all(got[0] == 0) and np.all(f64(scales)[0] == 1)


@pytest.mark.parametrize("rows,C", SHAPES + [(6000, 1024), (3000, 2048)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("stream_gradient", [True, False])
def test_gradients(linattn, rows, C, dtype, stream_gradient):
    g = generator(rows + C)
    h, dy = normal(g, rows, C, std=1.0, dtype=TYPES[dtype]), normal(g, rows, C, std=1.0, dtype=TYPES[dtype])
    dh = normal(g, rows, C, std=1.0, dtype=TYPES[dtype]) if stream_gradient else None
    w = 1.0 + normal(g, C, std=0.3)
    got = linattn.rms_norm_bwd(dy.cuda(), h.cuda(), w.cuda(), 1e-5, dh=None if dh is None else dh.cuda())
    torch.cuda.synchronize()
    a = [f64(dy), f64(h), f64(w)]
    ref = R.rms_norm_ref_backward(*a, 1e-5, None if dh is None else f64(dh))
    rms = np.sqrt(np.mean(a[1] ** 2, -1, keepdims=True) + 1e-5)
    n, dn = np.abs(a[1] / rms), np.abs(a[0] * a[2])
    size = (dn + n * np.mean(dn * n, -1, keepdims=True)) / rms + (0 if dh is None else np.abs(f64(dh)))
    within(f"dx {rows}x{C}", np.abs(f64(got["x"]) - ref["x"]), 120 * U * size + (BF if dtype == "bf16" else 0) * np.abs(ref["x"]))
    total = (np.abs(a[0]) * n).sum(0)
    within(f"dweight {rows}x{C}", np.abs(f64(got["weight"]) - ref["weight"]), (rows / 32 + 96) * U * total)
    rel = np.linalg.norm(f64(got["weight"]) - ref["weight"]) / np.linalg.norm(ref["weight"])
    assert rel <= 1e-6


def test_in_place(linattn):
    for dtype in ("bf16", "f32"):
        x, w, r = (None if t is None else t.cuda() for t in draw(40, 2048, dtype))
        y, h = linattn.rms_norm(x, w, residual=r)
        for name in ("x", "r"):
            x2, r2 = x.clone(), r.clone()
            y2, h2 = linattn.rms_norm(x2, w, residual=r2, h=x2 if name == "x" else r2)
            assert bits(y2, y) and bits(h2, h)
        want = linattn.rms_norm_bwd(y, h, w, dh=r)
        for name in ("dy", "dh"):
            y2, r2 = y.clone(), r.clone()
            g = linattn.rms_norm_bwd(y2, h, w, dh=r2, out=y2 if name == "dy" else r2)
            assert bits(g["x"], want["x"]) and bits(g["weight"], want["weight"])


def test_extremes(linattn):
    """Large and small rows, NaN and infinities stay in their rows; eps keeps zero rows finite."""
    x = normal(generator(1), 6, 256, std=1.0)
    x[1] *= 1e15
    x[2] *= 1e-15
    x[3, 7] = float("nan")
    x[4, 9] = float("inf")
    x[5] = 0
    w = torch.ones(256)
    y, _ = linattn.rms_norm(x.cuda(), w.cuda(), 1e-30)
    codes, scales, _ = linattn.rms_norm_q8(x.cuda(), w.cuda(), 1e-30)
    y = y.cpu()
    for row in (0, 1, 2):
        ref = R.rms_norm_ref(f64(x[row:row + 1]), f64(w), 1e-30)
        within(f"row {row}", np.abs(f64(y[row:row + 1]) - ref), 30 * U * np.abs(ref))
        assert float(codes.float()[row].abs().max()) == 448
    assert torch.isnan(y[3]).all() and torch.isnan(codes.float()[3]).all()
    assert torch.isnan(y[4, 9]) and torch.isnan(codes.float()[4, 9])
    assert torch.all(y[5] == 0) and torch.all(codes.float()[5] == 0) and torch.all(scales[5] == 1)


@pytest.mark.parametrize("group", [0, 128])
def test_tiny_outputs(linattn, group):
    """Outputs below the normal float32 range: scales stay normal, codes finite.

    y errs by 30 U of itself and by two steps of 2^-149 (the products that
    leave the normal range), the code by half a step: 2^-4 of it, or 2^-10."""
    x = normal(generator(2), 3, 384, std=1.0)
    w = torch.tensor([1e-42, 3e-45, 2e-37]).repeat_interleave(128)
    if not group:
        w = w.clamp(max=1e-42)
    codes, scales, _ = linattn.rms_norm_q8(x.cuda(), w.cuda(), 1e-5, group=group)
    y = R.rms_norm_ref(f64(x), f64(w), 1e-5)
    s = R.scales_ref(y, group)
    unit = 2.0 ** -126
    within("scales", np.abs(f64(scales) - s) / unit, 32 * U * s / unit)
    s = np.repeat(s, group or 384, -1)
    got = f64(codes) * s
    assert np.isfinite(got).all()
    within("values", np.abs(got - y) / unit, (2.0 ** -4 * np.abs(y) + 2.0 ** -10 * s + 2.0 ** -148) / unit)


def test_many_rows(linattn):
    """More rows than 2^22, as norms over the channels of a head have: both ends and one in the middle."""
    rows = 2 ** 22 + 5
    x = normal(generator(3), 64, 64, std=1.0, dtype=torch.bfloat16).cuda()
    big = x.repeat(rows // 64 + 1, 1)[:rows]
    w = torch.ones(64, device="cuda")
    y, _ = linattn.rms_norm(big, w)
    want, _ = linattn.rms_norm(x.repeat(40, 1), w)   # the same shape of workgroups
    for at in (0, 2 ** 21, 2 ** 22 - 64, rows - rows % 64):
        n = min(64, rows - at)
        assert bits(y[at:at + n], want[:n])
    g = linattn.rms_norm_bwd(big, big, w)
    assert torch.isfinite(g["weight"]).all() and bits(g["x"][:64], g["x"][2 ** 22 - 64:2 ** 22])


def test_shapes_and_empty(linattn):
    x = normal(generator(2), 3, 5, 64, dtype=torch.bfloat16).cuda()
    w = torch.ones(64, device="cuda")
    y, h = linattn.rms_norm(x, w)
    assert y.shape == x.shape and h is x
    codes, scales, _ = linattn.rms_norm_q8(x, w, group=0)
    assert codes.shape == x.shape and scales.shape == (3, 5, 1)
    assert linattn.rms_norm_bwd(x, x, w)["x"].shape == x.shape
    e = x[:0]
    assert linattn.rms_norm(e, w)[0].shape == e.shape
    g = linattn.rms_norm_bwd(e, e, w)
    assert torch.all(g["weight"] == 0)


def test_graph_and_streams(linattn):
    x, w, r = (t.cuda() for t in draw(64, 2048, "bf16"))
    run = lambda **kw: (linattn.rms_norm(x, w, residual=r, **kw) + linattn.rms_norm_q8(x, w, residual=r, **kw)  # noqa: E731
                        + tuple(linattn.rms_norm_bwd(x, r, w, **kw).values()))
    run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    side = torch.cuda.Stream()
    for _ in range(3):
        x.mul_(-0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = run(stream=side)
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert bits(a, b)
