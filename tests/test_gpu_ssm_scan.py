"""ssm.scan and scan_bwd against the oracle: every number of states a lane can
hold, groups, lengths from none to several blocks, padding, states, strides."""
import numpy as np
import pytest
import torch

from tests import ssm_util as S
from tests.ssm_util import bits, f64, generator, normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


# B, T, D, N, G
SHAPES = [(1, 1, 8, 8, 1), (3, 4, 24, 16, 1), (2, 5, 16, 16, 2), (1, 31, 40, 24, 1), (2, 33, 72, 64, 3), (1, 64, 32, 32, 1),
          (2, 128, 48, 16, 2), (1, 129, 136, 8, 1), (3, 257, 56, 16, 1), (1, 130, 64, 40, 4), (1, 700, 8, 16, 1),
          (2, 300, 80, 64, 1), (1, 1025, 16, 32, 2)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,N,G", SHAPES)
def test_scan(ssm, B, T, D, N, G, dtype):
    p = S.inputs(T + N, B, T, D, N, G, dtype)
    y, s = ssm.scan(**S.cuda(p), want_state=True)
    torch.cuda.synchronize()
    S.check_scan(f"{B}x{T}x{D} N{N} G{G} {dtype}", p, y, s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 40, 200])
@pytest.mark.parametrize("missing", [("z",), ("D", "dt_bias"), ("s_in", "z", "D"), ("dt_bias", "s_in")])
def test_optional_inputs(ssm, T, missing, dtype):
    p = S.inputs(T, 2, T, 24, 16, 1, dtype)
    for n in missing:
        p[n] = None
    y, s = ssm.scan(**S.cuda(p), want_state=True)
    dy, ds = normal(generator(1), 2, T, 24, dtype=y.dtype), normal(generator(2), 2, 24, 16)
    g = ssm.scan_bwd(**S.cuda(p), dy=dy.cuda(), ds_out=ds.cuda(), want_ds_in=True)
    torch.cuda.synchronize()
    assert set(g) == {"x", "dt", "A", "B", "C", "s_in"} | ({"D", "z", "dt_bias"} - set(missing))
    S.check_scan("without " + " ".join(missing), p, y, s)
    S.check_scan_bwd("without " + " ".join(missing), p, g, dy, ds)


@pytest.mark.parametrize("T", [2, 70])
def test_plain_steps(ssm, T):
    """Without softplus the steps are as given."""
    p = S.inputs(T, 2, T, 16, 16, 1, "f32")
    p["dt"], p["dt_bias"] = p["dt"].abs() * 0.1, p["dt_bias"].abs() * 0.01
    y, s = ssm.scan(**S.cuda(p), softplus=False, want_state=True)
    dy = normal(generator(1), 2, T, 16)
    g = ssm.scan_bwd(**S.cuda(p), dy=dy.cuda(), softplus=False)
    torch.cuda.synchronize()
    S.check_scan("plain steps", p, y, s, softplus=False)
    S.check_scan_bwd("plain steps", p, g, dy, softplus=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,lengths", [(4, [4, 0, 2]), (130, [130, 1, 0]), (300, [128, 300, 129]), (260, [-5, 1000, 256])])
def test_padded(ssm, T, lengths, dtype):
    """Rows behind a sequence are not read (here NaN), their outputs are zero, states are left at its end."""
    p = S.inputs(T, 3, T, 24, 16, 1, dtype)
    q, n = S.cuda(p), torch.tensor(lengths, dtype=torch.int32).cuda()
    dy, ds = normal(generator(1), 3, T, 24, dtype=p["x"].dtype), normal(generator(2), 3, 24, 16)
    dyc = dy.cuda()
    for b, k in enumerate(lengths):
        for t in [q[m] for m in ("x", "dt", "B", "C", "z")] + [dyc]:
            t[b, max(k, 0):] = float("nan")
    y, s = ssm.scan(**q, lengths=n, want_state=True, out=torch.full_like(q["x"], 7.0))
    g = ssm.scan_bwd(**q, dy=dyc, ds_out=ds.cuda(), lengths=n, want_ds_in=True)
    torch.cuda.synchronize()
    S.check_scan("padded", p, y, s, lengths)
    S.check_scan_bwd("padded", p, g, dy, ds, lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,T,D,N,G", SHAPES)
def test_gradients(ssm, B, T, D, N, G, dtype):
    p = S.inputs(T + N, B, T, D, N, G, dtype)
    dy = normal(generator(5), B, T, D, std=1.0, dtype=p["x"].dtype)
    ds = normal(generator(6), B, D, N, std=0.3)
    g = ssm.scan_bwd(**S.cuda(p), dy=dy.cuda(), ds_out=ds.cuda(), want_ds_in=True)
    torch.cuda.synchronize()
    S.check_scan_bwd(f"{B}x{T}x{D} N{N} G{G} {dtype}", p, g, dy, ds)


def test_gradients_are_differences(ssm):
    """Slopes of the forward call along random directions.  Each of its outputs errs by 2e-7 of itself (2-norm), so
    the loss by 2e-7 |y| |dy| at most, and the difference over a step of 2^-5 by that over 2^-5; its third order adds 2^-10 / 6
    of a slope of slopes, halved steps take away: both sides of 1e-4 of the size."""
    p = S.inputs(3, 2, 140, 16, 16, 1, "f32")
    q = S.cuda(p)
    dy = normal(generator(1), 2, 140, 16).cuda()
    g = ssm.scan_bwd(**q, dy=dy)
    h = 2.0 ** -5
    for i, n in enumerate(("x", "dt", "A", "B", "C", "D", "z", "dt_bias")):
        d = normal(generator(20 + i), *p[n].shape, std=0.1).cuda()
        slopes = []
        for step in (h, h / 2):
            up, down = (ssm.scan(**{**q, n: q[n] + k * step * d})[0].double() for k in (1.0, -1.0))
            slopes.append(float(((up - down) * dy.double()).sum()) / (2 * step))
        slope, want = (4 * slopes[1] - slopes[0]) / 3, float((g[n].double() * d.double()).sum())
        size = float(up.norm() * dy.double().norm())
        S.say(f"[ssm] d{n}: difference {slope:.7g}, gradient {want:.7g}, size {size:.3g}")
        assert abs(slope - want) <= 1e-4 * size


def test_slices_of_projections(ssm):
    """x and z of one buffer, dt, B and C of another, outputs into slices: as contiguous ones, bit for bit."""
    B, T, D, N = 2, 150, 24, 16
    p = S.cuda(S.inputs(9, B, T, D, N, 1, "bf16"))
    dy = normal(generator(1), B, T, D, dtype=torch.bfloat16).cuda()
    xz = torch.cat((p["x"], p["z"]), 2)
    rest = torch.cat((p["dt"], p["B"].flatten(2), p["C"].flatten(2)), 2)
    s = dict(p, x=xz[..., :D], z=xz[..., D:], dt=rest[..., :D], B=rest[..., D:D + N].unflatten(2, (1, N)),
             C=rest[..., D + N:].unflatten(2, (1, N)))
    both = torch.empty(B, T, 2 * D, dtype=torch.bfloat16, device="cuda")
    y, st = ssm.scan(**s, want_state=True, out=both[..., D:])
    want, want_s = ssm.scan(**p, want_state=True)
    assert bits(y, want) and bits(st, want_s)
    gxz, grest = torch.empty_like(xz), torch.empty_like(rest)
    out = {"x": gxz[..., :D], "z": gxz[..., D:], "dt": grest[..., :D], "B": grest[..., D:D + N].unflatten(2, (1, N)),
           "C": grest[..., D + N:].unflatten(2, (1, N))}
    g, w = ssm.scan_bwd(**s, dy=dy, out=out), ssm.scan_bwd(**p, dy=dy)
    torch.cuda.synchronize()
    for n in w:
        assert bits(g[n], w[n]), n
    # a distance of 0: B and C of every batch item alike
    e = dict(p, B=p["B"][:1].expand(B, -1, -1, -1), C=p["C"][:, :1].expand(-1, T, -1, -1))
    c = {n: v if v is None else v.contiguous() for n, v in e.items()}
    assert bits(ssm.scan(**e)[0], ssm.scan(**c)[0])
    g, w = ssm.scan_bwd(**e, dy=dy), ssm.scan_bwd(**c, dy=dy)
    torch.cuda.synchronize()
    assert all(bits(g[n], w[n]) for n in w)


@pytest.mark.parametrize("T", [1, 3, 140])
def test_state_in_place(ssm, T):
    p = S.cuda(S.inputs(7, 2, T, 16, 16, 1, "f32"))
    y, s = ssm.scan(**p, want_state=True)
    q = dict(p, s_in=p["s_in"].clone())
    y2, s2 = ssm.scan(**q, s_out=q["s_in"])
    assert s2 is q["s_in"] and bits(y, y2) and bits(s, s2)
    dy, ds = torch.ones_like(y), torch.ones_like(s)
    g = ssm.scan_bwd(**p, dy=dy, ds_out=ds, want_ds_in=True)
    g2 = ssm.scan_bwd(**p, dy=dy, ds_out=ds, out={"s_in": ds})
    torch.cuda.synchronize()
    assert g2["s_in"] is ds and all(bits(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("cut", [1, 4, 100, 128])
def test_pieces(ssm, cut):
    """A sequence in two calls is the sequence in one."""
    p = S.inputs(8, 2, 200, 24, 16, 1, "f32")
    q = S.cuda(p)
    part = lambda a, b: {n: v[:, a:b] if n in ("x", "dt", "B", "C", "z") else v for n, v in q.items()}  # noqa: E731
    y0, s0 = ssm.scan(**part(0, cut), want_state=True)
    y1, s1 = ssm.scan(**dict(part(cut, 200), s_in=s0), want_state=True)
    torch.cuda.synchronize()
    S.check_scan(f"in pieces at {cut}", p, torch.cat((y0, y1), 1), s1)


def test_slow_decays_over_many_steps(ssm):
    """Equal small steps, one token at a time and in one call: a state that lives for tens of thousands of tokens.
    In one call the decay rounds once for each of 32 blocks.  Token by token the state is stored in float32 each time, and a
    decrement of a fraction of its last place is lost or doubled the same way at every token, by up to T u in all, whatever computes
    it: that call is compared with the recurrence in 64 bits whose state is rounded to float32 after every token.  A decay rounded to
    float32 would add 2^-25 T = 2048 u to that; what is allowed is 64 u: steps off by up to 18 u of themselves (X e^-X of it), and
    results next to a tie that round the other way, by 2 u each, at random: 28 u for one in twenty tokens."""
    T, D, N = 4096, 8, 8
    p = S.inputs(1, 1, T, D, N, 1, "f32", slow=True)
    p["dt"] = torch.zeros(1, T, D)
    p["dt_bias"] = torch.linspace(-13.0, -9.0, D)
    p["s_in"] = p["s_in"].abs() + 1
    p["B"] = p["B"] * 1e-3
    q = S.cuda(p)
    a = S.oracle_args(p)
    ref = S.R.scan_ref(**a)[1]
    delta = S.R.step_sizes(a["dt"], a["dt_bias"])
    stored = a["s_in"][0]
    for t in range(T):
        stored = S.R.scan_states(delta[0, t:t + 1], (delta * a["x"])[0, t:t + 1], a["A"], a["Bm"][0, t:t + 1], 1, stored)[1]
        stored = stored.astype(np.float32).astype(np.float64)
    _, s = ssm.scan(**q, want_state=True)
    state = q["s_in"].clone()
    tok = {n: v for n, v in q.items() if n not in ("x", "dt", "B", "C", "z", "s_in")}
    for t in range(T):
        ssm.scan(**tok, **{n: q[n][:, t:t + 1] for n in ("x", "dt", "B", "C", "z")}, s_in=state, s_out=state)
    torch.cuda.synchronize()
    rel = lambda a, r: float(np.linalg.norm(f64(a) - r) / np.linalg.norm(r))  # noqa: E731
    e = rel(s, ref), rel(state, stored[None]), rel(state, ref)
    S.say(f"[ssm] slow decays: one call {e[0]:.3g}, token by token {e[1]:.3g} of stored states, {e[2]:.3g} of exact ones")
    assert e[0] <= 64 * S.U and e[1] <= 64 * S.U and e[2] <= T * S.U


@pytest.mark.parametrize("name", ["x", "dt", "B", "C", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_not_finite(ssm, name, bad):
    """What is not finite reaches no earlier token and no other sequence or channel (B and C: group)."""
    p = S.inputs(2, 2, 200, 32, 16, 2, "f32")
    p[name][1, 150].view(-1)[:2] = bad
    q = S.cuda(p)
    y, s = ssm.scan(**q, want_state=True)
    clean = S.cuda(S.inputs(2, 2, 200, 32, 16, 2, "f32"))
    want, want_s = ssm.scan(**clean, want_state=True)
    torch.cuda.synchronize()
    assert bits(y[0], want[0]) and bits(s[0], want_s[0]) and bits(y[1, :150], want[1, :150])
    spoiled = slice(0, 16) if name in ("B", "C") else slice(0, 2)
    rest = slice(spoiled.stop, 32)
    assert bits(y[1, :, rest], want[1, :, rest]) and bits(s[1, rest], want_s[1, rest])
    later = y[1, 151:, spoiled]
    if name in ("C", "z"):
        assert bits(later, want[1, 151:, spoiled])
    elif name != "dt" or bad != bad:
        assert not torch.isfinite(later).any()
    assert not torch.isfinite(y[1, 150, spoiled]).all()


def test_empty(ssm):
    p = S.cuda(S.inputs(1, 2, 3, 16, 16, 1, "f32"))
    none = {n: v[:, :0] if n in ("x", "dt", "B", "C", "z") else v for n, v in p.items()}
    y, s = ssm.scan(**none, want_state=True)
    ds = torch.randn_like(s)
    g = ssm.scan_bwd(**none, dy=y, ds_out=ds, want_ds_in=True)
    torch.cuda.synchronize()
    assert y.shape == (2, 0, 16) and bits(s, p["s_in"]) and bits(g["s_in"], ds) and not g["A"].any() and not g["D"].any()
    nobody = {n: v if n in ("A", "D", "dt_bias") else v[:0] for n, v in p.items()}
    y, s = ssm.scan(**nobody, want_state=True)
    g = ssm.scan_bwd(**nobody, dy=y)
    torch.cuda.synchronize()
    assert y.shape == (0, 3, 16) and not g["A"].any() and not g["dt_bias"].any()


def test_graph_and_streams(ssm):
    """Captured calls on states in place, replayed between eager ones, and calls on another stream."""
    p = S.cuda(S.inputs(4, 2, 150, 32, 16, 1, "bf16"))
    dy = torch.randn(2, 150, 32, device="cuda").bfloat16()
    tok = {n: v[:, :1].clone() if n in ("x", "dt", "B", "C", "z") else v for n, v in p.items()}

    def run(**kw):
        g = ssm.scan_bwd(**p, dy=dy, want_ds_in=True, **kw)
        return [*ssm.scan(**p, want_state=True, **kw), *(g[n] for n in sorted(g)), *ssm.scan(**tok, want_state=True, **kw)]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    side = torch.cuda.Stream()
    for _ in range(3):
        p["x"].mul_(-0.5)
        tok["x"].add_(0.25)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want, other = run(), run(stream=side)
        torch.cuda.synchronize()
        for a, b, c in zip(out, want, other):
            assert bits(a, b) and bits(a, c)


@pytest.mark.parametrize("D", [2048, 4096 + 64])
def test_many_channels(ssm, D):
    """More workgroups than CUs: ends and middle of batch items against calls of their own channels."""
    p = S.cuda(S.inputs(6, 3, 140, D, 16, 1, "bf16"))
    y, s = ssm.scan(**p, want_state=True)
    for c in (0, D // 2, D - 8):
        part = {n: v[..., c:c + 8] if n in ("x", "dt", "z", "D", "dt_bias") else v[:, c:c + 8] if n == "s_in"
                else v[c:c + 8] if n == "A" else v for n, v in p.items()}
        part = {n: v.contiguous() for n, v in part.items()}
        y2, s2 = ssm.scan(**part, want_state=True)
        torch.cuda.synchronize()
        assert bits(y[..., c:c + 8], y2) and bits(s[:, c:c + 8], s2)


# B, D, G: 408 and 1032 workgroups of 8 channels, more than a chip holds at once, with parts of the last blocks of 16 and 32
# channels left over; T: blocks of 32, 64 and 128 tokens
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("T", [20, 50, 133])
@pytest.mark.parametrize("B,D,G", [(8, 408, 1), (4, 2064, 2)])
def test_wide(ssm, B, D, G, T, N, dtype):
    p = S.inputs(T + N, B, T, D, N, G, dtype)
    lengths = [T, T - 3, 0, 17] * (B // 4)
    dy, ds = normal(generator(5), B, T, D, std=1.0, dtype=p["x"].dtype), normal(generator(6), B, D, N, std=0.3)
    q, n = S.cuda(p), torch.tensor(lengths, dtype=torch.int32).cuda()
    y, s = ssm.scan(**q, lengths=n, want_state=True)
    g = ssm.scan_bwd(**q, dy=dy.cuda(), ds_out=ds.cuda(), lengths=n, want_ds_in=True)
    torch.cuda.synchronize()
    S.check_scan(f"{B}x{T}x{D} N{N} G{G} {dtype}", p, y, s, lengths)
    S.check_scan_bwd(f"{B}x{T}x{D} N{N} G{G} {dtype}", p, g, dy, ds, lengths)
