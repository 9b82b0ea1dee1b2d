"""The operators together, as a layer runs them: norm between blocks, x and z
as slices of one projection, convolution, steps and state matrices as slices of another, scan
with its gate; a padded prompt batch, then single tokens, which continue it;
the training pass back through all of it; a decode step as one captured graph."""
import numpy as np
import pytest
import torch

from oracle import ssm_oracle as R
from tests.ssm_util import BF, U, bits, cuda, f64, generator, normal, say

pytestmark = pytest.mark.gpu

B, C, D, N, W = 3, 64, 128, 16, 4


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


def parameters():
    g = generator(70)
    return {"pre": 1 + normal(g, C, std=0.1), "post": 1 + normal(g, C, std=0.1), "conv": normal(g, D, W), "bias": normal(g, D, std=0.1),
            "A": -torch.exp(normal(g, D, N)) * torch.arange(1, N + 1), "skip": 1 + normal(g, D, std=0.1),
            "dt_bias": normal(g, D, std=1.0) - 4}


def inputs(T, dtype):
    """What projections (not part of this) hand the layer: x and z, then dt, B and C; also the block's own output."""
    g = generator(T)
    return {"xz": normal(g, B, T, 2 * D, std=1.0, dtype=dtype), "rest": normal(g, B, T, D + 2 * N, dtype=dtype),
            "out": normal(g, B, T, C, std=1.0, dtype=dtype), "res": normal(g, B, T, C, std=1.0, dtype=dtype),
            "gate": normal(g, B, T, C, dtype=dtype)}


def parts(x):
    rest = x["rest"]
    state = lambda a: rest[..., a:a + N].unflatten(2, (1, N))  # noqa: E731
    return x["xz"][..., :D], x["xz"][..., D:], rest[..., :D], state(D), state(D + N)


def layer(ssm, p, x, lengths=None, states=(None, None), out=(None, None)):
    """(u, y, conv state, scan state, normalised, h) of whatever tokens x holds."""
    a, z, dt, Bm, Cm = parts(x)
    n, h = ssm.block_norm(x["out"], residual=x["res"], gate=x["gate"], post_weight=p["post"], pre_weight=p["pre"],
                          scale=0.5, activation="sigmoid")
    u, c = ssm.conv(a, p["conv"], p["bias"], lengths=lengths, s_in=states[0], s_out=out[0], want_state=True)
    y, s = ssm.scan(u, dt, p["A"], Bm, Cm, D=p["skip"], z=z, dt_bias=p["dt_bias"], lengths=lengths, s_in=states[1],
                    s_out=out[1], want_state=True)
    return u, y, c, s, n, h


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens(ssm, dtype):
    T, steps, lengths = 140, 5, [140, 2, 77]
    p = parameters()
    q = cuda(p)
    x = inputs(T + steps, dtype)
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    got = [layer(ssm, q, {m: t[:, :T].cuda() for m, t in x.items()}, n)]
    for i in range(steps):
        got.append(layer(ssm, q, {m: t[:, T + i:T + i + 1].cuda() for m, t in x.items()}, None, got[-1][2:4]))
    torch.cuda.synchronize()
    rel = lambda a, b: float(np.linalg.norm(a - b) / np.linalg.norm(b))  # noqa: E731
    r = {m: f64(v) for m, v in p.items()}
    for b, k in enumerate(lengths):
        rows = list(range(k)) + list(range(T, T + steps))
        mine = {m: t[b:b + 1, rows] for m, t in x.items()}
        a, z, dt, Bm, Cm = (f64(t) for t in parts(mine))
        u, y = (torch.cat([got[0][i][b, :k]] + [t[i][b] for t in got[1:]])[None] for i in (0, 1))
        u_ref, c_ref = R.conv_ref(a, r["conv"], r["bias"])
        y_ref, s_ref = R.scan_ref(f64(u), dt, r["A"], Bm, Cm, r["skip"], z, r["dt_bias"])
        e = [rel(f64(u), u_ref), rel(f64(y), y_ref), rel(f64(got[-1][3][b]), s_ref[0])]
        say(f"[layer] sequence {b}: convolution {e[0]:.3g}, scan {e[1]:.3g}, state {e[2]:.3g}")
        tol = 2e-6 if dtype == torch.float32 else BF
        assert e[0] <= tol and e[1] <= tol and e[2] <= 2e-6 and np.array_equal(f64(got[-1][2][b]), c_ref[0])
        assert not f64(got[0][1][b, k:]).any() and not f64(got[0][0][b, k:]).any()
        flat = lambda m: f64(mine[m][0])  # noqa: E731
        h_ref = R.block_h_ref(flat("out"), flat("res"), flat("gate"), r["post"], 0.5, "sigmoid")
        h = torch.cat([got[0][5][b, :k]] + [t[5][b] for t in got[1:]])
        v = torch.cat([got[0][4][b, :k]] + [t[4][b] for t in got[1:]])
        assert rel(f64(h), h_ref) <= tol and rel(f64(v), R.block_norm_ref(f64(h), r["pre"])) <= tol


def test_training_pass(ssm):
    """Gradients of all parameters and inputs through convolution, scan and norm equal differences along random
    directions: the calls' float32 errors of 2e-7 of the loss's size over a step of 2^-6, with both orders below taken out."""
    T = 130
    p, x = cuda(parameters()), {m: t.cuda() for m, t in inputs(T, torch.float32).items()}
    g = generator(8)
    dy, gate, weight = normal(g, B, T, D).cuda(), normal(g, B, 1, D).cuda(), (1 + normal(g, D, std=0.1)).cuda()

    def forward(p, x):
        u, y = layer(ssm, p, x)[:2]
        return u, y, ssm.block_norm(y, gate=gate, post_weight=weight, activation="silu")[1]

    u, y, h = forward(p, x)
    a, z, dt, Bm, Cm = parts(x)
    gn = ssm.block_norm_bwd(y, None, dh=dy, gate=gate, post_weight=weight, activation="silu", want_residual=False)
    gs = ssm.scan_bwd(u, dt, p["A"], Bm, Cm, gn["x"], D=p["skip"], z=z, dt_bias=p["dt_bias"])
    gc = ssm.conv_bwd(a, p["conv"], gs["x"], p["bias"])
    got = {"conv": gc["weight"], "bias": gc["bias"], "A": gs["A"], "skip": gs["D"], "dt_bias": gs["dt_bias"],
           "xz": torch.cat((gc["x"], gs["z"]), 2), "rest": torch.cat((gs["dt"], gs["B"].flatten(2), gs["C"].flatten(2)), 2)}
    for i, (n, v) in enumerate(got.items()):
        base = p if n in p else x
        d = normal(generator(30 + i), *base[n].shape, std=0.1).cuda()
        slopes = []
        for step in (2.0 ** -5, 2.0 ** -6):
            up, down = (forward(*({**t, n: t[n] + k * step * d} if t is base else t for t in (p, x)))[2].double() for k in (1.0, -1.0))
            slopes.append(float(((up - down) * dy.double()).sum()) / (2 * step))
        slope, want = (4 * slopes[1] - slopes[0]) / 3, float((v.double() * d.double()).sum())
        size = float(up.norm() * dy.double().norm())
        say(f"[layer] d{n}: difference {slope:.8g}, gradient {want:.8g}, size {size:.3g}")
        assert abs(slope - want) <= 1e-4 * size


def test_decode_step_as_a_graph(ssm):
    """One captured step whose states are updated in place, replayed for token after token."""
    p, x = cuda(parameters()), {n: t.cuda() for n, t in inputs(6, torch.bfloat16).items()}
    now = {n: t[:, :1].clone() for n, t in x.items()}
    states = [torch.zeros(B, W - 1, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, D, N, device="cuda")]
    eager = [t.clone() for t in states]
    layer(ssm, p, now, None, eager)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(ssm, p, now, None, states, states)
    for t in range(6):
        for n in now:
            now[n].copy_(x[n][:, t:t + 1])
        torch.cuda.synchronize()
        graph.replay()
        want = layer(ssm, p, now, None, eager)
        eager = [want[2], want[3]]
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert bits(a, b), t
