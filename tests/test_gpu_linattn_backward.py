"""linattn.bwd against the oracle's gradients (which CPU tests hold against
differences) and against differences of linattn.fwd itself."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import TYPES, bits, check, f64, generator, normal, say
from tests.test_gpu_linattn import cuda, inputs, linattn  # noqa: F401

pytestmark = pytest.mark.gpu


def with_gradients(x, seed, dtype, states=True):
    g = generator(seed)
    B, T, H, K = x["q"].shape
    V = x["v"].shape[3]
    x["do"] = normal(g, B, T, H, V, dtype=TYPES[dtype])
    x["ds_out"] = normal(g, B, H, K, V, std=0.3) if states else None
    if not states:
        x["s_in"] = None
    return x


def reference(x, scale, lengths=None):
    a = {n: None if t is None else f64(t) for n, t in x.items()}
    ab = {n: None if t is None else (t if n == "log_decay" else np.abs(t)) for n, t in a.items()}
    return [R.linattn_ref_backward(y["q"], y["k"], y["v"], y["log_decay"], y["do"], s, lengths, y["s_in"], y["ds_out"])
            for y, s in ((a, scale), (ab, abs(scale)))]


def call(linattn, d, scale=1.0, **kw):
    return linattn.bwd(d["q"], d["k"], d["v"], d["log_decay"], d["do"], scale=scale, s_in=d["s_in"],
                       ds_out=d["ds_out"], **kw)


CASES = [(2, 1, 3, 64, 64), (1, 5, 2, 8, 128), (2, 64, 2, 64, 64), (2, 65, 3, 72, 24), (1, 130, 2, 128, 128),
         (1, 300, 2, 40, 96), (1, 1100, 1, 64, 64)]


@pytest.mark.parametrize("B,T,H,K,V", CASES)
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_matches_oracle(linattn, B, T, H, K, V, dtype, grad):  # noqa: F811
    say(f"[linattn] B={B} T={T} H={H} K={K} V={V} {dtype}->{grad}")
    for states in (True, False):
        x = with_gradients(inputs(T, B, T, H, K, V, dtype), T + 1, dtype, states)
        g = call(linattn, cuda(x), 0.7, want_ds_in=states, grad_dtype=TYPES[grad])
        torch.cuda.synchronize()
        ref, size = reference(x, 0.7)
        assert set(g) == ({"q", "k", "v", "s_in"} if states else {"q", "k", "v"})
        for n in g:
            check(f"d{n}", g[n], ref[n], size[n], T, max(K, V), grad == "bf16" and n != "s_in")


@pytest.mark.parametrize("T,lengths", [(3, [3, 0, 1]), (200, [0, 1, 64, 65, 200]), (1500, [1500, 0, 700])])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f32", "f32")])
def test_padded_batch(linattn, T, lengths, dtype, grad):  # noqa: F811
    """NaN behind a sequence is not read; gradients there are zero."""
    x = with_gradients(inputs(T, len(lengths), T, 2, 64, 40, dtype), T, dtype)
    ref, size = reference(x, 1.0, lengths)
    for b, n in enumerate(lengths):
        for t in ("q", "k", "v", "do"):
            x[t][b, n:] = float("nan")
    g = call(linattn, cuda(x), lengths=torch.tensor(lengths, dtype=torch.int32).cuda(), want_ds_in=True,
             grad_dtype=TYPES[grad])
    torch.cuda.synchronize()
    for n in g:
        check(f"d{n}", g[n], ref[n], size[n], T, 64, grad == "bf16" and n != "s_in")


@pytest.mark.parametrize("T", [100, 1400])
def test_decays(linattn, T):  # noqa: F811
    decay = [0.0, -1e-5, -30.0, -float("inf"), 1e-3]
    x = with_gradients(inputs(T, 1, T, 5, 64, 64, "f32", decay=decay), T, "f32")
    g = call(linattn, cuda(x), want_ds_in=True)
    ref, size = reference(x, 1.0)
    for n in g:
        check(f"d{n}", g[n], ref[n], size[n], T, 64, False)


def test_equals_differences_of_the_forward(linattn):  # noqa: F811
    """Along a random direction d: (L(x + e d) - L(x - e d)) / 2e, exact for the
    linear arguments one at a time, against the gradient's product with d.
    L sums T H V + K V products of outputs that are off by 1e-6 of their norm:
    tolerance 2 * 1e-6 |L|/e summed in quadrature, with |d| = |x| and e = 1."""
    x = with_gradients(inputs(11, 1, 150, 2, 64, 64, "f32"), 12, "f32")
    d = cuda(x)
    g = call(linattn, d, want_ds_in=True)

    def parts(**new):
        y = dict(d, **new)
        o, S = linattn.fwd(y["q"], y["k"], y["v"], y["log_decay"], s_in=y["s_in"], want_state=True)
        return o.double(), S.double()

    for i, n in enumerate(("q", "k", "v", "s_in")):
        step = normal(generator(20 + i), *x[n].shape).cuda()
        (o1, S1), (o0, S0) = parts(**{n: d[n] + step}), parts(**{n: d[n] - step})
        slope = float(((o1 - o0) * d["do"].double()).sum() + ((S1 - S0) * d["ds_out"].double()).sum()) / 2
        want = float((g[n].double() * step.double()).sum())
        size = float(o1.norm() * d["do"].norm() + S1.norm() * d["ds_out"].norm())
        say(f"[linattn] d{n}: difference {slope:.8g}, gradient {want:.8g}, size {size:.3g}")
        assert abs(slope - want) <= 3e-6 * size


@pytest.mark.parametrize("T", [7, 100, 1400, 2500])
def test_layouts_do_not_matter(linattn, T):  # noqa: F811
    """Inputs and gradients as slices of one buffer each; heads that share keys; states in place."""
    B, H, K = 2, 3, 64
    x = with_gradients(inputs(T, B, T, H, K, K, "bf16"), T, "bf16")
    d = cuda(x)
    want = call(linattn, d, want_ds_in=True, grad_dtype=torch.bfloat16)
    fused = torch.stack([d["q"], d["k"], d["v"], d["do"]], 2)
    grads = torch.full((B, T, 3, H, K), 5.0, dtype=torch.bfloat16, device="cuda")
    ds = d["ds_out"].clone()
    e = dict(d, q=fused[:, :, 0], k=fused[:, :, 1], v=fused[:, :, 2], do=fused[:, :, 3], ds_out=ds)
    g = call(linattn, e, out={"q": grads[:, :, 0], "k": grads[:, :, 1], "v": grads[:, :, 2], "s_in": ds})
    for n in want:
        assert bits(g[n], want[n]), n
    by_head = {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v", "do")}
    g = call(linattn, dict(d, **by_head), want_ds_in=True, grad_dtype=torch.bfloat16)
    for n in want:
        assert bits(g[n], want[n]), n
    shared = d["k"][:, :, :1].expand(B, T, H, K)
    a = call(linattn, dict(d, k=shared))
    b = call(linattn, dict(d, k=shared.contiguous()))
    for n in a:
        assert bits(a[n], b[n]), n


@pytest.mark.parametrize("K,V", [(128, 40), (40, 128)])
def test_wide_and_narrow_sweeps(linattn, K, V):  # noqa: F811
    """Many float32 heads whose keys and values differ in width; states in place."""
    B, T, H = 20, 300, 5
    x = with_gradients(inputs(7, B, T, H, K, V, "f32"), 8, "f32")
    d = cuda(x)
    ds = d["ds_out"].clone()
    g = call(linattn, dict(d, ds_out=ds), 0.7, out={"s_in": ds}, grad_dtype=torch.float32)
    want = call(linattn, d, 0.7, want_ds_in=True, grad_dtype=torch.float32)
    torch.cuda.synchronize()
    ref, size = reference(x, 0.7)
    for n in ref:
        assert bits(g[n], want[n]), n
        check(f"d{n}", g[n], ref[n], size[n], T, 128, False)


def test_no_tokens(linattn):  # noqa: F811
    x = cuda(with_gradients(inputs(1, 2, 1, 2, 64, 32, "bf16"), 1, "bf16"))
    e = dict(x, **{n: x[n][:, :0] for n in ("q", "k", "v", "do")})
    g = call(linattn, e, want_ds_in=True)
    assert g["q"].shape == (2, 0, 2, 64) and bits(g["s_in"], x["ds_out"])
    assert torch.all(call(linattn, dict(e, ds_out=None), want_ds_in=True)["s_in"] == 0)


@pytest.mark.parametrize("T", [60, 2500])
def test_graphs_and_streams(linattn, T):  # noqa: F811
    x = [cuda(with_gradients(inputs(T + i, 1, T, 2, 64, 64, "bf16"), i, "bf16")) for i in range(2)]
    graphs, outs = [], []
    for d in x:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(linattn, d, want_ds_in=True)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(linattn, d, want_ds_in=True))
        graphs.append(g)
    side = torch.cuda.Stream()
    for rep in range(3):
        for d in x:
            d["do"].mul_(-0.5)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for d, out in zip(x, outs):
            for eager in (call(linattn, d, want_ds_in=True), call(linattn, d, want_ds_in=True, stream=side)):
                torch.cuda.synchronize()
                for n in eager:
                    assert bits(eager[n], out[n]), (rep, n)
