"""linattn.fwd against the float64 oracle: lengths from one token on, odd
sizes, states in and out, padded batches, strides, streams, graphs."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import TYPES, bits, check, f64, generator, normal, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def linattn():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import linattn

    return linattn


def inputs(seed, B, T, H, K, V, dtype, state=True, decay=None):
    g = generator(seed)
    x = {"q": normal(g, B, T, H, K, dtype=TYPES[dtype]), "k": normal(g, B, T, H, K, dtype=TYPES[dtype]),
         "v": normal(g, B, T, H, V, dtype=TYPES[dtype]),
         "log_decay": torch.tensor(decay if decay is not None else
                                   [float(np.log1p(-2.0 ** -(1 + 8 * (h + 0.5) / H))) for h in range(H)])}
    x["s_in"] = normal(g, B, H, K, V) if state else None
    return x


def cuda(x):
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def reference(x, scale, lengths=None):
    a = {n: None if t is None else f64(t) for n, t in x.items()}
    args = [a["q"], a["k"], a["v"], a["log_decay"], scale, lengths, a["s_in"]]
    size = [np.abs(t) if i in (0, 1, 2, 6) and t is not None else t for i, t in enumerate(args)]
    size[4] = abs(scale)
    return R.linattn_ref(*args), R.linattn_ref(*size)


def run_and_check(linattn, x, scale, out, lengths=None, want_state=True, label=""):
    B, T, H, K = x["q"].shape
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    d = cuda(x)
    o, S = linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=scale, lengths=n, s_in=d["s_in"],
                       want_state=want_state, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    (o_ref, S_ref), (o_size, S_size) = reference(x, scale, lengths)
    check(f"{label} o", o, o_ref, o_size, T, K, out == "bf16")
    if want_state:
        check(f"{label} s_out", S, S_ref, S_size, T, K, False)
    return o, S


CASES = [  # B, T, H, K, V
    (2, 1, 3, 64, 64), (1, 2, 2, 8, 128), (3, 8, 2, 128, 40), (2, 9, 3, 64, 64), (1, 63, 2, 40, 72), (2, 64, 2, 64, 64),
    (2, 65, 3, 72, 24), (1, 127, 2, 128, 128), (2, 130, 1, 96, 64), (1, 300, 2, 64, 96), (1, 1100, 1, 64, 64),
    (1, 1000, 2, 128, 8)]


@pytest.mark.parametrize("B,T,H,K,V", CASES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_matches_oracle(linattn, B, T, H, K, V, dtype, out):
    say(f"[linattn] B={B} T={T} H={H} K={K} V={V} {dtype}->{out}")
    x = inputs(B * 1000 + T, B, T, H, K, V, dtype)
    run_and_check(linattn, x, K ** -0.5, out, label="state in and out")
    x["s_in"] = None
    run_and_check(linattn, x, 1.0, out, want_state=False, label="no state")


@pytest.mark.parametrize("T", [5, 150, 1400])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decays(linattn, T, dtype):
    """a = 1, nearly 1, tiny, 0, and (mildly) growing."""
    x = inputs(7 + T, 1, T, 6, 64, 32, dtype, decay=[0.0, -1e-5, -30.0, -float("inf"), -2900.0, 1e-3])
    run_and_check(linattn, x, 0.5, "f32", label=f"T={T}")


@pytest.mark.parametrize("T,lengths", [(4, [0, 1, 4, 9, -3]), (200, [0, 1, 63, 64, 65]), (200, [200, 199, 128, 129, 10 ** 6]),
                                       (1500, [1500, 0, 700])])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_padded_batch(linattn, T, lengths, dtype, out):
    """Rows behind a sequence hold NaN and must not be read; theirs of o are zero."""
    x = inputs(T, len(lengths), T, 2, 64, 72, dtype)
    for b, n in enumerate(lengths):
        for t in ("q", "k", "v"):
            x[t][b, max(n, 0):] = float("nan")
    clean = {n: t.clone() if t is not None else None for n, t in x.items()}
    for t in ("q", "k", "v"):
        clean[t] = torch.nan_to_num(clean[t])
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    d = cuda(x)
    o, S = linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], scale=0.3, lengths=n, s_in=d["s_in"], want_state=True,
                       out=torch.full((len(lengths), T, 2, 72), float("nan"), dtype=TYPES[out], device="cuda"))
    torch.cuda.synchronize()
    (o_ref, S_ref), (o_size, S_size) = reference(clean, 0.3, lengths)
    check("padded o", o, o_ref, o_size, T, 64, out == "bf16")
    check("padded s_out", S, S_ref, S_size, T, 64, False)
    for b, m in enumerate(lengths):
        assert torch.all(o[b, max(m, 0):] == 0)
        if m <= 0:
            assert bits(S[b], d["s_in"][b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [3, 77, 1300])
def test_layouts_do_not_matter(linattn, dtype, T):
    """Slices of one buffer, heads before tokens, keys shared by the heads, an
    output inside a larger buffer: bit for bit the contiguous call."""
    B, H, K, V = 2, 3, 64, 64
    x = inputs(T, B, T, H, K, V, dtype, state=False)
    d = cuda(x)
    d["k"] = d["k"][:, :, :1].expand(B, T, H, K)
    want, _ = linattn.fwd(d["q"], d["k"].contiguous(), d["v"], d["log_decay"])
    assert bits(linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"])[0], want)
    fused = torch.full((B, T, 4, H, K), float("nan"), dtype=TYPES[dtype], device="cuda")
    for i, n in enumerate(("q", "k", "v")):
        fused[:, :, i] = d[n]
    o, _ = linattn.fwd(fused[:, :, 0], fused[:, :, 1], fused[:, :, 2], d["log_decay"], out=fused[:, :, 3])
    assert bits(o, want) and bits(fused[:, :, 2], d["v"])
    by_head = {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v")}
    o = torch.empty((B, H, T, V), dtype=TYPES[dtype], device="cuda").transpose(1, 2)
    linattn.fwd(by_head["q"], by_head["k"], by_head["v"], d["log_decay"], out=o)
    assert bits(o, want)
    guard = torch.full((B, T + 2, H, V), 7.0, dtype=TYPES[dtype], device="cuda")
    linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], out=guard[:, 1:-1])
    assert bits(guard[:, 1:-1], want) and torch.all(guard[:, 0] == 7) and torch.all(guard[:, -1] == 7)


@pytest.mark.parametrize("T", [6, 70, 2100, 2500])
def test_state_in_place_and_pieces(linattn, T):
    """s_out may be s_in; a sequence in pieces equals the whole within the bounds; no token, no change."""
    x = inputs(T, 2, T, 2, 64, 64, "bf16")
    d = cuda(x)
    o, S = linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], s_in=d["s_in"], want_state=True, out_dtype=torch.float32)
    s = d["s_in"].clone()
    o2, s2 = linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], s_in=s, s_out=s, out_dtype=torch.float32)
    assert s2 is s and bits(o, o2) and bits(S, s)
    (o_ref, S_ref), (o_size, S_size) = reference(x, 1.0)
    for cut in (1, T // 3, T - 1):
        s, got = d["s_in"].clone(), []
        for a, b in ((0, cut), (cut, cut), (cut, T)):
            got.append(linattn.fwd(d["q"][:, a:b], d["k"][:, a:b], d["v"][:, a:b], d["log_decay"], s_in=s, s_out=s,
                                   out_dtype=torch.float32)[0])
        check(f"cut at {cut} o", torch.cat(got, 1), o_ref, o_size, T, 64, False)
        check(f"cut at {cut} s_out", s, S_ref, S_size, T, 64, False)


def test_no_tokens(linattn):
    x = cuda(inputs(1, 2, 1, 2, 64, 32, "bf16"))
    e = {n: x[n][:, :0] for n in ("q", "k", "v")}
    o, S = linattn.fwd(e["q"], e["k"], e["v"], x["log_decay"], s_in=x["s_in"], want_state=True)
    assert o.shape == (2, 0, 2, 32) and bits(S, x["s_in"])
    assert torch.all(linattn.fwd(e["q"], e["k"], e["v"], x["log_decay"], want_state=True)[1] == 0)
    o, S = linattn.fwd(x["q"][:0], x["k"][:0], x["v"][:0], x["log_decay"], want_state=True)
    assert o.shape[0] == 0 and S.shape[0] == 0


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_later_tokens_do_not_matter(linattn, dtype, out):
    x = cuda(inputs(5, 1, 400, 2, 64, 64, dtype))
    o, _ = linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], out_dtype=TYPES[out])
    for cut in (1, 17, 64, 301):
        y = {n: x[n].clone() for n in ("q", "k", "v")}
        for t in y.values():
            t[:, cut:] = -3.0 * t[:, cut:] + 1.0
        assert bits(linattn.fwd(y["q"], y["k"], y["v"], x["log_decay"], s_in=x["s_in"], out_dtype=TYPES[out])[0][:, :cut],
                    o[:, :cut])


def test_rows_far_apart(linattn):
    """Token rows 64 KiB apart: offsets pass 2^32 bytes; bit for bit the packed call."""
    T, K = 70000, 64
    wide = torch.empty((1, T, 1, 32768), dtype=torch.bfloat16, device="cuda")
    for i in range(3):
        wide[..., i * K:(i + 1) * K] = normal(generator(i), 1, T, 1, K, dtype=torch.bfloat16).cuda()
    q, k, v, o = (wide[..., i * K:(i + 1) * K] for i in range(4))
    g = torch.tensor([-0.01], device="cuda")
    linattn.fwd(q, k, v, g, out=o)
    want, _ = linattn.fwd(q.contiguous(), k.contiguous(), v.contiguous(), g)
    assert bits(o, want)


def test_many_heads(linattn):
    """More workgroups than a grid of one dimension of 16 bits: every head is the same small problem."""
    H = 70000
    x = inputs(3, 1, 20, 1, 8, 8, "f32", state=False, decay=[-0.1])
    d = cuda(x)
    e = {n: d[n].expand(1, 20, H, 8) for n in ("q", "k", "v")}
    o, S = linattn.fwd(e["q"], e["k"], e["v"], d["log_decay"].expand(H).contiguous(), want_state=True)
    one, s1 = linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], want_state=True)
    assert bits(o, one.expand(1, 20, H, 8)) and bits(S, s1.expand(1, H, 8, 8))


def test_nan_stays_with_its_sequence(linattn):
    x = cuda(inputs(9, 3, 130, 2, 64, 64, "bf16"))
    want, S = linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], want_state=True)
    x["v"][1, 70] = float("nan")
    o, S2 = linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], want_state=True)
    for b in (0, 2):
        assert bits(o[b], want[b]) and bits(S2[b], S[b])
    assert bits(o[1, :64], want[1, :64]) and torch.isnan(o[1, 70:]).all() and torch.isnan(S2[1]).all()


@pytest.mark.parametrize("T", [1, 300, 2000])
def test_same_call_same_bits_on_any_stream(linattn, T):
    x = cuda(inputs(T, 2, T, 2, 64, 64, "bf16"))
    call = lambda **kw: linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], want_state=True, **kw)  # noqa: E731
    o, S = call()
    side = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for i in range(6):   # two streams at once, and torch's current one
        with torch.cuda.stream(side[i % 2]):
            got.append(call())
        got.append(call(stream=side[(i + 1) % 2]))
    torch.cuda.synchronize()
    for a, b in got:
        assert bits(a, o) and bits(b, S)


@pytest.mark.parametrize("T", [1, 100, 3000])
def test_graphs(linattn, T):
    """Two captured graphs (the longest call takes a workspace) replayed in turn with eager calls between."""
    x = [cuda(inputs(T + i, 1, T, 2, 64, 64, "bf16")) for i in range(2)]
    need = linattn.fwd_workspace_bytes(1, T, 2, 64, 64, state_out=True)
    assert (need > 0) == (T == 3000)
    graphs, outs = [], []
    for d in x:
        call = lambda d=d: linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], s_in=d["s_in"], want_state=True)  # noqa: E731
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for rep in range(3):
        for d in x:
            d["v"].mul_(-0.5)
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        eager = [linattn.fwd(d["q"], d["k"], d["v"], d["log_decay"], s_in=d["s_in"], want_state=True) for d in x]
        torch.cuda.synchronize()
        for (o, S), (a, b) in zip(outs, eager):
            assert bits(o, a) and bits(S, b), f"replay {rep}"


def test_given_workspace(linattn):
    x = cuda(inputs(4, 1, 2000, 1, 64, 64, "f32"))
    n = linattn.fwd_workspace_bytes(1, 2000, 1, 64, 64, torch.float32, state_out=True)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")   # NaN patterns
    o, S = linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], want_state=True)
    o2, S2 = linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], s_in=x["s_in"], want_state=True, workspace=ws[:n])
    assert bits(o, o2) and bits(S, S2) and torch.all(ws[n:] == 255)
    with pytest.raises(linattn.LinattnError):
        linattn.fwd(x["q"], x["k"], x["v"], x["log_decay"], workspace=ws[:n // 2].contiguous())
