"""The operators together, as a layer runs them: norm with the residual, q, k
and v as slices of one projection, rotary positions, attention, the library's
per-head group norm and gate; a padded prompt batch, then single tokens, which
continue it; the training pass back through all of it; a decode step as one
captured graph."""
import numpy as np
import pytest
import torch

from oracle import group_norm_heads
from oracle import linattn_oracle as R
from tests.linattn_util import BF, bits, f64, generator, normal, say

pytestmark = pytest.mark.gpu

B, H, D = 3, 4, 64
C = H * D


@pytest.fixture(scope="module")
def linattn():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import linattn

    return linattn


def layer_inputs(T, dtype):
    g = generator(T)
    return {"x": normal(g, B, T, C, std=1.0, dtype=dtype), "res": normal(g, B, T, C, std=1.0, dtype=dtype),
            "qkv": normal(g, B, T, 3, H, D, dtype=dtype), "gate": normal(g, B, T, C, dtype=dtype)}


W = 1.0 + normal(generator(90), C, std=0.1)
GAMMA, BETA = 1.0 + normal(generator(91), C, std=0.1), normal(generator(92), C, std=0.1)
DECAY = torch.tensor([-0.5, -0.1, -0.02, -0.004])


@pytest.fixture(scope="module")
def weights():
    return {"w": W.cuda(), "decay": DECAY.cuda(), "gamma": GAMMA.cuda(), "beta": BETA.cuda()}


def gpu_layer(linattn, p, x, freqs, positions, lengths=None, s_in=None, s_out=None):
    """(codes, scales, h, o, s_out, out) of one pass over whatever tokens x holds."""
    from linear_attention_rnn_amd import wkv6

    codes, scales, h = linattn.rms_norm_q8(x["x"], p["w"], residual=x["res"])
    qkv = x["qkv"]
    o, s = linattn.retention(qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2], p["decay"], freqs, positions=positions,
                             scale=D ** -0.5, lengths=lengths, s_in=s_in, s_out=s_out, want_state=True,
                             out_dtype=torch.float32)
    T = o.shape[1]
    out = wkv6.group_norm_gate(o.view(B, T, C), x["gate"], p["gamma"], p["beta"], H)
    return codes, scales, h, o, s, out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_prompt_then_tokens(linattn, weights, dtype):
    T, steps = 140, 5
    lengths = [140, 3, 77]
    freqs = linattn.rope_freqs(D, scaling="bands", factor=4.0)
    x = layer_inputs(T + steps, dtype)
    # the sequences as they are: each its prompt rows, then `steps` more of its own
    rows = [list(range(n)) + list(range(T, T + steps)) for n in lengths]
    prompt = {n: t[:, :T].cuda() for n, t in x.items()}
    pos = torch.arange(T, dtype=torch.int32).expand(B, T).contiguous().cuda()
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    codes, scales, h, o, s, out = gpu_layer(linattn, weights, prompt, freqs, pos, n)
    got_o, got_out, states = [o], [out], [s]
    for i in range(steps):
        tok = {m: t[:, T + i:T + i + 1].cuda() for m, t in x.items()}
        r = gpu_layer(linattn, weights, tok, freqs, (n + i)[:, None].contiguous(), None, states[-1])
        got_o.append(r[3])
        got_out.append(r[5])
        states.append(r[4])
    torch.cuda.synchronize()
    for b in range(B):
        q, k, v = (f64(x["qkv"][b, rows[b], i])[None] for i in range(3))
        at = np.arange(lengths[b] + steps)[None]
        turn = lambda t: R.rope_ref(t, at, f64(freqs))  # noqa: E731
        if dtype == torch.bfloat16:   # the rotation's outputs are stored in bfloat16
            q, k = (f64(torch.from_numpy(turn(t)).to(torch.bfloat16)) for t in (q, k))
        else:
            q, k = turn(q), turn(k)
        o_ref, s_ref = R.linattn_ref(q, k, v, f64(DECAY), D ** -0.5)
        o = torch.cat([got_o[0][b, :lengths[b]]] + [t[b] for t in got_o[1:]])
        y = torch.cat([got_out[0][b, :lengths[b]]] + [t[b] for t in got_out[1:]])
        y_ref = group_norm_heads(o_ref.reshape(1, -1, C), H, f64(GAMMA), f64(BETA), 64e-5) * f64(x["gate"][b, rows[b]])[None]
        # float32 attention of 1e-6; with bfloat16 inputs a rotated value next to a tie may round
        # the other way than the oracle's: one in 2^16 / 2^8, by 2^-7 of it; the group norm
        # multiplies errors by at most 1 / sqrt(64e-5 + var), and its output is bfloat16
        rel = lambda a, b: float(np.linalg.norm(a - b) / np.linalg.norm(b))  # noqa: E731
        e = [rel(f64(o), o_ref[0]), rel(f64(states[-1][b]), s_ref[0]), rel(f64(y), y_ref[0])]
        say(f"[layer] sequence {b}: o {e[0]:.3g}, state {e[1]:.3g}, gated {e[2]:.3g}")
        tol = 2e-6 if dtype == torch.float32 else 2.0 ** -7 * 2.0 ** -4
        assert e[0] <= tol and e[1] <= tol and e[2] <= BF
        y = R.rms_norm_ref(f64((x["x"][b, :lengths[b]].float() + x["res"][b, :lengths[b]].float()).to(dtype)), f64(W), 1e-6)
        deq = f64(codes[b, :lengths[b]].float()) * np.repeat(f64(scales[b, :lengths[b]]), 128, -1)
        assert rel(deq, y) <= 2.0 ** -4


def test_training_pass(linattn):
    """Gradients through rotation and attention equal differences along random directions."""
    T = 130
    g = generator(5)
    q, k, v, do = (normal(g, B, T, H, D).cuda() for _ in range(4))
    freqs = linattn.rope_freqs(D)
    decay = DECAY.cuda()
    got = linattn.retention_bwd(q, k, v, decay, do, freqs, layout="interleaved", scale=0.2)
    x = {"q": q, "k": k, "v": v}
    for i, n in enumerate(x):
        d = normal(generator(30 + i), B, T, H, D).cuda()
        up, down = (linattn.retention(*[x[m] + (s * d if m == n else 0) for m in x], decay, freqs, layout="interleaved",
                                      scale=0.2)[0].double() for s in (1.0, -1.0))
        slope, want = float(((up - down) * do.double()).sum()) / 2, float((got[n].double() * d.double()).sum())
        size = float(up.norm() * do.double().norm())
        say(f"[layer] d{n}: difference {slope:.8g}, gradient {want:.8g}, size {size:.3g}")
        assert abs(slope - want) <= 3e-6 * size


@pytest.mark.parametrize("handle", [False, True])
def test_turned_copies_outlive_the_call(linattn, handle):
    """On a stream of the caller's, behind other work: memory that the call has
    given back is not written by torch's own stream before it has run."""
    g = generator(6)
    q, k, v, do = (normal(g, B, 200, H, D, dtype=torch.bfloat16).cuda() for _ in range(4))
    freqs, decay = linattn.rope_freqs(D), DECAY.cuda()
    want, _ = linattn.retention(q, k, v, decay, freqs)
    grads = linattn.retention_bwd(q, k, v, decay, do, freqs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    stream = side.cuda_stream if handle else side
    got, _ = linattn.retention(q, k, v, decay, freqs, stream=stream)
    got_grads = linattn.retention_bwd(q, k, v, decay, do, freqs, stream=stream)
    spoiled = [torch.full_like(q, float("nan")) for _ in range(8)]
    torch.cuda.synchronize()
    assert bits(got, want) and all(bits(got_grads[n], grads[n]) for n in grads) and spoiled


def test_decode_step_as_a_graph(linattn, weights):
    """One captured step whose state is updated in place, replayed for token after token."""
    freqs = linattn.rope_freqs(D)
    x = {n: t.cuda() for n, t in layer_inputs(6, torch.bfloat16).items()}
    now = {n: t[:, :1].clone() for n, t in x.items()}
    pos = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    state = torch.zeros((B, H, D, D), device="cuda")
    gpu_layer(linattn, weights, now, freqs, pos, None, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gpu_layer(linattn, weights, now, freqs, pos, None, state, state)
    eager = torch.zeros_like(state)
    for t in range(6):
        for n in now:
            now[n].copy_(x[n][:, t:t + 1])
        pos.fill_(t)
        torch.cuda.synchronize()
        graph.replay()
        want = gpu_layer(linattn, weights, now, freqs, pos, None, eager)
        eager = want[4]
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert bits(a, b), t
        assert bits(state, eager)
