"""linattn.fwd and bwd with decays above 1 over sequences that are cut into
segments: a state of zeros stays zero over tokens that add nothing, however
large a to the power of a segment's tokens is.

Bounds as in linattn_util; a factor a^x errs by 2 u x |log a| of itself, which
its size no longer makes up for: 2 u x |log a| of each term on top, x = 20."""
import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import BF, TYPES, U, f64, generator, normal, say, steps
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu

GROWTH, ACTIVE, T = [1.0, 0.7], 20, 1400


def check(name, got, ref, size, K, bf16):
    x = f64(got)
    assert np.isfinite(ref).all() and np.isfinite(x).all(), f"{name}: not finite"
    err = np.abs(x - ref)
    grown = 2 * ACTIVE * max(GROWTH) * U
    bound = ((16 + 2 * steps(T, K)) * U + grown) * size + 1e-37
    if bf16:
        bound = bound + BF * np.abs(ref) + (BF + BF * BF) * size
    rel = np.linalg.norm(err) / np.linalg.norm(ref)
    say(f"[linattn] {name}: {np.max(err / bound):.3g} of the bound, rel {rel:.3g}")
    assert np.all(err <= bound), name
    assert rel <= (BF if bf16 else 1e-6 + grown), name


@pytest.mark.parametrize("K,V", [(64, 64), (128, 72)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_leading_rows_of_zeros(linattn, K, V, dtype, out):  # noqa: F811
    """A prompt padded on the left: keys of zero but for the last tokens."""
    g = generator(K)
    H = len(GROWTH)
    q, k, v = (normal(g, 1, T, H, n, dtype=TYPES[dtype]) for n in (K, K, V))
    k[:, :-ACTIVE] = 0
    decay = torch.tensor(GROWTH)
    assert linattn.fwd_workspace_bytes(1, T, H, K, V, TYPES[dtype], TYPES[out], True) > 0
    o, S = linattn.fwd(q.cuda(), k.cuda(), v.cuda(), decay.cuda(), want_state=True, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    a = [f64(x) for x in (q, k, v)]
    o_ref, S_ref = R.linattn_ref(*a, f64(decay))
    o_size, S_size = R.linattn_ref(*[np.abs(x) for x in a], f64(decay))
    check("o", o, o_ref, o_size, K, out == "bf16")
    check("s_out", S, S_ref, S_size, K, False)
    assert torch.all(o[:, :-ACTIVE] == 0)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 72)])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("f32", "f32")])
def test_gradients_of_the_first_tokens_alone(linattn, K, V, dtype, grad):  # noqa: F811
    g = generator(K + 1)
    H = len(GROWTH)
    x = {n: normal(g, 1, T, H, d, dtype=TYPES[dtype]) for n, d in (("q", K), ("k", K), ("v", V), ("do", V))}
    x["do"][:, ACTIVE:] = 0
    x["k"][:, ACTIVE:] = 0
    decay = torch.tensor(GROWTH)
    assert linattn.bwd_workspace_bytes(1, T, H, K, V, TYPES[dtype], TYPES[grad], True) > 0
    got = linattn.bwd(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), decay.cuda(), x["do"].cuda(), want_ds_in=True,
                      grad_dtype=TYPES[grad])
    torch.cuda.synchronize()
    first = {n: f64(t)[:, :ACTIVE] for n, t in x.items()}
    ref, size = (R.linattn_ref_backward(f(first["q"]), f(first["k"]), f(first["v"]), f64(decay), f(first["do"]))
                 for f in (np.asarray, np.abs))
    for n in ("k", "v"):
        check("d" + n, got[n][:, :ACTIVE], ref[n], size[n], max(K, V), grad == "bf16")
        assert torch.all(got[n][:, ACTIVE:] == 0)
    check("ds_in", got["s_in"], ref["s_in"], size["s_in"], max(K, V), False)


@pytest.mark.parametrize("copies", [100, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_overflow_shows(linattn, copies, dtype):  # noqa: F811
    """Past the documented range (a^64 is infinite) a state is infinite or NaN, never a wrong number: in one run of chunks
    and in segments."""
    g = generator(9)
    q, k, v = (normal(g, 1, 1500, 2, 64, dtype=TYPES[dtype]).cuda().repeat(1, 1, copies, 1) for _ in range(3))
    decay = torch.tensor([2.0, 1.5] * copies, device="cuda")
    assert (linattn.fwd_workspace_bytes(1, 1500, 2 * copies, 64, 64, TYPES[dtype], state_out=True) > 0) == (copies == 1)
    o, S = linattn.fwd(q, k, v, decay, want_state=True)
    assert not torch.isfinite(S).any() and not torch.isfinite(o[:, 200:]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_overflow_of_the_entering_state_shows(linattn, dtype):  # noqa: F811
    """a^63 is finite and a^64 is not; nothing but the entering state grows."""
    g = generator(10)
    q, v = (normal(g, 1, 70, 1, 64, dtype=TYPES[dtype]).cuda() for _ in range(2))
    s0 = 1 + normal(g, 1, 1, 64, 64).abs().cuda()
    _, S = linattn.fwd(q, torch.zeros_like(q), v, torch.tensor([1.4], device="cuda"), s_in=s0, want_state=True)
    assert not torch.isfinite(S).any()
