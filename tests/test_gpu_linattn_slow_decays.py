"""linattn.fwd with decays close to 1: a state that lives for 10^4 to 10^6
tokens decays at its own rate, token by token, chunk by chunk and segment by
segment.  A factor a^n rounded to float32 is off by up to 2^-25, the same in
every step, so that the memory's length is off by 2^-25 / (1 - a^n).

Bounds (u = 2^-24).  What a step rounds is at most u of the state; errors of
many steps are independent, uniform ones of standard deviation u / sqrt(3) at
most each, so the 2-norm of the error of N roundings stays under
3 sqrt(N) u / sqrt(3) of the state's (three standard deviations).  The rate
itself, n log_decay of n tokens and expm1 of it, is off by u and 2 u of
itself, so that a state that has decayed by e^-x is off by 3 u x of itself."""
import math

import numpy as np
import pytest
import torch

from oracle import linattn_oracle as R
from tests.linattn_util import TYPES, U, f64, generator, normal, say
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu

DECAYS = [-1e-6, -2.2e-5, -3e-5, -1e-5, -1e-4, -3.2e-4]


def close(name, got, ref, roundings, tokens):
    """Per head (dimension 1), the 2-norms of the errors."""
    got, worst = f64(got), 0.0
    for h in range(ref.shape[1]):
        rel = np.linalg.norm(got[:, h] - ref[:, h]) / np.linalg.norm(ref[:, h])
        bound = 3 * math.sqrt(roundings) * U / math.sqrt(3) + 3 * U * tokens * abs(DECAYS[h])
        worst = max(worst, rel / bound)
        say(f"[linattn] {name}, log decay {DECAYS[h]}: relative error {rel:.3g}, {rel / bound:.3g} of the bound")
    assert worst <= 1.0, name


@pytest.mark.parametrize("per_call", [1, 8])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tokens_one_by_one(linattn, per_call, dtype):  # noqa: F811
    """4096 tokens after a large state: three roundings a token (k v, and the two sums of the update)."""
    g = generator(1)
    T, H, K, V = 4096, len(DECAYS), 16, 8
    q, k, v = (normal(g, 1, T, H, n, dtype=TYPES[dtype]) for n in (K, K, V))
    s0, decay = normal(g, 1, H, K, V, std=100.0), torch.tensor(DECAYS)
    _, ref = R.linattn_ref(f64(q), f64(k), f64(v), f64(decay), 1.0, None, f64(s0))
    q, k, v, s, decay = q.cuda(), k.cuda(), v.cuda(), s0.cuda(), decay.cuda()
    for t in range(0, T, per_call):
        linattn.fwd(*(x[:, t:t + per_call] for x in (q, k, v)), decay, s_in=s, s_out=s)
    torch.cuda.synchronize()
    close(f"{per_call} tokens a call, {dtype}", s, ref, 3 * T, T)


@pytest.mark.parametrize("K,V", [(64, 64), (128, 72)])
@pytest.mark.parametrize("copies", [40, 1])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_piece_by_piece(linattn, K, V, copies, dtype):  # noqa: F811
    """A state alone (keys of zero), through 16 pieces of 16384 tokens: one rounding a chunk of 64 tokens.  Of 40 copies of
    the heads every sequence is one run of chunks; of one copy it is cut into segments, which join their states by two
    roundings more a segment of at least a chunk."""
    T, pieces, H = 16384, 16, len(DECAYS)
    g = generator(2)
    decay = torch.tensor(DECAYS * copies).cuda()
    q, v = (normal(g, 1, T, 1, n, dtype=TYPES[dtype]).cuda().expand(1, T, H * copies, n) for n in (K, V))
    k = torch.zeros(1, T, 1, K, dtype=TYPES[dtype], device="cuda").expand(1, T, H * copies, K)
    s0 = normal(g, 1, H * copies, K, V, std=1.0)
    s = s0.cuda()
    need = linattn.fwd_workspace_bytes(1, T, H * copies, K, V, TYPES[dtype], state_out=True)
    assert (need > 0) == (copies == 1)
    out = torch.empty(1, T, H * copies, V, dtype=TYPES[dtype], device="cuda")
    for _ in range(pieces):
        linattn.fwd(q, k, v, decay, s_in=s, s_out=s, out=out)
    torch.cuda.synchronize()
    n = T * pieces
    ref = f64(s0) * np.exp(n * f64(decay))[None, :, None, None]
    close(f"{copies * H} heads of {K} x {V}, {dtype}", s[:, :H], ref[:, :H], 3 * n / 64, n)


@pytest.mark.parametrize("T", [4, 100, 1500])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_decay_that_is_no_number(linattn, T, dtype):  # noqa: F811
    """It spoils its head's state and no other's: also where nothing but the entering state is decayed."""
    g = generator(4)
    q, v = (normal(g, 1, T, 2, 64, dtype=TYPES[dtype]).cuda() for _ in range(2))
    s0, decay = normal(g, 1, 2, 64, 64).cuda(), torch.tensor([-0.1, float("nan")]).cuda()
    _, s = linattn.fwd(q, torch.zeros_like(q), v, decay, s_in=s0, want_state=True)
    assert torch.isfinite(s[:, 0]).all() and torch.isnan(s[:, 1]).all()
