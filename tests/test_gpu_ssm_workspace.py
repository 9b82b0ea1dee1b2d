"""Workspaces of the caller's: exactly as many bytes as asked for, in captured
calls that share one, and calls of several host threads at once."""
import threading

import pytest
import torch

from tests import ssm_util as S
from tests.ssm_util import bits, generator, normal

pytestmark = pytest.mark.gpu

GUARD = 4096


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


def calls(ssm, seed, B=2, T=150, D=72, N=24):
    """(workspace bytes, the call) of each gradient."""
    g = generator(seed)
    p = S.cuda(S.inputs(seed, B, T, D, N, 1, "bf16"))
    x, dy, gate = (normal(g, B, T, D, std=1.0, dtype=torch.bfloat16).cuda() for _ in range(3))
    w, cw, cb = normal(g, D, std=1.0).cuda(), normal(g, D, 4, std=0.5).cuda(), normal(g, D, std=0.1).cuda()
    h = ssm.block_norm(x, pre_weight=w)[1]
    one = gate[:, :1].contiguous()
    return [(ssm.scan_bwd_workspace_bytes(B, T, D, N), lambda **k: ssm.scan_bwd(**p, dy=dy, want_ds_in=True, **k)),
            (ssm.conv_bwd_workspace_bytes(B, T, D, 4), lambda **k: ssm.conv_bwd(x, cw, dy, bias=cb, want_ds_in=True, **k)),
            (ssm.block_norm_bwd_workspace_bytes(B * T, D, T), lambda **k: ssm.block_norm_bwd(
                x, h, dy=dy, gate=one, post_weight=w, pre_weight=w, activation="silu", **k))], [x, dy, p["x"]]


def same(a, b):
    assert set(a) == set(b) and all(bits(a[n], b[n]) for n in a)


@pytest.mark.parametrize("T", [1, 20, 150, 700])
@pytest.mark.parametrize("i", [0, 1, 2])
def test_given(ssm, i, T):
    """The bytes asked for are enough, nothing behind them is written, and what was in them does not matter."""
    n, call = calls(ssm, 1, T=T)[0][i]
    want = call()
    for fill in (0, 255):
        buffer = torch.full((n + GUARD,), fill, dtype=torch.uint8, device="cuda")
        same(call(workspace=buffer[:n]), want)
        torch.cuda.synchronize()
        assert torch.all(buffer[n:] == fill)
    from linear_attention_rnn_amd.linattn import LinattnError
    with pytest.raises(LinattnError):
        call(workspace=torch.empty(n - 16, dtype=torch.uint8, device="cuda"))


def test_graphs_share_a_workspace(ssm):
    """Two graphs on a stream of the caller's that use the same workspace, replayed one after the other."""
    side = torch.cuda.Stream()
    made, inputs = calls(ssm, 2)
    n = max(m for m, _ in made)
    workspace = torch.empty(n, dtype=torch.uint8, device="cuda")
    for _, call in made:
        call(workspace=workspace)
    torch.cuda.synchronize()
    graphs = []
    for part in (made[:2], made[1:]):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = [call(workspace=workspace, stream=side) for _, call in part]
        graphs.append((graph, out, part))
    for turn in range(3):
        for t in inputs:
            t.mul_(-0.75)
        torch.cuda.synchronize()
        for graph, _, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, out, part in graphs:
            for got, (_, call) in zip(out, part):
                same(got, call())
        torch.cuda.synchronize()


def test_threads(ssm):
    """Four host threads at once, each on a stream of its own with the pool's workspace."""
    made = [calls(ssm, 3 + i, T=100 + 50 * i)[0] for i in range(4)]
    want = [[call() for _, call in m] for m in made]
    torch.cuda.synchronize()
    got, failed = [None] * 4, []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(3):
                got[i] = [call(stream=stream) for _, call in made[i]]
                stream.synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for a, b in zip(got, want):
        for x, y in zip(a, b):
            same(x, y)
