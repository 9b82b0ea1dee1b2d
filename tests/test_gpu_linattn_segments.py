"""Calls cut into many segments, of every width: the carry kernel of more than
64 key channels, two blocks of values, states in and out, segments that lengths
leave short or empty; gradients of padded batches whose keys and values differ
in width."""
import pytest
import torch

from tests.linattn_util import TYPES, check
from tests.test_gpu_linattn import inputs, linattn, run_and_check  # noqa: F401
from tests.test_gpu_linattn_backward import call, cuda, reference, with_gradients

pytestmark = pytest.mark.gpu


def segments(need, B, H, K, V, sweeps=1):
    """How many a plan has whose workspace is `need` bytes."""
    pad = lambda n: 64 if n <= 64 else 128  # noqa: E731
    return need // (sweeps * B * H * pad(K) * pad(V) * 4)


@pytest.mark.parametrize("K,V", [(128, 128), (72, 128), (128, 40), (64, 128)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("H", [1, 2])
def test_many_segments(linattn, K, V, dtype, out, H):  # noqa: F811
    T = 2000
    need = linattn.fwd_workspace_bytes(1, T, H, K, V, TYPES[dtype], TYPES[out], True)
    assert segments(need, 1, H, K, V) > 8
    x = inputs(T + K + H, 1, T, H, K, V, dtype, decay=[-0.002, -0.05][:H])
    run_and_check(linattn, x, K ** -0.5, out, label=f"H={H} K={K} V={V} {dtype}->{out}")


@pytest.mark.parametrize("K,V", [(128, 128), (72, 128), (128, 40)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("lengths", [[2000, 1, 0], [1999, 641, 640], [64, 65, 1537]])
def test_padded_prompts(linattn, K, V, dtype, out, lengths):  # noqa: F811
    T = 2000
    x = inputs(T + K, len(lengths), T, 1, K, V, dtype, decay=[-0.003])
    for b, n in enumerate(lengths):
        for t in ("q", "k", "v"):
            x[t][b, n:] = 0
    need = linattn.fwd_workspace_bytes(len(lengths), T, 1, K, V, TYPES[dtype], TYPES[out], True)
    assert segments(need, len(lengths), 1, K, V) > 8
    run_and_check(linattn, x, 0.3, out, lengths=lengths, label=f"{lengths} K={K} V={V}")


@pytest.mark.parametrize("K,V", [(128, 128), (72, 128), (128, 40), (64, 64)])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_gradients_of_many_segments(linattn, K, V, dtype, grad):  # noqa: F811
    T = 2000
    need = linattn.bwd_workspace_bytes(1, T, 1, K, V, TYPES[dtype], TYPES[grad], True)
    assert segments(need, 1, 1, max(K, V), max(K, V), 3) > 8
    x = with_gradients(inputs(T + V, 1, T, 1, K, V, dtype, decay=[-0.004]), T, dtype)
    g = call(linattn, cuda(x), 0.5, want_ds_in=True, grad_dtype=TYPES[grad])
    torch.cuda.synchronize()
    ref, size = reference(x, 0.5)
    for n in g:
        check(f"d{n} K={K} V={V} {dtype}->{grad}", g[n], ref[n], size[n], T, max(K, V), grad == "bf16" and n != "s_in")


@pytest.mark.parametrize("K,V", [(128, 64), (64, 128), (128, 128)])
@pytest.mark.parametrize("T,lengths", [(200, [0, 1, 64, 65, 200]), (777, [777, 194]), (1500, [1500, 0, 700]), (2000, [10, 2000])])
@pytest.mark.parametrize("dtype,grad", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_gradients_of_padded_batches(linattn, K, V, T, lengths, dtype, grad):  # noqa: F811
    """NaN behind a sequence is not read; gradients there are zero; the state's gradient in place."""
    x = with_gradients(inputs(T + K, len(lengths), T, 2, K, V, dtype), T, dtype)
    ref, size = reference(x, 1.0, lengths)
    for b, n in enumerate(lengths):
        for t in ("q", "k", "v", "do"):
            x[t][b, n:] = float("nan")
    d = cuda(x)
    g = call(linattn, d, lengths=torch.tensor(lengths, dtype=torch.int32).cuda(), out={"s_in": d["ds_out"]},
             grad_dtype=TYPES[grad])
    torch.cuda.synchronize()
    for n in ref:
        check(f"d{n}", g[n], ref[n], size[n], T, max(K, V), grad == "bf16" and n != "s_in")
    for b, m in enumerate(lengths):
        assert all(torch.all(g[n][b, m:] == 0) for n in ("q", "k", "v"))
