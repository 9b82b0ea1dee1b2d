"""ssm.scan, conv and their gradients at sizes whose launches the other tests do
not reach: calls of 513 to 1024 workgroups of 8 channels, many groups of few
channels on the instances of 16 and 32, every number of states there, and
convolutions of so many tokens that a gradient's run is 32 of them."""
import pytest
import torch

from tests import ssm_util as S
from tests.ssm_util import generator, normal
from tests.test_gpu_ssm_conv import check, check_bwd, cuda, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ssm():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from linear_attention_rnn_amd import ssm

    return ssm


# B, D, G: 640 workgroups of 8 channels; 768 and 1152 groups of 8 channels; 512 of 24 (1536 workgroups of 8, 1024 of 16)
CALLS = [((8, 640, 1), N, T, t) for N in (8, 16, 32, 64) for T, t in ((20, "f32"), (50, "bf16"), (133, "f32"), (133, "bf16"))]
CALLS += [((6, 1024, 128), N, T, t) for N in (24, 40) for T, t in ((133, "f32"), (20, "bf16"))]
CALLS += [((9, 1024, 128), N, T, t) for N in (16, 24, 48, 56) for T, t in ((133, "bf16"), (20, "f32"))]
CALLS += [((8, 1536, 64), N, T, t) for N in (24, 40) for T, t in ((133, "bf16"), (50, "f32"))]


@pytest.mark.parametrize("size,N,T,dtype", CALLS)
def test_scan_of_many_workgroups(ssm, size, N, T, dtype):
    B, D, G = size
    p = S.inputs(T + N, B, T, D, N, G, dtype)
    lengths = [T, T - 3, 0, 17] * (B // 4) + [T - 1] * (B % 4)
    dy, ds = normal(generator(5), B, T, D, std=1.0, dtype=p["x"].dtype), normal(generator(6), B, D, N, std=0.3)
    q, n = S.cuda(p), torch.tensor(lengths, dtype=torch.int32).cuda()
    y, s = ssm.scan(**q, lengths=n, want_state=True)
    g = ssm.scan_bwd(**q, dy=dy.cuda(), ds_out=ds.cuda(), lengths=n, want_ds_in=True)
    torch.cuda.synchronize()
    name = f"{B}x{T}x{D} N{N} G{G} {dtype}"
    S.check_scan(name, p, y, s, lengths)
    S.check_scan_bwd(name, p, g, dy, ds, lengths)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("activation", ["silu", None])
def test_conv_of_many_tokens(ssm, W, activation, dtype):
    """16 x 1037 tokens of 1024 channels: 8192 threads for each of more than 32 runs of 16, so runs of 32, the last of 13."""
    B, T, D = 16, 1037, 1024
    p = draw(B, T, D, W, dtype)
    lengths = [1037, 1, 0, 32, 33, 1024, 31, 700] * 2
    n = torch.tensor(lengths, dtype=torch.int32).cuda()
    q = cuda(p)
    y, s = ssm.conv(**q, activation=activation, lengths=n, want_state=True)
    dy, ds = normal(generator(1), B, T, D, dtype=y.dtype), normal(generator(2), B, W - 1, D, dtype=y.dtype)
    g = ssm.conv_bwd(**q, dy=dy.cuda(), activation=activation, lengths=n, ds_out=ds.cuda(), want_ds_in=True)
    torch.cuda.synchronize()
    check(p, y, s, activation, lengths)
    check_bwd(p, g, dy, ds, activation, lengths)


@pytest.mark.parametrize("N", [8, 16])
@pytest.mark.parametrize("T", [7, 8, 9, 16, 17, 32, 33, 63, 64, 65, 127, 256])
def test_scan_around_blocks(ssm, T, N):
    """One token more or fewer than go token by token, than a block of 32, 64 or 128 tokens holds, or than a lane."""
    p = S.inputs(T, 2, T, 24, N, 1, "f32")
    dy, ds = normal(generator(5), 2, T, 24, std=1.0), normal(generator(6), 2, 24, N, std=0.3)
    q, n = S.cuda(p), torch.tensor([T, T - 1], dtype=torch.int32).cuda()
    y, s = ssm.scan(**q, lengths=n, want_state=True)
    g = ssm.scan_bwd(**q, dy=dy.cuda(), ds_out=ds.cuda(), lengths=n, want_ds_in=True)
    torch.cuda.synchronize()
    S.check_scan(f"{T} tokens", p, y, s, [T, T - 1])
    S.check_scan_bwd(f"{T} tokens", p, g, dy, ds, [T, T - 1])


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 13, 15, 16, 17, 18, 19, 31, 32, 33, 48])
@pytest.mark.parametrize("state", [True, False])
def test_conv_around_runs(ssm, T, W, state):
    p = draw(2, T, 40, W, "f32", state)
    q, n = cuda(p), torch.tensor([T, T - 1], dtype=torch.int32).cuda()
    y, s = ssm.conv(**q, lengths=n, want_state=True)
    dy, ds = normal(generator(1), 2, T, 40), normal(generator(2), 2, W - 1, 40)
    g = ssm.conv_bwd(**q, dy=dy.cuda(), lengths=n, ds_out=ds.cuda(), want_ds_in=True)
    torch.cuda.synchronize()
    check(p, y, s, "silu", [T, T - 1])
    check_bwd(p, g, dy, ds, "silu", [T, T - 1])
