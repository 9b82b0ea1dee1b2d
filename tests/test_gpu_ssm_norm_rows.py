"""ssm.block_norm and block_norm_bwd where a workgroup goes through several rows
one after the other, and at the widths between those of test_gpu_ssm_norm.py:
sums of dpost, dpre and dgate over rows, buffers of the rows' sums in turn.
Bounds as there: chains of at most 32 rows, then 64 bits."""
import numpy as np
import pytest
import torch

from oracle import ssm_oracle as R
from tests.ssm_util import U, f64, generator, normal, within
from tests.test_gpu_ssm_norm import check, draw, sizes, ssm  # noqa: F401

pytestmark = pytest.mark.gpu

# rows, C, rows that share a gate; turns of a workgroup's rows
SHAPES = [(520000, 8, 260000),   # 8 threads a row: 32 turns of 32 rows
          (40000, 64, 20000), (25000, 128, 5), (12000, 256, 6000), (9000, 512, 4500),   # 8, 16, 32 and 64 threads a row: 2 to 5
          (6200, 768, 3100), (4200, 1024, 1),   # 64 threads, two pieces
          (1100, 1032, 550), (1100, 2048, 1), (17000, 2048, 17000),   # 256 threads, one piece: 3 turns, and the most, 32
          (7, 2056, 1), (1030, 4096, 515), (1030, 4096, 1),   # two pieces
          (530, 4104, 265), (800, 8192, 400), (530, 8200, 265), (600, 16384, 1)]   # 512 threads, two and four pieces


@pytest.mark.parametrize("rows,C,per", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_in_turn(ssm, rows, C, per, dtype):  # noqa: F811
    check(ssm, draw(rows, C, per, dtype))


@pytest.mark.parametrize("parts", [("pre",), ("post",), ("gate",), ("gate", "post"), ("gate", "pre"), ("residual", "post", "pre")])
@pytest.mark.parametrize("rows,C,per", [(1100, 1032, 550), (800, 8192, 400), (40000, 64, 20000)])
def test_parts_of_rows_in_turn(ssm, rows, C, per, parts):  # noqa: F811
    check(ssm, draw(rows, C, per, "f32", parts), activation="sigmoid")


@pytest.mark.parametrize("shared", [True, False])
def test_sums_of_many_rows(ssm, shared):  # noqa: F811
    """2^22 + 4 rows, 64 different ones over and over: each sum is that of the 64 rows as often as they come, in 64 bits."""
    rows, C, n = 2 ** 22 + 4, 64, 64
    g = generator(3)
    x, res, dy, dh = (normal(g, n, C, std=1.0) for _ in range(4))
    gate = normal(g, 1 if shared else n, C, std=1.0)
    post, pre = 1 + normal(g, C, std=0.3), 1 + normal(g, C, std=0.3)
    times = np.full(n, rows // n) + (np.arange(n) < rows % n)
    far = lambda t: t.cuda().repeat(rows // n + 1, 1)[:rows]  # noqa: E731
    kw = dict(gate=gate.cuda() if shared else far(gate), post_weight=post.cuda(), pre_weight=pre.cuda(), scale=0.5, activation="silu")
    y, h = ssm.block_norm(far(x), residual=far(res), **kw)
    got = ssm.block_norm_bwd(far(x), h, dy=far(dy), dh=far(dh), **kw)
    torch.cuda.synchronize()
    names = ("post_weight", "pre_weight") + (("gate",) if shared else ())
    ref, size = ({m: np.zeros(C) for m in names} for _ in range(2))
    for i in range(n):
        row = lambda t: f64(t[i:i + 1])  # noqa: E731
        a = (row(x), f64(h[i:i + 1]), row(dy), row(dh), f64(gate) if shared else row(gate), f64(post), f64(pre), 0.5, "silu", 1e-6)
        r, s = R.block_norm_ref_backward(*a), sizes(*a)
        for m in names:
            ref[m] += times[i] * r[m].reshape(C)
            size[m] += times[i] * s[m].reshape(C)
    for m in names:
        within("d" + m, got[m].reshape(C), ref[m], size[m], 160 + 32, False)
