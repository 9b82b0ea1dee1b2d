"""linattn.rope at positions far from zero, where the product of a position
and a frequency no longer fits a float64: the bounds are those of any other
position (tests/test_gpu_linattn_rope.py)."""
import numpy as np
import pytest
import torch

from tests.linattn_util import TYPES, f64, generator, normal
from tests.test_gpu_linattn_rope import check, linattn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start", [2 ** 31, 2 ** 40 + 12345, 2 ** 49 - 1, 2 ** 52, -(2 ** 52), -(2 ** 51) - 77])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_far_positions(linattn, start, layout, dtype):  # noqa: F811
    g = generator(3)
    B, T, H, D = 2, 37, 3, 64
    q, k = normal(g, B, T, H, D, dtype=TYPES[dtype]), normal(g, B, T, H, D, dtype=TYPES[dtype])
    pos = torch.randint(-(2 ** 31), 2 ** 31 - 1, (B, T), generator=g, dtype=torch.int32)
    pos[0, 0], pos[0, 1] = 2 ** 31 - 1, -(2 ** 31)
    freqs = linattn.rope_freqs(D)
    for inverse in (False, True):
        a, b = linattn.rope(q.cuda(), k.cuda(), freqs, positions=pos.cuda(), start=start, layout=layout, inverse=inverse)
        torch.cuda.synchronize()
        for name, got, x in (("q", a, q), ("k", b, k)):
            check(f"from {start}, {layout} {dtype} {name}", got, x, start + pos.numpy().astype(np.int64), f64(freqs), layout,
                  inverse, dtype == "bf16")
