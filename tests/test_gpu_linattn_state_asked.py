"""Outputs and gradients do not depend on whether the state, or its gradient,
is asked for: the same bits either way."""
import pytest
import torch

from tests.linattn_util import TYPES, bits, generator, normal
from tests.test_gpu_linattn import linattn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [8, 64, 200, 1500])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 72)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_same_bits(linattn, T, K, V, dtype, out):  # noqa: F811
    g = generator(T + K)
    q, k, v, do = (normal(g, 2, T, 3, n, dtype=TYPES[dtype]).cuda() for n in (K, K, V, V))
    s_in, ds = (normal(g, 2, 3, K, V).cuda() for _ in range(2))
    decay = torch.tensor([-0.3, -0.02, -1e-4], device="cuda")
    a, none = linattn.fwd(q, k, v, decay, s_in=s_in, out_dtype=TYPES[out])
    b, s = linattn.fwd(q, k, v, decay, s_in=s_in, out_dtype=TYPES[out], want_state=True)
    assert none is None and s is not None and bits(a, b)
    a = linattn.bwd(q, k, v, decay, do, s_in=s_in, ds_out=ds, grad_dtype=TYPES[out])
    b = linattn.bwd(q, k, v, decay, do, s_in=s_in, ds_out=ds, grad_dtype=TYPES[out], want_ds_in=True)
    for n in a:
        assert bits(a[n], b[n]), n
