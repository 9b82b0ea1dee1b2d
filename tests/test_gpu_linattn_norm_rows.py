"""linattn.rms_norm_bwd over many rows: the weights' gradient is a sum over all
of them whose error does not grow with their number.

2-norm of the error over that of the result, with u = 2^-24 and independent
errors of standard deviation 1 / sqrt(3) of their bounds: a term dy h r errs by 3
u for r and u for its product (sqrt(10) u / sqrt(3) = 1.83 u); eight terms are
added in float32, partial sums of 1 to 8 of them (sqrt(36 / 8) u / sqrt(3) = 1.22
u), and so are the sums of eight workgroups; three more roundings (a thread's sum,
a workgroup's, the result) add u each (u): in all sqrt(1.83^2 + 2 x 1.22^2 + 1) u =
2.7 u."""
import pytest
import torch

from tests.linattn_util import TYPES, U, say
from tests.test_gpu_linattn_norm import linattn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,C", [(300, 2048), (2 ** 19, 64), (2 ** 22, 64), (70001, 512), (32768, 2048), (9001, 8192)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_weights(linattn, rows, C, dtype):  # noqa: F811
    g = torch.Generator("cuda")
    g.manual_seed(rows)
    h, dy = (torch.empty(rows, C, device="cuda").normal_(generator=g).to(TYPES[dtype]) for _ in range(2))
    w = torch.empty(C, device="cuda").normal_(1.0, 0.1, generator=g)
    got = linattn.rms_norm_bwd(dy, h, w, 1e-6)["weight"].double()
    want = torch.zeros(C, dtype=torch.float64, device="cuda")
    for at in range(0, rows, 1 << 16):
        x = h[at:at + (1 << 16)].double()
        want += (dy[at:at + (1 << 16)].double() * x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-6)).sum(0)
    rel = float((got - want).norm() / want.norm())
    say(f"[norm] dweight of {rows} x {C} {dtype}: relative error {rel:.3g}")
    assert rel <= 2.75 * U
