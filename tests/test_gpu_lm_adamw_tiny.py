"""AdamW with second moments below float32's normal numbers."""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import U32, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


@pytest.mark.parametrize("p", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_roots_of_subnormal_second_moments(p, bits):
    """Gradients of 1e-20 and beta2 = 0.95: second moments of 5e-42, 3567 steps of 2^-149. A
    moment is two products and a sum, off by a step and a half of those at most; the root has
    half of that relative error. The first step from zero moments moves by
    lr g / (|g| + eps): with eps 0 by lr to either side."""
    tbe = lib()
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[p]
    desc = tbe.AdamWDesc(p, "f32", bits=bits, beta1=0.9, beta2=0.95, eps=0.0, weight_decay=0.0)
    x = torch.zeros(700, dtype=dt, device="cuda")
    g = (torch.rand(700, generator=gen(bits)) + 1).mul_(1e-20).cuda()
    g[1::2] *= -1
    state = tbe.AdamWState(desc, [x])
    lr = torch.full((1,), 0.5, device="cuda")
    tbe.tbe_adamw_step(desc, [x], [g], state, torch.ones(1, dtype=torch.int64, device="cuda"), lr)
    torch.cuda.synchronize()
    want = -0.5 * torch.sign(g).double()
    off = 0.5 * (1.5 / 3567 / 2) * 1.01 + 0.5 * 32 * U32 + 0.5 * torch.finfo(dt).eps / 2
    assert ((x.double() - want).abs() <= off).all(), (x.double() - want).abs().max().item()
    if bits == 8:   # roots of 2e-21 to 5e-21 are above 2^-100 and are kept
        assert (state.v[0].float() > 0).all() and (state.vs[0] > 0).all()
