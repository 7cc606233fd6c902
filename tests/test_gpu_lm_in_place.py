"""The combine's gradient written over its input: the bits of a call with a
matrix of its own, at the widths where a row's end meets another wave's part."""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, U32, close, gen, new, randn, say, view_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# a row is cut into vectors of 4 (f32) or 8 columns, 64 of them a wave: widths with 1
# to VE - 1 columns after a whole number of waves' vectors, and around them
WIDTHS = {"f32": (513, 514, 515, 769, 771, 1025, 1027, 2049, 4099, 511, 517, 5, 6),
          "bf16": (1025, 1026, 1031, 1537, 1543, 2049, 4097, 4100, 1023, 1033, 9, 15),
          "f16": (1025, 1030, 1537, 2055)}


@pytest.mark.parametrize("K", [1, 7, 64])
@pytest.mark.parametrize("t,D", [(t, D) for t in WIDTHS for D in WIDTHS[t]])
def test_combine_gradient_in_place(t, D, K):
    say("combine gradient in place", t, D, K)
    tbe = lib()
    g = gen(D + K)
    N, E = (97, 9) if K > 1 else (700, 9)
    M = N * K
    desc = tbe.ExpertDesc(N, K, E, D, dtype=t)
    ids = torch.randint(-1, E, (N, K), generator=g).cuda()
    plan = tbe.ExpertPlan(desc)
    tbe.tbe_expert_plan(desc, ids, plan, tbe.expert_workspace(desc))
    dout, ys = randn(g, N, D).to(DT[t]), randn(g, M, D).to(DT[t])
    w = torch.rand(N, K, generator=g).cuda()
    ok = (plan.slots >= 0).view(N, K)
    place = torch.where(plan.slots >= 0, plan.slots, -1 - plan.slots).long()
    y = torch.where(ok[:, :, None], ys[place].to(F64).view(N, K, D), 0.0)
    prod = dout.to(F64)[:, None, :] * y
    for stride in (0, 3):
        rows = view_of(ys.clone(), stride)
        dys, dw = new(M, D, DT[t], stride), new(N, K, torch.float32, 0)
        tbe.tbe_expert_combine_backward(desc, dout, rows, plan.slots, w, dys, dw)
        close(dw, prod.sum(2), (D + 2) * U32 * prod.abs().sum(2), "f32", "dw")
        dw2 = new(N, K, torch.float32, 0)
        tbe.tbe_expert_combine_backward(desc, dout, rows, plan.slots, w, rows, dw2)
        assert torch.equal(rows, dys), "dys"
        assert torch.equal(dw2, dw), "dw"
