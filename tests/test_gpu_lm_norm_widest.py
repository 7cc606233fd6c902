"""The norm's gradients up to the widest rows: a launch has less than 2^32 threads, and the
columns' sums are joined by 1024 for 16 columns."""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import F64, U32, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


# beyond 2^19 columns a workgroup of the join takes 16 columns more than once
@pytest.mark.parametrize("N,D,w", [(3, 1 << 19, "f32"), (3, (1 << 19) + 1, "bf16"), (70, 600007, "f32"),
                                   (2, 1 << 25, "f32"), (3, (1 << 25) + 5, "bf16"), (1, 1 << 28, "f32")])
def test_widest(N, D, w):
    """db is a sum of N rows of bf16 in float32. dw is dy xh: the mean and the deviation are
    sums of D / 1024 values in a lane and 16 more, as for other widths."""
    say("norm widest", N, D, w)
    tbe = lib()
    g = torch.Generator(device="cuda")
    g.manual_seed(N + D)
    x = torch.randn(N, D, generator=g, device="cuda", dtype=torch.bfloat16)
    dy = torch.randn(N, D, generator=g, device="cuda", dtype=torch.bfloat16)
    wt = {"f32": torch.float32, "bf16": torch.bfloat16}[w]
    d = tbe.NormDesc(N, D, wdtype=w)
    y, dx, stats = torch.empty_like(x), torch.empty_like(x), torch.empty(N, 2, device="cuda")
    dw, db = (torch.full((D,), float("nan"), device="cuda", dtype=wt) for _ in "wb")
    tbe.tbe_norm_forward(d, x, None, None, y, stats)
    ws = tbe.norm_workspace(d)
    tbe.tbe_norm_backward(d, dy, x, None, stats, dx, dw, db, ws)
    torch.cuda.synchronize()
    del ws, y, dx
    half = torch.finfo(wt).eps / 2
    want, size = torch.zeros(D, dtype=F64, device="cuda"), torch.zeros(D, dtype=F64, device="cuda")
    for row in dy:
        want += row
        size += row.abs()
    assert ((db.to(F64) - want).abs() <= N * U32 * size + half * want.abs()).all()
    want.zero_()
    size.zero_()
    n = D / 512 + 64
    for row, up in zip(x, dy):
        xh = row.to(F64)
        xh -= xh.mean()
        xh *= 1 / torch.sqrt(xh.square().mean() + 1e-5)
        want += up * xh
        size += up.abs() * (xh.abs() + 1)
    assert ((dw.to(F64) - want).abs() <= (n + N) * U32 * size * (1 + half) + half * want.abs()).all()
