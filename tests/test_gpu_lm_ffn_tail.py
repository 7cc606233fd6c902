"""The experts' activations far below zero, where their values are small against 1."""
import math

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, TINY, U32, half
from tests.test_gpu_lm_ffn import ACT, act

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_tail(name, t):
    """One column with every matrix 1 and rows g: ys = act(g) g and no sum in between.
    Relative to act(g): ACT (|g| + 1) for the exponential, and for GELU's exp(-g^2 / 2) and
    complement of the error function a rounding of the exponent, (g^2 + 2) u, and 16
    roundings. dg is a difference of two terms near GELU's minimum: relative to both."""
    tbe = lib()
    low = -4.0 if t == "f16" else -9.0     # (f16 holds no smaller values)
    x = torch.linspace(low, 3.0, 1201, device="cuda").to(DT[t])[:, None].contiguous()
    M = x.shape[0]
    d = tbe.FfnDesc(M, 1, 1, 1, dtype=t, act=name)
    one = torch.ones(1, 1, 1, dtype=DT[t], device="cuda")
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    ys, pre, dxs = torch.empty_like(x), torch.empty(M, 2, dtype=DT[t], device="cuda"), torch.empty_like(x)
    ws = tbe.ffn_workspace(d)
    tbe.tbe_ffn_forward(d, x, offsets, one, one, one, pre, ys, ws)
    dw = [torch.empty_like(one) for _ in range(3)]
    tbe.tbe_ffn_backward(d, torch.ones_like(x), x, offsets, one, one, one, pre, dxs, *dw, ws)
    torch.cuda.synchronize()
    g = x.to(F64)[:, 0]
    a, _ = act(name, g)
    rel = ACT * (g.abs() + 1) + 16 * U32 + ((g * g + 2) * U32 if name == "gelu" else 0)
    h = half(t)
    off = (rel + 2 * h + h * h) * (a * g).abs() + 2 * TINY[t]
    err = (ys.to(F64)[:, 0] - a * g).abs()
    assert (err <= off).all(), f"ys at {g[(err / off).argmax()].item()}: {(err / off).max().item():.3g} of the bound"
    # dxs = dg + du, du = a, dg = u act'(g) = g (a / g + the slope's other part)
    if name == "silu":
        s = torch.sigmoid(g)
        parts = (s, s * g * (1 - s))
    else:
        parts = (0.5 * torch.erfc(-g / math.sqrt(2)), g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi))
    want = a + g * (parts[0] + parts[1])
    size = a.abs() + g.abs() * (parts[0].abs() + parts[1].abs())
    off = (rel + 2 * h + 8 * U32) * size + h * want.abs() + 4 * TINY[t]
    err = (dxs.to(F64)[:, 0] - want).abs()
    assert (err <= off).all(), f"dxs at {g[(err / off).argmax()].item()}: {(err / off).max().item():.3g} of the bound"
