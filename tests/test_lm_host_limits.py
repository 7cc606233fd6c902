"""Language-model operators: limits of the descriptions and refusals of the
compiled calls that need no GPU."""
import ctypes

import pytest
import torch

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
from bwd_tbe_pooled_amd import _lmcall, lm  # noqa: E402


def test_widths_are_limited():
    for d, f, args in ((tbe.TokenDesc(0, 4, 2 ** 28), lm._token_forward, [1 << 20, 2 ** 28, None, None, 2 ** 28]),
                       (tbe.ExpertDesc(0, 1, 1, 2 ** 28), lm._expert_dispatch, [None, 2 ** 28, None, None, 2 ** 28])):
        assert f(d.ref, *args, None) == tbe.TBE_OK
        d.c.D = 2 ** 28 + 1
        assert f(d.ref, *args, None) == tbe.TBE_ERR_UNSUPPORTED


def test_workspace_of_more_tokens_is_no_smaller():
    sizes = [lm._token_workspace_bytes(tbe.TokenDesc(n, 1000, 64).ref)
             for n in (0, 1, 1024, 1025, 4096, 4097, 65536, 1 << 20)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_calls_refuse_a_wrong_number_of_arguments():
    d = tbe.TokenDesc(4, 10, 8)
    with pytest.raises(TypeError, match="expected 5 arguments, got 2"):
        _lmcall.token_forward(d.ref, None)
    with pytest.raises(TypeError):
        _lmcall.bind(())
    with pytest.raises(TypeError, match="expected a description"):
        _lmcall.token_forward(0, None, None, None, None)


@pytest.mark.parametrize("call,n", [("expert_plan", 5), ("expert_dispatch", 3), ("expert_combine", 4),
                                    ("expert_dispatch_backward", 3), ("expert_combine_backward", 6)])
def test_expert_calls_refuse_host_tensors(call, n):
    d = tbe.ExpertDesc(2, 2, 3, 8)
    with pytest.raises(TypeError, match="must be a device tensor"):
        getattr(_lmcall, call)(d.ref, *[torch.zeros(1)] * n, None)


@pytest.mark.parametrize("call,n", [("distill_forward", 6), ("distill_backward", 6), ("distill_step", 7)])
def test_distill_calls_refuse_host_tensors(call, n):
    d = tbe.DistillDesc(2, 30, 3)
    with pytest.raises(TypeError, match="x: must be a device tensor"):
        getattr(_lmcall, call)(d.ref, *[torch.zeros(1)] * n, None)
    with pytest.raises(TypeError, match="x: expected a torch.Tensor, got int"):
        getattr(_lmcall, call)(d.ref, *[3] * n, None)
    assert ctypes.sizeof(lm.tbe_distill_desc) == ctypes.sizeof(d.c)
