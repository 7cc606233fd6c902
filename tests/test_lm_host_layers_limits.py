"""Layer norm, experts' feed-forward and AdamW: limits and refusals that need no GPU, at the
values next to them."""
import ctypes
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
from tests.test_lm_host_layers import OK, UNSUP, adamw, calls, ffn, lm, status, step  # noqa: E402


@pytest.mark.parametrize("eps,want", [(0.0, OK), (2.0 ** -126, OK), (1e-8, OK), (2.0 ** -126 * (1 - 2.0 ** -20), UNSUP),
                                      (1e-40, UNSUP), (1e-50, UNSUP), (5e-324, UNSUP)])
def test_adamw_refuses_an_eps_that_is_no_normal_number(eps, want):
    """0 / eps would be NaN: the parameters of elements without a gradient."""
    assert step(adamw(eps=eps)) == want


def test_ffn_rows_leave_room_for_a_tile():
    """A tile counts up to 256 rows from its first one in 32 bits, beyond the last row too."""
    def size(M):
        return lm._ffn_workspace_bytes(ctypes.byref(ffn(M=M, D=8, F=8)))
    assert size(2 ** 31 - 1025) > 0
    for M in (2 ** 31 - 1024, 2 ** 31 - 256, 2 ** 31 - 64, 2 ** 31 - 2):
        assert size(M) == 0
        d = ffn(M=M, D=8, F=8)
        for f, args, *_ in calls(d):
            assert status(f, d, args) == UNSUP, f.__name__


@pytest.mark.parametrize("D,F", [(0, 1), (1, 0), (0, 0), (0, 5), (5, 0)])
def test_matrices_without_columns_are_refused(D, F):
    """By the description's check, after the tensors': their rows' strides may be zero."""
    M, E = 3, 1
    d = tbe.FfnDesc(M, E, D, F)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")   # torch's on the address of a tensor without memory

        def new(*shape, dtype=torch.bfloat16):
            return torch.empty(shape, dtype=dtype, device="cuda:0")
        x, pre, offsets = new(M, D), new(M, 2 * F), new(E + 1, dtype=torch.int32)
        ws = new(1 << 20, dtype=torch.uint8)
        gate, down = new(E, F, D), new(E, D, F)
        stream = types.SimpleNamespace(cuda_stream=64, device_index=0)
        for w in (gate, gate.as_strided(gate.shape, (0, 0, 1))):
            with pytest.raises((tbe.TbeError, TypeError)):
                tbe.tbe_ffn_backward(d, x, x, offsets, gate, gate, down, pre, x, w, w, down, ws, stream)
        with pytest.raises(tbe.TbeError) as e:
            tbe.tbe_ffn_forward(d, x, offsets, gate, gate, down, pre, x, ws, stream)
        assert e.value.status == tbe.TBE_ERR_ARG
