"""Layer norm, experts' feed-forward and AdamW: limits and refusals that need no GPU, at the
values next to them."""
import ctypes

import pytest

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
