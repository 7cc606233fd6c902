"""Layer norm, experts' feed-forward and AdamW: limits and refusals that need no GPU, at the
values next to them."""
import pytest

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
from tests.test_lm_host_layers import OK, UNSUP, adamw, step  # noqa: E402


@pytest.mark.parametrize("eps,want", [(0.0, OK), (2.0 ** -126, OK), (1e-8, OK), (2.0 ** -126 * (1 - 2.0 ** -20), UNSUP),
                                      (1e-40, UNSUP), (1e-50, UNSUP), (5e-324, UNSUP)])
def test_adamw_refuses_an_eps_that_is_no_normal_number(eps, want):
    """0 / eps would be NaN: the parameters of elements without a gradient."""
    assert step(adamw(eps=eps)) == want
