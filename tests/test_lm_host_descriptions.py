"""Language-model operators: a call takes its own operator's description alone.
Refused on the host; no GPU is needed."""
import pytest

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")

DESCS = {"token": tbe.TokenDesc(5, 40, 8), "expert": tbe.ExpertDesc(5, 2, 4, 8),
         "distill": tbe.DistillDesc(5, 40, 8), "table": tbe.Desc(T=1, D=8, B=5, rows=[40], dtype="f32"),
         "nothing": None}
# call, its arguments beside the description
CALLS = [("tbe_token_forward", 3), ("tbe_token_backward", 4), ("tbe_expert_plan", 3), ("tbe_expert_dispatch", 3),
         ("tbe_expert_dispatch_backward", 3), ("tbe_expert_combine", 4), ("tbe_expert_combine_backward", 6),
         ("tbe_distill_forward", 6), ("tbe_distill_backward", 6), ("tbe_distill_step", 7),
         ("token_workspace", 0), ("expert_workspace", 0), ("distill_workspace", 0), ("ExpertPlan", 0)]


@pytest.mark.parametrize("call,n", CALLS)
def test_another_operators_description_is_refused(call, n):
    operator = next(k for k in DESCS if k in call.lower())
    kind = type(DESCS[operator]).__name__
    for other, desc in DESCS.items():
        if other != operator:
            with pytest.raises(TypeError, match=f"desc: expected {kind}, got {type(desc).__name__}"):
                getattr(tbe, call)(desc, *[None] * n)


def test_a_subclass_is_taken():
    class Mine(tbe.TokenDesc):
        pass
    with pytest.raises(TypeError, match="W: expected a torch.Tensor"):
        tbe.tbe_token_forward(Mine(5, 40, 8), None, None, None)


@pytest.mark.parametrize("make", [
    lambda big: tbe.TokenDesc(5, 40, big + 8), lambda big: tbe.ExpertDesc(5, big + 2, 4, 8),
    lambda big: tbe.ExpertDesc(5, 2, big + 4, 8), lambda big: tbe.ExpertDesc(5, 2, 4, big + 8),
    lambda big: tbe.DistillDesc(5, 40, big + 8), lambda big: tbe.TokenDesc(big * big + 5, 40, 8),
    lambda big: tbe.DistillDesc(5, big * big + 40, 8)])
def test_sizes_beyond_their_field_are_refused(make):
    """2^32 + 8 columns are not 8 columns."""
    with pytest.raises(tbe.TbeError, match="= [0-9]{10}") as e:
        make(2 ** 32)
    assert e.value.status == tbe.TBE_ERR_UNSUPPORTED
    make(0)


def test_temperatures_without_a_factor_are_refused():
    """log2(e) / temperature has to be a float32."""
    from bwd_tbe_pooled_amd import lm
    for t, want in ((1e-45, tbe.TBE_ERR_UNSUPPORTED), (4.2e-39, tbe.TBE_ERR_UNSUPPORTED), (4.3e-39, tbe.TBE_OK),
                    (3.4e38, tbe.TBE_OK), (1e-46, tbe.TBE_ERR_ARG)):   # (1e-46 is 0 in float32)
        d = tbe.DistillDesc(0, 5, 2, temperature=t)
        assert lm._distill_backward(d.ref, None, 5, None, None, None, None, None, 5, None) == want, t
        assert (lm._distill_workspace_bytes(d.ref) > 0) == (want == tbe.TBE_OK)
