"""AdamWState: the step writes through addresses that the state took when it was made, so
its buffers are what they were then, or the call is refused. No GPU is needed."""
import copy
import pickle
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")

NAMES = ("bits", "m_flat", "v_flat", "m", "v", "ms", "vs")


def state_of(bits, device=None):
    return tbe.AdamWState(tbe.AdamWDesc(bits=bits), [torch.zeros(3, 100, device=device), torch.zeros(7, device=device)])


@pytest.mark.parametrize("bits", [32, 8])
def test_buffers_cannot_be_exchanged(bits):
    s = state_of(bits)
    for name in NAMES + (("ms_flat", "vs_flat") if bits == 8 else ()):
        value = getattr(s, name)
        with pytest.raises(AttributeError, match="copy into"):
            setattr(s, name, value.clone() if isinstance(value, torch.Tensor) else value)
        with pytest.raises(AttributeError):
            delattr(s, name)
        assert getattr(s, name) is value
    with pytest.raises(TypeError):
        s.m[0] = torch.zeros(3, 100)
    # what is meant instead
    s.v_flat.copy_(torch.ones(s.v_flat.shape).to(s.v_flat.dtype))
    assert (s.v[1].float() == 1).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_copies_that_would_share_addresses_are_refused(bits):
    for make in (copy.deepcopy, pickle.dumps):
        with pytest.raises((TypeError, ValueError)):
            make(state_of(bits))


@pytest.mark.parametrize("bits", [32, 8])
def test_buffers_whose_memory_was_exchanged_are_refused(bits):
    """By `data`, the one way left, for each buffer in turn."""
    for name in ("m_flat", "v_flat") + (("ms_flat", "vs_flat") if bits == 8 else ()):
        s = state_of(bits)
        params = [torch.zeros(3, 100), torch.zeros(7)]
        flat = getattr(s, name)
        flat.data = flat.clone()
        with pytest.raises(TypeError, match="state: its buffers"):
            tbe.tbe_adamw_step(tbe.AdamWDesc(gdtype="f32", bits=bits), params, params, s, None, None)


SHAPES = [   # parameter's, gradient's or copy's, whether they belong together
    ((3, 100), (3, 100), True), ((3, 100), (300,), True), ((300,), (3, 100), True), ((1, 300), (300,), True),
    ((3, 100), (100, 3), False), ((3, 100), (30, 10), False), ((3, 100), (1, 3, 100), False),
    ((2, 3, 50), (3, 2, 50), False), ((2, 150), (2, 3, 50), False)]


@pytest.mark.parametrize("p,other,fits", SHAPES)
def test_gradients_and_copies_have_their_parameters_shape(p, other, fits):
    """Or are flat, or their parameter is: in the order of memory."""
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")   # torch's on the address of a tensor without memory
        desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", cdtype="bf16")

        def new(shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda:0")
        one = [new(p)]
        state = tbe.AdamWState(desc, one)
        step, lr = new(1, torch.int64), new(1)
        stream = types.SimpleNamespace(cuda_stream=64, device_index=0)
        for grads, copies, name in (([new(other)], [new(p, torch.bfloat16)], "grads"),
                                    ([new(p)], [new(other, torch.bfloat16)], "copies")):
            # (tensors without memory that are accepted end with the library's refusal of null pointers)
            with pytest.raises(tbe.TbeError if fits else TypeError) as e:
                tbe.tbe_adamw_step(desc, one, grads, state, step, lr, None, copies, stream)
            if not fits:
                assert f"{name}: expected its parameter's shape" in str(e.value)
