"""Language-model calls: tensors and stream of one device. Tensors here have a
device, shape and strides but no memory, so no GPU is needed: a call whose tensors
are accepted ends with the library's refusal of null pointers."""
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")

F, B, I, L, U = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8
N, V, D, K, E, M = 5, 40, 8, 2, 4, 10
W = ((1 << 20,), U)
CALLS = [   # call, description, shapes and types of its tensors
    ("tbe_token_forward", tbe.TokenDesc(N, V, D), [((V, D), B), ((N,), L), ((N, D), B)]),
    ("tbe_token_backward", tbe.TokenDesc(N, V, D), [((N, D), B), ((N,), L), ((V, D), B), W]),
    ("tbe_expert_plan", tbe.ExpertDesc(N, K, E, D), [((N, K), L), ((E + 1,), I), ((M,), I), ((M,), I), W]),
    ("tbe_expert_dispatch", tbe.ExpertDesc(N, K, E, D), [((N, D), B), ((M,), I), ((M, D), B)]),
    ("tbe_expert_dispatch_backward", tbe.ExpertDesc(N, K, E, D), [((M, D), B), ((M,), I), ((N, D), B)]),
    ("tbe_expert_combine", tbe.ExpertDesc(N, K, E, D), [((M, D), B), ((M,), I), ((N, K), F), ((N, D), B)]),
    ("tbe_expert_combine_backward", tbe.ExpertDesc(N, K, E, D),
     [((N, D), B), ((M, D), B), ((M,), I), ((N, K), F), ((M, D), B), ((N, K), F)]),
    ("tbe_distill_forward", tbe.DistillDesc(N, V, K),
     [((N, V), B), ((N, K), L), ((N, K), F), ((N,), F), ((N, 2), F), W]),
    ("tbe_distill_backward", tbe.DistillDesc(N, V, K),
     [((N, V), B), ((N, K), L), ((N, K), F), ((N, 2), F), ((N,), F), ((N, V), B)]),
    ("tbe_distill_step", tbe.DistillDesc(N, V, K),
     [((N, V), B), ((N, K), L), ((N, K), F), ((N,), F), ((N,), F), ((N, V), B), W])]


def call(name, desc, tensors, stream):
    if name == "tbe_expert_plan":
        ids, offsets, order, slots, ws = tensors
        tensors = [ids, types.SimpleNamespace(offsets=offsets, order=order, slots=slots), ws]
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")   # torch's on the address of a tensor without memory
        getattr(tbe, name)(desc, *tensors, stream)


def stream_on(device):
    return types.SimpleNamespace(cuda_stream=64, device_index=device)


@pytest.mark.parametrize("name,desc,shapes", CALLS)
def test_tensors_of_another_device_are_refused(name, desc, shapes):
    with FakeTensorMode():
        def make(devices):
            return [torch.empty(s, dtype=t, device=f"cuda:{d}") for (s, t), d in zip(shapes, devices)]
        for one in range(2):
            with pytest.raises(tbe.TbeError) as e:
                call(name, desc, make([one] * len(shapes)), stream_on(one))
            assert e.value.status in (tbe.TBE_ERR_ARG, tbe.TBE_ERR_WORKSPACE)
            for i in range(1, len(shapes)):
                devices = [one] * len(shapes)
                devices[i] = 1 - one
                with pytest.raises(TypeError, match="must be on the device of the call's other tensors"):
                    call(name, desc, make(devices), stream_on(one))
            with pytest.raises(TypeError, match="stream: must be of the tensors' device"):
                call(name, desc, make([one] * len(shapes)), stream_on(1 - one))
        # a handle without a device is taken at its word
        with pytest.raises(tbe.TbeError):
            call(name, desc, make([0] * len(shapes)), types.SimpleNamespace(cuda_stream=64))
