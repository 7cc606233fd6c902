"""Layer norm, experts' feed-forward and AdamW: refusals and sizes that need no GPU.
Every call here is refused on the host before anything is enqueued, or has nothing
to do; the pointers stand for device memory that is never touched."""
import ctypes
import types
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
from bwd_tbe_pooled_amd import _lmcall, lm  # noqa: E402

OK, ARG, UNSUP, WS = (tbe.TBE_OK, tbe.TBE_ERR_ARG, tbe.TBE_ERR_UNSUPPORTED, tbe.TBE_ERR_WORKSPACE)
P = 1 << 20     # stands for a device pointer
BIG = 1 << 50   # workspace bytes


def fields(struct, **kw):
    for k, v in kw.items():
        setattr(struct, k, v)
    return struct


def norm(**kw):
    return fields(lm.tbe_norm_desc(N=5, D=16, dtype=2, wdtype=0, eps=1e-5), **kw)


def ffn(**kw):
    return fields(lm.tbe_ffn_desc(M=5, E=3, D=16, F=32, dtype=2, act=0), **kw)


def adamw(**kw):
    return fields(lm.tbe_adamw_desc(pdtype=0, gdtype=2, cdtype=-1, bits=32, beta1=0.9, beta2=0.99, eps=1e-8,
                                    weight_decay=0.1), **kw)


def stack(ld, stride, data=P):
    return ctypes.byref(lm.tbe_stack(data, ld, stride))


GATE, DOWN = (16, 512), (32, 512)


def calls(d):
    """(name, arguments without desc and stream, indexes of required pointers, of row strides,
    of output row strides with their widths)"""
    if isinstance(d, lm.tbe_norm_desc):
        return [(lm._norm_forward, [P, 16, P, P, P, 16, P], [0, 4, 6], [1, 5], [(5, 16)]),
                (lm._norm_backward, [P, 16, P, 16, P, P, P, 16, P, P, P, BIG], [0, 2, 5, 6], [1, 3, 7], [(7, 16)])]
    g, u, w = stack(*GATE), stack(*GATE), stack(*DOWN)
    return [(lm._ffn_forward, [P, 16, P, g, u, w, P, 64, P, 16, P, BIG], [0, 2, 3, 4, 5, 8], [1, 7, 9],
             [(7, 64), (9, 16)]),
            (lm._ffn_backward, [P, 16, P, 16, P, g, u, w, P, 64, P, 16, g, u, w, P, BIG],
             [0, 2, 4, 5, 6, 7, 8, 10, 12, 13, 14], [1, 3, 9, 11], [(11, 16)])]


def status(f, d, args):
    return f(ctypes.byref(d) if d is not None else None, *args, None)


NAN, INF = float("nan"), float("inf")
BAD = [(norm(N=-1), ARG), (norm(D=0), ARG), (norm(eps=-1e-5), ARG), (norm(eps=NAN), ARG), (norm(eps=INF), ARG),
       (norm(dtype=3), UNSUP), (norm(wdtype=-1), UNSUP), (norm(N=2 ** 31 - 1), UNSUP), (norm(D=2 ** 28 + 1), UNSUP),
       (ffn(M=-1), ARG), (ffn(E=0), ARG), (ffn(D=0), ARG), (ffn(F=-3), ARG), (ffn(act=2), ARG), (ffn(act=-1), ARG),
       (ffn(dtype=4), UNSUP), (ffn(E=1024), UNSUP), (ffn(D=65537), UNSUP), (ffn(F=65537), UNSUP),
       (ffn(M=2 ** 31 - 1), UNSUP), (ffn(M=2 ** 25, D=4096), UNSUP), (ffn(M=2 ** 25, F=2048), UNSUP),
       (ffn(E=1000, D=16384, F=8192), UNSUP)]


@pytest.mark.parametrize("d,want", BAD)
def test_bad_descriptions_are_refused(d, want):
    for f, args, *_ in calls(d):
        assert status(f, d, args) == want, f.__name__
    size = lm._norm_workspace_bytes if isinstance(d, lm.tbe_norm_desc) else lm._ffn_workspace_bytes
    assert size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("d", [norm(), ffn()], ids=["norm", "ffn"])
def test_bad_arguments_are_refused(d):
    for f, args, pointers, strides, outputs in calls(d):
        def with_(i, v):
            return args[:i] + [v] + args[i + 1:]
        assert status(f, None, args) == ARG
        for i in pointers:
            assert status(f, d, with_(i, None)) == ARG, (f.__name__, i)
        for i in strides:
            assert status(f, d, with_(i, -1)) == ARG, (f.__name__, i)
        for i, width in outputs:
            assert status(f, d, with_(i, width - 1)) == ARG, (f.__name__, i)
        if args[-1] == BIG:
            assert status(f, d, args[:-2] + [None, BIG]) == WS, f.__name__
            assert status(f, d, args[:-2] + [P, 8]) == WS, f.__name__
            assert status(f, d, args[:-2] + [P + 64, BIG]) == ARG, f.__name__


def test_stacks_of_matrices():
    """Inputs may share matrices; the matrices and rows of an output must be apart."""
    d = ffn(M=0)
    for f, args, *_ in calls(d):
        for i in ((3, 4, 5) if f is lm._ffn_forward else (5, 6, 7)):
            for ld, stride, data in ((-1, 512, P), (16, -1, P), (16, 512, None)):
                assert status(f, d, args[:i] + [stack(ld, stride, data)] + args[i + 1:]) == ARG, (f.__name__, i)
    args = calls(d)[1][1]
    for i, rows, cols in ((12, 32, 16), (13, 32, 16), (14, 16, 32)):
        for ld, stride in ((cols - 1, 10 ** 6), (cols, rows * cols - 1), (cols + 8, rows * (cols + 8) - 1), (cols, 0)):
            assert status(lm._ffn_backward, d, args[:i] + [stack(ld, stride)] + args[i + 1:]) == ARG
    one = ffn(M=0, E=1)   # of one matrix the distance to the next says nothing
    assert status(lm._ffn_forward, one, [None, 16, P, stack(0, 0), stack(16, 0), stack(32, 0), None, 0, None, 16,
                                         P, BIG]) == OK


def test_empty_calls_succeed_without_buffers():
    assert status(lm._norm_forward, norm(N=0), [None, 16, None, None, None, 16, None]) == OK
    assert status(lm._norm_backward, norm(N=0), [None, 16, None, 16, None, None, None, 16, None, None, P, BIG]) == OK
    assert status(lm._ffn_forward, ffn(M=0), [None, 16, P, stack(*GATE), stack(*GATE), stack(*DOWN), None, 0, None,
                                              16, P, BIG]) == OK


def test_workspace_sizes():
    def n(**kw):
        return lm._norm_workspace_bytes(ctypes.byref(norm(**kw)))
    assert n(N=0) >= 256 and n(N=10 ** 6, D=4096) >= 2 * 4 * 4096 * 256
    assert n(N=10 ** 6, D=2 ** 28) < 2 ** 33     # a partial row or two of the widest
    def w(**kw):
        return lm._ffn_workspace_bytes(ctypes.byref(ffn(**kw)))
    assert w(M=0) >= 256 and w(M=1000, F=96) >= 1000 * 96 * 3 * 2 and w(M=1000, F=97, dtype=0) >= 1000 * 97 * 3 * 4
    for make in (lambda: tbe.norm_workspace(tbe.NormDesc(4, 0)), lambda: tbe.ffn_workspace(tbe.FfnDesc(4, 0, 8, 8))):
        with pytest.raises(tbe.TbeError) as e:
            make()
        assert e.value.status == ARG


# --- AdamW ---------------------------------------------------------------------------
def tensor(n=10, p=P, m=P, **kw):
    return fields(lm.tbe_adamw_tensor(p=p, g=P, m=m, v=P, mscale=P, vscale=P, c=P, n=n), **kw)


def step(d, *tensors, count=None, step=P, lr=P):
    t = (lm.tbe_adamw_tensor * max(1, len(tensors)))(*tensors)
    return status(lm._adamw_step, d, [t, len(tensors) if count is None else count, step, lr, None])


@pytest.mark.parametrize("d,want", [
    (adamw(bits=16), ARG), (adamw(beta1=1.0), ARG), (adamw(beta1=-0.1), ARG), (adamw(beta2=NAN), ARG),
    (adamw(beta2=1.5), ARG), (adamw(eps=-1e-9), ARG), (adamw(eps=INF), ARG), (adamw(eps=1e300), ARG),
    (adamw(weight_decay=-1.0), ARG), (adamw(weight_decay=NAN), ARG), (adamw(pdtype=3), UNSUP), (adamw(gdtype=-1), UNSUP),
    (adamw(cdtype=0), UNSUP), (adamw(cdtype=3), UNSUP), (adamw(pdtype=2, cdtype=1), UNSUP)])
def test_adamw_descriptions(d, want):
    assert step(d) == want


def test_adamw_arguments():
    d = adamw(cdtype=2, bits=8)
    assert step(None) == ARG and step(d, count=-1) == ARG and step(d, count=1 << 24) == UNSUP
    assert status(lm._adamw_step, d, [None, 1, P, P, None]) == ARG
    assert step(d, tensor(n=-1)) == ARG and step(d, tensor(n=1 << 40)) == UNSUP
    for name in ("p", "g", "m", "v", "mscale", "vscale", "c"):
        assert step(d, tensor(**{name: None})) == ARG, name
    assert step(d, tensor(m=P + 4)) == ARG and step(d, tensor(v=P + 1)) == ARG
    assert step(d, tensor(), step=None) == ARG and step(d, tensor(), lr=None) == ARG
    # nothing to do
    assert step(d) == OK and step(d, tensor(n=0, p=None), tensor(n=0)) == OK


def test_adamw_refuses_parameters_that_overlap():
    d, c = adamw(), adamw(cdtype=1)
    far = [tensor(p=P + 4096 * i, c=P + 4096 * i, n=1024) for i in range(4)]
    assert step(d, *far[::-1], tensor(p=P + 4 * 1023, n=1)) == ARG
    assert step(d, far[0], far[0]) == ARG
    assert step(d, far[1], tensor(p=P + 2048, n=1000)) == ARG
    assert step(c, *[fields(t, p=P + 8192 * i) for i, t in enumerate(far)], tensor(p=P + 2 ** 19, c=P + 10, n=1)) == ARG


# --- Python calls ----------------------------------------------------------------------
DESCS = {"norm": tbe.NormDesc(5, 8), "ffn": tbe.FfnDesc(5, 2, 8, 4), "adamw": tbe.AdamWDesc(),
         "token": tbe.TokenDesc(5, 40, 8), "nothing": None}
CALLS = [("tbe_norm_forward", 5), ("tbe_norm_backward", 8), ("tbe_ffn_forward", 8), ("tbe_ffn_backward", 12),
         ("tbe_adamw_step", 5), ("norm_workspace", 0), ("ffn_workspace", 0), ("AdamWState", 1)]


@pytest.mark.parametrize("call,n", CALLS)
def test_another_operators_description_is_refused(call, n):
    operator = next(k for k in DESCS if k in call.lower())
    kind = type(DESCS[operator]).__name__
    for other, desc in DESCS.items():
        if other != operator:
            with pytest.raises(TypeError, match=f"desc: expected {kind}, got {type(desc).__name__}"):
                getattr(tbe, call)(desc, *[None] * n)


@pytest.mark.parametrize("make", [
    lambda big: tbe.NormDesc(5, big + 8), lambda big: tbe.NormDesc(big * big + 5, 8), lambda big: tbe.FfnDesc(5, big + 2, 8, 8),
    lambda big: tbe.FfnDesc(5, 2, big + 8, 8), lambda big: tbe.FfnDesc(5, 2, 8, big + 8),
    lambda big: tbe.AdamWDesc(bits=big + 32)])
def test_sizes_beyond_their_field_are_refused(make):
    with pytest.raises(tbe.TbeError, match="= [0-9]{10}") as e:
        make(2 ** 32)
    assert e.value.status == UNSUP
    make(0)


def test_names_that_are_none():
    for make in (lambda: tbe.FfnDesc(5, 2, 8, 8, act="relu"), lambda: tbe.NormDesc(5, 8, wdtype="f64"),
                 lambda: tbe.AdamWDesc(cdtype="f8")):
        with pytest.raises(KeyError):
            make()
    with pytest.raises(tbe.TbeError):
        tbe.AdamWState(tbe.AdamWDesc(bits=4), [])


F, B, I, L, U, F8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8, torch.float8_e4m3fn
M, E, D, H = 5, 2, 8, 16
W = ((1 << 20,), U)
UP, DN = ((E, H, D), B), ((E, D, H), B)
TENSORS = [   # call, description, shapes and types of its tensors
    ("tbe_norm_forward", tbe.NormDesc(M, D), [((M, D), B), ((D,), F), ((D,), F), ((M, D), B), ((M, 2), F)]),
    ("tbe_norm_backward", tbe.NormDesc(M, D),
     [((M, D), B), ((M, D), B), ((D,), F), ((M, 2), F), ((M, D), B), ((D,), F), ((D,), F), W]),
    ("tbe_ffn_forward", tbe.FfnDesc(M, E, D, H),
     [((M, D), B), ((E + 1,), I), UP, UP, DN, ((M, 2 * H), B), ((M, D), B), W]),
    ("tbe_ffn_backward", tbe.FfnDesc(M, E, D, H),
     [((M, D), B), ((M, D), B), ((E + 1,), I), UP, UP, DN, ((M, 2 * H), B), ((M, D), B), UP, UP, DN, W])]


def stream_on(device):
    return types.SimpleNamespace(cuda_stream=64, device_index=device)


@pytest.mark.parametrize("name,desc,shapes", TENSORS)
def test_tensors_of_another_device_shape_or_type_are_refused(name, desc, shapes):
    def call(tensors, stream):
        with warnings.catch_warnings():
            warnings.simplefilter("ignore")   # torch's on the address of a tensor without memory
            getattr(tbe, name)(desc, *tensors, stream)
    with FakeTensorMode():
        def make(devices, change=()):
            out = []
            for i, ((s, t), d) in enumerate(zip(shapes, devices)):
                if i in change:
                    s, t = change[i]
                out.append(torch.empty(s, dtype=t, device=f"cuda:{d}"))
            return out
        for one in range(2):
            same = [one] * len(shapes)
            with pytest.raises(tbe.TbeError) as e:
                call(make(same), stream_on(one))
            assert e.value.status in (ARG, WS)
            for i in range(1, len(shapes)):
                with pytest.raises(TypeError, match="must be on the device of the call's other tensors"):
                    call(make([1 - one if j == i else one for j in range(len(shapes))]), stream_on(one))
            with pytest.raises(TypeError, match="stream: must be of the tensors' device"):
                call(make(same), stream_on(1 - one))
        zero = [0] * len(shapes)
        for i, (s, t) in enumerate(shapes):
            if shapes[i] is W:
                continue
            with pytest.raises(TypeError, match="expected shape"):
                call(make(zero, {i: (s[:-1] + (s[-1] + 1,), t)}), stream_on(0))
            with pytest.raises(TypeError, match="expected torch"):
                call(make(zero, {i: (s, F if t is not F else B)}), stream_on(0))


def test_calls_refuse_host_tensors_and_wrong_counts():
    d = tbe.NormDesc(2, 8)
    with pytest.raises(TypeError, match="x: must be a device tensor"):
        tbe.tbe_norm_forward(d, torch.zeros(2, 8, dtype=B), None, None, None, None)
    with pytest.raises(TypeError, match="expected 10 arguments, got 2"):
        _lmcall.norm_backward(d.ref, None)
    with pytest.raises(TypeError, match="xs: expected a torch.Tensor"):
        tbe.tbe_ffn_forward(tbe.FfnDesc(2, 1, 8, 8), 3, *[None] * 7)


def test_adamw_state():
    """Moments of each tensor, views of one buffer in whole blocks, zero before the first step."""
    params = [torch.zeros(3, 100), torch.zeros(256), torch.zeros(0), torch.zeros(1)]
    for bits, kind in ((32, F), (8, F8)):
        s = tbe.AdamWState(tbe.AdamWDesc(bits=bits), params)
        assert s.m_flat.dtype == kind and s.m_flat.numel() == 256 * 4 and not s.m_flat.float().any()
        assert [tuple(m.shape) for m in s.m] == [(3, 100), (256,), (0,), (1,)]
        assert [v.storage_offset() for v in s.v] == [0, 512, 768, 768]
        if bits == 8:
            assert [x.numel() for x in s.ms] == [2, 1, 0, 1] and s.vs_flat.numel() == 4
        else:
            assert s.ms is None
    with pytest.raises(TypeError, match="state: expected an AdamWState of the description's bits"):
        tbe.tbe_adamw_step(tbe.AdamWDesc(bits=32), params, params, s, None, None)
    with pytest.raises(TypeError, match="state: must be a device tensor"):
        tbe.tbe_adamw_step(tbe.AdamWDesc(bits=8), params, params, s, None, None)


def test_adamw_state_of_an_iterator():
    params = [torch.zeros(3, 5), torch.zeros(300)]
    s = tbe.AdamWState(tbe.AdamWDesc(bits=8), (p for p in params))
    assert [m.shape for m in s.m] == [p.shape for p in params]
    assert s.m_flat.device == params[0].device and len(s.ms[1]) == 2
