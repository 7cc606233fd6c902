"""Language-model operators: refusals and sizes that need no GPU. Every call
here is refused on the host before anything is enqueued; the pointers stand
for device memory that is never touched."""
import ctypes

import pytest
import torch

tbe = pytest.importorskip("bwd_tbe_pooled_amd", reason="libtbe.so not built")
from bwd_tbe_pooled_amd import lm  # noqa: E402

OK, ARG, UNSUP, WS = (tbe.TBE_OK, tbe.TBE_ERR_ARG, tbe.TBE_ERR_UNSUPPORTED, tbe.TBE_ERR_WORKSPACE)
P = 1 << 20     # stands for a device pointer
BIG = 1 << 40   # workspace bytes


def token(**kw):
    d = lm.tbe_token_desc(N=5, V=100, D=16, wdtype=2, xdtype=2, idx64=1, scale=1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def expert(**kw):
    d = lm.tbe_expert_desc(N=5, K=2, E=8, D=16, dtype=2, idx64=1)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def distill(**kw):
    d = lm.tbe_distill_desc(N=5, V=100, K=4, dtype=2, tdtype=0, idx64=1, temperature=1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return d


def calls(d):
    """(name, arguments without desc and stream, indexes of required pointers,
    indexes of output row strides)"""
    if isinstance(d, lm.tbe_token_desc):
        return [(lm._token_forward, [P, 16, P, P, 16], [0, 2, 3], [4]),
                (lm._token_backward, [P, 16, P, P, 16, P, BIG], [0, 2, 3], [4])]
    if isinstance(d, lm.tbe_expert_desc):
        return [(lm._expert_plan, [P, P, P, P, P, BIG], [0, 1, 2, 3], []),
                (lm._expert_dispatch, [P, 16, P, P, 16], [0, 2, 3], [4]),
                (lm._expert_dispatch_backward, [P, 16, P, P, 16], [0, 2, 3], [4]),
                (lm._expert_combine, [P, 16, P, P, P, 16], [0, 2, 3, 4], [5]),
                (lm._expert_combine_backward, [P, 16, 2 * P, 16, P, P, P, 16, P],
                 [0, 2, 4, 5, 6, 8], [7])]
    return [(lm._distill_forward, [P, 100, P, P, P, P, P, BIG], [0, 2, 3, 4, 5], []),
            (lm._distill_backward, [P, 100, P, P, P, P, 2 * P, 100], [0, 2, 3, 4, 5, 6], [7]),
            (lm._distill_step, [P, 100, P, P, P, P, 2 * P, 100, P, BIG], [0, 2, 3, 4, 5, 6], [7])]


def status(f, d, args):
    return f(ctypes.byref(d) if d is not None else None, *args, None)


BAD = [(token(N=-1), ARG), (token(V=0), ARG), (token(D=0), ARG), (token(idx64=2), ARG),
       (token(wdtype=3), UNSUP), (token(xdtype=7), UNSUP), (token(N=1 << 30), UNSUP),
       (token(V=1023 * 1024 + 1), UNSUP),
       (expert(N=-1), ARG), (expert(K=0), ARG), (expert(E=0), ARG), (expert(D=-4), ARG),
       (expert(idx64=-1), ARG), (expert(dtype=9), UNSUP), (expert(K=65), UNSUP),
       (expert(E=1024), UNSUP), (expert(N=1 << 30, K=2), UNSUP), (expert(N=2 ** 62, K=4), UNSUP),
       (distill(N=-2), ARG), (distill(V=0), ARG), (distill(K=0), ARG), (distill(idx64=3), ARG),
       (distill(temperature=0.0), ARG), (distill(temperature=-1.0), ARG),
       (distill(temperature=float("nan")), ARG), (distill(temperature=float("inf")), ARG),
       (distill(dtype=5), UNSUP), (distill(tdtype=-1), UNSUP), (distill(K=1025), UNSUP),
       (distill(V=2 ** 31 - 1), UNSUP), (distill(N=2 ** 31 - 1), UNSUP)]


@pytest.mark.parametrize("d,want", BAD)
def test_bad_descriptions_are_refused(d, want):
    for f, args, _, _ in calls(d):
        assert status(f, d, args) == want, f.__name__
    size = {lm.tbe_token_desc: lm._token_workspace_bytes,
            lm.tbe_expert_desc: lm._expert_workspace_bytes,
            lm.tbe_distill_desc: lm._distill_workspace_bytes}[type(d)]
    assert size(ctypes.byref(d)) == 0


@pytest.mark.parametrize("d", [token(), expert(), distill()], ids=["token", "expert", "distill"])
def test_bad_arguments_are_refused(d):
    for f, args, pointers, strides in calls(d):
        assert status(f, None, args) == ARG
        for i in pointers:
            assert status(f, d, args[:i] + [None] + args[i + 1:]) == ARG, (f.__name__, i)
        for i, a in enumerate(args):
            if a in (16, 100):
                assert status(f, d, args[:i] + [-1] + args[i + 1:]) == ARG, (f.__name__, i)
        for i in strides:
            assert status(f, d, args[:i] + [args[i] - 1] + args[i + 1:]) == ARG, (f.__name__, i)
        if args[-1] == BIG:
            assert status(f, d, args[:-2] + [None, BIG]) == WS, f.__name__
            assert status(f, d, args[:-2] + [P, 8]) == WS, f.__name__
            assert status(f, d, args[:-2] + [P + 64, BIG]) == ARG, f.__name__


def test_in_place_calls_need_equal_strides():
    d = expert()
    assert status(lm._expert_combine_backward, d, [P, 16, P, 16, P, P, P, 32, P]) == ARG
    d = distill()
    assert status(lm._distill_backward, d, [P, 100, P, P, P, P, P, 128]) == ARG
    assert status(lm._distill_step, d, [P, 100, P, P, P, P, P, 128, P, BIG]) == ARG


def test_empty_calls_succeed_without_buffers():
    d = token(N=0)
    assert status(lm._token_forward, d, [P, 16, None, None, 16]) == OK
    d = expert(N=0)
    for f in (lm._expert_dispatch, lm._expert_dispatch_backward):
        assert status(f, d, [None, 16, None, None, 16]) == OK
    assert status(lm._expert_combine, d, [None, 16, None, None, None, 16]) == OK
    assert status(lm._expert_combine_backward, d,
                  [None, 16, None, 16, None, None, None, 16, None]) == OK
    d = distill(N=0)
    assert status(lm._distill_backward, d, [None, 100, None, None, None, None, None, 100]) == OK


def test_workspace_sizes():
    def tok(**kw):
        return lm._token_workspace_bytes(ctypes.byref(token(**kw)))
    assert tok(N=0) >= 4 * 101
    assert tok(N=100000) >= tok(N=1000) >= tok(N=0)
    # partial rows: two per chunk of 64 sorted places
    assert tok(N=1 << 18, D=1024) >= 4 * 2 * 1024 * (1 << 12)
    assert lm._expert_workspace_bytes(ctypes.byref(expert())) >= 256
    assert lm._expert_workspace_bytes(ctypes.byref(expert(N=1 << 20))) >= 256 * 9 * 4
    assert lm._distill_workspace_bytes(ctypes.byref(distill())) >= 256
    with pytest.raises(tbe.TbeError) as e:
        tbe.token_workspace(tbe.TokenDesc(4, 0, 8))
    assert e.value.status == ARG


def test_binding_refuses_host_tensors():
    d = tbe.TokenDesc(4, 10, 8)
    W = torch.zeros(10, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="W: must be a device tensor"):
        tbe.tbe_token_forward(d, W, torch.zeros(4, dtype=torch.int64), torch.zeros(4, 8))
    with pytest.raises(TypeError, match="W: expected a torch.Tensor"):
        tbe.tbe_token_forward(d, [1.0], None, None)
    with pytest.raises(KeyError):
        tbe.TokenDesc(4, 10, 8, wdtype="f8")


def test_header_limits_match_the_library():
    assert status(lm._token_forward, token(V=1023 * 1024, N=0), [P, 16, None, None, 16]) == OK
    d = expert(N=0, K=64, E=1023)
    assert status(lm._expert_dispatch, d, [None, 16, None, None, 16]) == OK
    d = distill(N=0, K=1024, V=2 ** 31 - 2)
    assert status(lm._distill_backward, d,
                  [None, 2 ** 31, None, None, None, None, None, 2 ** 31]) == OK
