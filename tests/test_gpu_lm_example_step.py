"""examples/lm_distill.py with gated experts: the optimizer's steps of the whole model are
AdamW of the gradients that it returns, with moments of 32 and of 8 bits."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import F64, U32

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "lm_distill.py")


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()
    spec = importlib.util.spec_from_file_location("lm_distill", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_follow_the_gradients(example, bits, monkeypatch):
    """Each call of the optimizer in training, against the formula on what it was given. The
    move takes the moments before they are rounded to 8 bits; a moment is off by four
    roundings of its terms, the move by sixteen more."""
    tbe, lr, eps, b1, b2 = lib(), 3e-3, 1e-8, 0.9, 0.999
    real, seen = tbe.tbe_adamw_step, []

    def moments(state):
        if state.bits == 32:
            return [(m.to(F64), v.to(F64)) for m, v in zip(state.m, state.v)]
        out = []
        for m, v, ms, vs in zip(state.m, state.v, state.ms, state.vs):
            a, b = (q.reshape(-1).float().to(F64) * s.to(F64).repeat_interleave(256)[:q.numel()]
                    for q, s in ((m, ms), (v, vs)))
            out.append((a.view(m.shape), b.square().view(v.shape)))
        return out

    def checked(desc, params, grads, state, step, rate, *more):
        t = int(step)
        before, old = [p.to(F64) for p in params], moments(state)
        real(desc, params, grads, state, step, rate, *more)
        torch.cuda.synchronize()
        for i, (p, q, g, (m, v)) in enumerate(zip(params, before, grads, old)):
            g = g.to(F64)
            dm = 4 * U32 * (b1 * m.abs() + (1 - b1) * g.abs())
            m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
            by = float(rate) / (1 - b1 ** t) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
            off = by * dm + 16 * U32 * by * m.abs() + 3 * U32 * q.abs() + 2.0 ** -126
            assert ((p.to(F64) - (q - by * m)).abs() <= off).all(), (t, i)
        seen.append(t)

    monkeypatch.setattr(example.tbe, "tbe_adamw_step", checked, raising=False)
    losses, model = example.train_gated(steps=4, lr=lr, bits=bits)
    assert seen == [1, 2, 3, 4] and len(losses) == 4
    start = example.GatedModel(2003, 64, 8, 2, 96, seed=2).params
    assert set(start) == set(model.params)
    for name, p in model.params.items():
        assert not torch.equal(p, start[name]), name
