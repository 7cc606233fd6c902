"""examples/lm_distill.py: the operators together, and their gradients through a
whole step against differences of its loss."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_common import lib

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


def test_training_lowers_the_loss(example):
    losses, model = example.train(steps=40)
    assert all(l == l for l in losses)
    assert sum(losses[-5:]) < 0.8 * sum(losses[:5])
    tokens = example.generate(model, length=5)
    assert len(tokens) == 6 and all(0 <= t < model.V for t in tokens)


def test_step_gradients_against_differences(example):
    """Each parameter's gradient along a direction against the change of the
    loss along it. The change is a central difference over 2 h = 2^-6 of a unit
    direction: its own rounding is below 2^-18 / h of a loss of order one, and a
    third derivative of order ten adds h^2 / 6 of that."""
    tbe = lib()
    N, V, D, E, K, top = 64, 211, 16, 4, 4, 8    # K = E: no choice changes in between
    teacher, model = example.Model(V, D, E, K, seed=5), example.Model(V, D, E, K, seed=6)
    model.scale = 1.0
    b = model.buffers(N)
    ids = torch.arange(N, device="cuda") % 37
    t, places = torch.topk(teacher.forward(ids, teacher.buffers(N))[0], top, dim=1)
    dd = tbe.DistillDesc(N, V, top, dtype="f32")
    ws = tbe.distill_workspace(dd)
    gl = torch.full((N,), 1.0 / N, device="cuda")
    loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")

    def value():
        logits, _ = model.forward(ids, b)
        tbe.tbe_distill_forward(dd, logits, places, t.contiguous(), loss, stats, ws)
        return loss.double().mean().item()

    logits, state = model.forward(ids, b)
    tbe.tbe_distill_step(dd, logits, places, t.contiguous(), gl, loss, logits, ws)
    grads = model.backward(logits, state, b)
    h = 2.0 ** -7
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    for name, p in model.params.items():
        grad = grads[name]
        for direction in (grad, torch.randn(p.shape, generator=g, device="cuda")):
            d = direction / direction.norm()
            before = p.clone()
            p += h * d
            up = value()
            p.copy_(before - h * d)
            down = value()
            p.copy_(before)
            want = (grad.double() * d.double()).sum().item()
            assert abs((up - down) / (2 * h) - want) <= 2.0 ** -18 / h + 10 * h * h / 6, name
