"""examples/lm_distill.py with gated experts: norm, routing, the experts' products, the
loss, all gradients and the optimizer's step together."""
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


@pytest.mark.parametrize("bits", [32, 8])
def test_training_and_generation_run(example, bits):
    losses, model = example.train_gated(steps=12, bits=bits)
    assert all(l == l for l in losses) and losses[-1] != losses[0]
    assert all(torch.isfinite(p).all() for p in model.params.values())
    tokens = example.generate(model, length=5)
    assert len(tokens) == 6 and all(0 <= t < model.V for t in tokens)


def test_step_gradients_against_differences(example):
    """Each parameter's gradient along a direction against the change of the loss along it.
    The change is a central difference over 2 h = 2^-6 of a unit direction: its own rounding
    is below 2^-17 / h of a loss of order one, and a third derivative of order 50 (the norm's
    and the gate's curvature beside the softmax's) adds h^2 / 6 of that."""
    tbe = lib()
    N, V, D, E, K, F, top = 64, 211, 16, 4, 4, 24, 8    # K = E: no choice changes in between
    teacher, model = example.GatedModel(V, D, E, K, F, seed=5), example.GatedModel(V, D, E, K, F, seed=6)
    model.params["table"] *= D    # rows of order 4, so that a step along them is small
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
    assert set(grads) == set(model.params)
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
            assert abs((up - down) / (2 * h) - want) <= 2.0 ** -17 / h + 50 * h * h / 6, name


def test_a_step_replayed(example):
    """Forward, loss, gradients and the optimizer's step of a fixed batch captured once and
    replayed, against the same steps made eagerly: no call waits for the host."""
    tbe = lib()
    N, V, D, E, K, F, top = 96, 301, 32, 6, 2, 40, 8

    def run(replay):
        model, teacher = example.GatedModel(V, D, E, K, F, seed=2), example.GatedModel(V, D, E, K, F, seed=1)
        b, g = model.buffers(N), torch.Generator(device="cuda")
        g.manual_seed(4)
        ids = torch.randint(0, V, (N,), generator=g, device="cuda")
        t, places = torch.topk(teacher.forward(ids, teacher.buffers(N))[0], top, dim=1)
        t = t.contiguous()
        dd = tbe.DistillDesc(N, V, top, dtype="f32")
        ws = tbe.distill_workspace(dd)
        loss, gl = torch.empty(N, device="cuda"), torch.full((N,), 1.0 / N, device="cuda")
        ad = tbe.AdamWDesc(pdtype="f32", gdtype="f32")
        params = list(model.params.values())
        state = tbe.AdamWState(ad, params)
        step, rate = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.full((1,), 1e-2, device="cuda")

        def once():
            logits, saved = model.forward(ids, b)
            tbe.tbe_distill_step(dd, logits, places, t, gl, loss, logits, ws)
            grads = model.backward(logits, saved, b)
            step.add_(1)
            tbe.tbe_adamw_step(ad, params, [grads[k] for k in model.params], state, step, rate)
        once()
        torch.cuda.synchronize()
        if not replay:
            for _ in range(4):
                once()
                torch.cuda.synchronize()
        else:
            s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
            with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
                once()
            for _ in range(4):
                graph.replay()
                torch.cuda.synchronize()
                torch.ones(1000, device="cuda").mul_(2)   # the program's own work between
        torch.cuda.synchronize()
        return loss.clone(), params

    (a, p), (c, q) = run(False), run(True)
    # torch's own products may take other kernels while captured: losses to their rounding
    assert torch.allclose(a, c, rtol=1e-3, atol=1e-4)
    for x, y in zip(p, q):
        assert torch.isfinite(y).all() and (x - y).abs().max() <= 1e-2
