"""Distillation: the statistics as tbe_lm.h states them, and rows far from zero or
masked with the type's lowest value, with error bounds that weigh each element
by what it adds. A logit y = (x - largest) / tau below the row's largest has a power
e^y whose relative error is at most (6 |y| + 3) u, u = 2^-24 (three roundings of
the exponent, again through a rescaled sum, and the power's own): in a sum it
counts e^y times that, so a mask of the lowest value counts nothing."""
import math

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, U32, close, gen, run_distill, say

pytestmark = pytest.mark.gpu
FLUSH = 2.0 ** -126   # powers below it are taken for zero


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Ref:
    """64-bit statistics, loss and gradient of rows with a teacher, and their bounds."""

    def __init__(self, x, ids, t, tau, gl):
        N, V = x.shape
        K = ids.shape[1]
        x, t, gl, ids = x.to(F64), t.to(F64), gl.to(F64), ids.long()
        self.m = x.amax(1)
        y = (x - self.m[:, None]) / tau
        e = torch.exp(y)
        self.s = e.sum(1)
        # relative error of the sum: its terms', and of n additions V / 64 + 256 at most
        add = V / 64 + 256
        near = e * torch.where(y > -800, -y, 0.0)
        self.rs = U32 * (6 * near.sum(1) / self.s + add) + V * FLUSH / self.s
        logq = y - torch.log(self.s)[:, None]
        q = torch.exp(logq)
        z = t / tau
        logp = torch.log_softmax(z, 1)
        p = torch.exp(logp)
        lq = logq.gather(1, ids)
        rp = U32 * (6 * (z.amax(1) - z.amin(1)) + K + 32)[:, None]
        self.loss = tau * tau * (p * (logp - lq)).sum(1)
        el = U32 * 8 * (1 + logp.abs() + lq.abs()) + rp + self.rs[:, None]
        self.bl = tau * tau * (p * ((rp + (K + 4) * U32) * (logp - lq).abs() + el)).sum(1)
        ps = torch.zeros_like(x).scatter_add_(1, ids, p)
        c = (gl * tau)[:, None]
        self.gx = c * (q - ps)
        rq = U32 * (6 * torch.where(y > -800, -y, 0.0) + 7) + self.rs[:, None]
        self.bg = c.abs() * (rq * q + 2 * FLUSH + (rp + (K + 4) * U32) * ps)
        # the bounds are of use: a wrong power, or a sum without it, is far outside
        assert (self.rs < 2e-3).all() and (self.bg <= 2e-3 * c.abs()).all()
        assert (self.bl <= 2e-3 * tau * tau * (1 + self.loss.abs())).all()


def rows(x, V, tau, seed):
    """Logits by kind of row: (name, values [V]), with K distinct places each."""
    g = gen(seed)
    low = torch.finfo(DT[x]).min

    def r():
        return torch.randn(V, generator=g)
    places = torch.randperm(V, generator=g)[:5]
    at = torch.zeros(V, dtype=torch.bool)
    at[places] = True
    half = torch.arange(V) < V // 2
    lower, upper, one = torch.where(half, 2 * r(), low), torch.where(half, low, 2 * r()), torch.full((V,), low)
    for v in (lower, upper, one):
        v[places[0]] = 3.0
    kinds = [("plain", 2 * r()), ("negative", 0.1 * r() - 30), ("far below", 0.1 * r() - 3000),
             ("far above", 0.1 * r() + 3000), ("around 40000", r() * 32 + 40000),
             ("masked from the middle", lower),
             ("masked up to the middle", upper),
             ("masked but for the places", torch.where(at, r(), low)),
             ("masked but for places far below", torch.where(at, -40000 + r(), low)),
             ("lowest", torch.full((V,), low)), ("all but one lowest", one)]
    if x != "f16":
        kinds += [("1e30 at the places", torch.where(at, 1e30, 0.0)), ("-1e30", torch.full((V,), -1e30)),
                  ("near 2^23", -2.0 ** 23 * tau * math.log(2) * (1 + torch.rand(V, generator=g) * 2 ** -8)),
                  ("above 2^23", 2.0 ** 23 * tau * math.log(2) * (1 + torch.rand(V, generator=g) * 2 ** -8)),
                  ("near 2^24", -2.0 ** 24 * tau * math.log(2) * (1 + torch.rand(V, generator=g) * 2 ** -8)),
                  ("below 2^23", 2.0 ** 22 * tau * (1 + torch.rand(V, generator=g) * 2 ** -18))]
    return [k for k, _ in kinds], torch.stack([v for _, v in kinds]).to(DT[x]).cuda(), places.cuda()


def teacher(N, g):
    """Five logits a row. The first place, which no row masks, has a good part of
    p: with all of it at masked places the loss would be at the end of float32's range."""
    t = torch.randn(N, 5, generator=g)
    t[:, 0] = t[:, 0].abs() + 2
    return t.cuda()


@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [37, 1003, 3001, 20011, 70001, 140003])
def test_far_and_masked_rows(x, V, tau):
    say("distill bounds", x, V, tau)
    tbe = lib()
    kinds, xs, places = rows(x, V, tau, V)
    # each kind once, and often enough for the variants of many rows
    for times in (1, 24):
        if times > 1 and V > 3001:
            continue
        xr = xs.repeat(times, 1)
        N = xr.shape[0]
        g = gen(V + times)
        ids = places.expand(N, 5).contiguous()
        ts = teacher(N, g)
        gl = torch.randn(N, generator=g).cuda()
        want = Ref(xr, ids, ts, tau, gl)
        desc = tbe.DistillDesc(N, V, 5, dtype=x, temperature=tau)
        outs = run_distill(tbe, desc, xr, ids, ts, gl)
        for loss, grad in (outs[:2], outs[2:]):
            for i, kind in enumerate(kinds):
                sl = slice(i, None, len(kinds))
                close(loss[sl], want.loss[sl], want.bl[sl], "f32", f"loss, {kind}")
                close(grad[sl], want.gx[sl], want.bg[sl], x, f"gradient, {kind}")


@pytest.mark.parametrize("tau", [1.0, 0.7])
@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [37, 1003, 20011, 140003])
def test_statistics(x, V, tau):
    """Largest logit and sum of exp((x - largest) / tau); the backward takes such
    statistics from anywhere."""
    say("distill statistics", x, V, tau)
    tbe = lib()
    kinds, xs, places = rows(x, V, tau, V + 1)
    N = xs.shape[0]
    ids = places.expand(N, 5).contiguous()
    ts = teacher(N, gen(V))
    gl = torch.randn(N, generator=gen(V + 2)).cuda()
    want = Ref(xs, ids, ts, tau, gl)
    desc = tbe.DistillDesc(N, V, 5, dtype=x, temperature=tau)
    loss, stats = torch.empty(N, device="cuda"), torch.full((N, 2), float("nan"), device="cuda")
    tbe.tbe_distill_forward(desc, xs, ids, ts, loss, stats, tbe.distill_workspace(desc))
    for i, kind in enumerate(kinds):
        assert stats[i, 0].to(F64) == want.m[i], kind
        close(stats[i, 1:], want.s[i:i + 1], (want.rs * want.s)[i:i + 1], "f32", f"sum, {kind}")
    own = torch.stack([want.m, want.s], 1).float()
    gx = torch.full_like(xs, float("nan"))
    tbe.tbe_distill_backward(desc, xs, ids, ts, own, gl, gx)
    for i, kind in enumerate(kinds):
        close(gx[i], want.gx[i], want.bg[i], x, f"gradient, {kind}")


@pytest.mark.parametrize("x", ["f32", "bf16"])
@pytest.mark.parametrize("tau", [5e-39, 2.0 ** -126, 2.0 ** -100, 2.0 ** -20, 2.0 ** 20, 2.0 ** 100, 3e38])
def test_temperatures(tau, x):
    """Logits and gradients in units of a very low or high temperature. (The loss
    is in units of its square, 0 or inf in float32.)"""
    say("distill temperature", tau, x)
    tbe = lib()
    g = gen(7)
    for N, V in ((3, 700), (40, 5003)):
        xs = (tau * 0.2 * torch.randn(N, V, generator=g)).to(DT[x]).cuda()
        ids = torch.stack([torch.randperm(V, generator=g)[:5] for _ in range(N)]).cuda()
        ts = (tau * 0.2 * torch.randn(N, 5, generator=g)).cuda()
        gl = (0.2 / tau * torch.randn(N, generator=g)).cuda()
        tau32 = torch.tensor(tau).to(F64).item()
        want = Ref(xs, ids, ts, tau32, gl)
        desc = tbe.DistillDesc(N, V, 5, dtype=x, temperature=tau)
        outs = run_distill(tbe, desc, xs, ids, ts, gl)
        for loss, grad in (outs[:2], outs[2:]):
            close(loss, want.loss.float(), want.bl, "f32", "loss")
            close(grad, want.gx, want.bg, x, "gradient")
