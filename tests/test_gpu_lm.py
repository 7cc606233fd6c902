"""Language-model operators against plain 64-bit implementations.

Tolerances count roundings: u = 2^-24 per float32 operation, n u times the sum
of magnitudes for a sum of n terms, and half a step of the result's type. Where
a result is a copy or a whole number it must be equal.
"""
import math

import pytest
import torch

from tests.gpu_common import lib

pytestmark = pytest.mark.gpu

F64 = torch.float64
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
# absolute floor: half the smallest subnormal step of the type
TINY = {"f32": 2.0 ** -126, "f16": 2.0 ** -25, "bf16": 2.0 ** -126}


def half(t):
    return torch.finfo(DT[t]).eps / 2


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import bwd_tbe_pooled_amd  # noqa: F401  (fails loudly if the library is missing)


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def randn(g, *shape):
    return torch.randn(*shape, generator=g).cuda()


def close(got, want, bound, t, what):
    """|got - want| <= bound + half a step of t, NaN and infinities equal."""
    got, want = got.to(F64), want.to(F64)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN differ"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    fine = torch.isfinite(want)
    if not torch.is_tensor(bound):
        bound = torch.full_like(want, bound)
    err = (got - want).abs()[fine]
    lim = (bound * (1 + half(t)) + half(t) * want.abs() + TINY[t])[fine]
    worst = (err / lim).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: error is {worst:.3g} of the bound"


def view_of(t, pad):
    """t's values in a matrix whose rows are pad elements longer and whose
    first element is not 16-byte aligned."""
    if not pad:
        return t.contiguous()
    base = torch.full((t.shape[0], t.shape[1] + pad + 1), float("nan"), dtype=t.dtype, device=t.device)
    v = base[:, 1:1 + t.shape[1]]
    v.copy_(t)
    return v


def new(rows, cols, dtype, pad):
    return view_of(torch.full((rows, cols), float("nan"), dtype=dtype, device="cuda"), pad)


def around(v, pad):
    """The elements of a padded matrix outside its columns must stay NaN."""
    if pad:
        base = v._base
        assert torch.isnan(base[:, :1]).all() and torch.isnan(base[:, 1 + v.shape[1]:]).all()


def say(*a):
    print("\n[lm]", *a, flush=True)


# --- token table ---------------------------------------------------------------------
def token_ids(g, N, V, idx, dist, pad):
    if dist == "same":
        ids = torch.full((N,), V // 2, dtype=torch.int64)
    elif dist == "few":
        ids = torch.randint(0, min(V, 3), (N,), generator=g) * max(1, (V - 1) // 2)
    elif dist == "square":   # skewed: long and short runs
        ids = (torch.rand(N, generator=g) ** 4 * V).long().clamp(max=V - 1)
    else:
        ids = torch.randint(0, V, (N,), generator=g)
    if pad:
        bad = torch.tensor([-1, V, -2 ** 31, 2 ** 31 - 1] +
                           ([2 ** 40, -2 ** 62] if idx == torch.int64 else []))
        hit = torch.rand(N, generator=g) < pad
        ids = torch.where(hit, bad[torch.randint(0, len(bad), (N,), generator=g)], ids)
    return ids.to(idx).cuda()


TOKEN = [  # N, V, D, w, x, idx64, distribution, padding, stride padding
    (0, 7, 16, "bf16", "bf16", True, "uniform", 0, 0),
    (1, 1, 1, "f32", "f16", False, "uniform", 0, 0),
    (3, 5, 7, "bf16", "f32", True, "uniform", 0.3, 0),
    (16, 1000, 2048, "bf16", "bf16", True, "uniform", 0, 0),
    (17, 1000, 8, "f16", "f16", False, "uniform", 0.2, 3),
    (100, 33, 9, "f32", "bf16", True, "uniform", 1.0, 0),
    (777, 3203, 1030, "f32", "f16", False, "square", 0.05, 0),
    (1000, 2048, 513, "bf16", "bf16", True, "same", 0, 5),
    (1009, 300, 100, "f16", "f32", False, "few", 0.1, 0),
    (8192, 5000, 64, "bf16", "bf16", True, "square", 0.0, 0),
    (8193, 5000, 72, "bf16", "f16", True, "square", 0.1, 1),
    (20000, 1023, 256, "f32", "bf16", False, "square", 0.0, 0),
    (20000, 1024, 130, "f32", "f32", False, "same", 0.0, 0),
    (40001, 131072, 96, "bf16", "bf16", True, "square", 0.3, 0),
    (300000, 70001, 33, "f16", "bf16", False, "square", 0.1, 0),
    (5000, 1023 * 1024, 24, "f16", "bf16", True, "uniform", 0.0, 0),
    (12000, 1023 * 1024, 24, "bf16", "f16", False, "square", 0.1, 0),
]


@pytest.mark.parametrize("N,V,D,w,x,idx64,dist,pad,stride", TOKEN)
def test_token(N, V, D, w, x, idx64, dist, pad, stride):
    say("token", N, V, D, w, x, dist, pad, stride)
    tbe = lib()
    g = gen(N + V + D)
    idx = torch.int64 if idx64 else torch.int32
    scale = 1.7
    ids = token_ids(g, N, V, idx, dist, pad)
    desc = tbe.TokenDesc(N, V, D, wdtype=w, xdtype=x, idx64=idx64, scale=scale)
    s32 = torch.tensor(scale, dtype=torch.float32).to(F64).item()
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids.long(), 0)

    W = view_of(randn(g, V, D).to(DT[w]), stride)
    out = new(N, D, DT[x], stride)
    tbe.tbe_token_forward(desc, W, ids, out)
    want = torch.where(ok[:, None], W[at].to(F64) * s32, 0.0)
    close(out, want, U32 * want.abs(), x, "forward")
    around(out, stride)

    grad = view_of(randn(g, N, D).to(DT[x]), stride)
    gW = new(V, D, DT[w], stride)
    ws = tbe.token_workspace(desc)
    ws.fill_(0xFF)
    tbe.tbe_token_backward(desc, grad, ids, gW, ws)
    want = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, at[ok], grad[ok].to(F64)) * s32
    size = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, at[ok], grad[ok].to(F64).abs()) * s32
    count = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, at[ok], torch.ones_like(at[ok], dtype=F64))
    close(gW, want, (count[:, None] + 2) * U32 * size, w, "backward")
    around(gW, stride)
    # the same bits again
    again = new(V, D, DT[w], stride)
    tbe.tbe_token_backward(desc, grad, ids, again, ws)
    assert torch.equal(gW, again)


def test_token_gradient_is_the_forwards_adjoint():
    """<g, forward(W)> = <backward(g), W>: the forward is linear in W."""
    tbe = lib()
    g = gen(5)
    N, V, D = 3001, 400, 96
    ids = token_ids(g, N, V, torch.int64, "square", 0.1)
    desc = tbe.TokenDesc(N, V, D, wdtype="f32", xdtype="f32", scale=0.5)
    W, grad = randn(g, V, D), randn(g, N, D)
    out, gW = new(N, D, torch.float32, 0), new(V, D, torch.float32, 0)
    tbe.tbe_token_forward(desc, W, ids, out)
    tbe.tbe_token_backward(desc, grad, ids, gW, tbe.token_workspace(desc))
    a, b = (grad.to(F64) * out.to(F64)), (gW.to(F64) * W.to(F64))
    size = a.abs().sum() + b.abs().sum()
    assert (a.sum() - b.sum()).abs() <= (N + 3) * U32 * size


def test_token_broadcast_gradient():
    """A gradient whose rows are one row (stride 0)."""
    tbe = lib()
    g = gen(6)
    N, V, D = 1500, 20, 40
    ids = token_ids(g, N, V, torch.int32, "uniform", 0.1)
    row = randn(g, 1, D)
    desc = tbe.TokenDesc(N, V, D, wdtype="f32", xdtype="f32", idx64=False)
    ws = tbe.token_workspace(desc)
    got = []
    for grad in (row.expand(N, D), row.repeat(N, 1)):
        gW = new(V, D, torch.float32, 0)
        tbe.tbe_token_backward(desc, grad, ids, gW, ws)
        got.append(gW)
    assert torch.equal(*got)


def test_token_offsets_beyond_32_bits():
    """A table and gradient of 2.4e9 elements."""
    tbe = lib()
    g = gen(7)
    N, V, D = 300, 600000, 4096
    ids = torch.randint(0, V, (N,), generator=g)
    ids[-1], ids[-2] = V - 1, V - 1
    ids = ids.cuda()
    desc = tbe.TokenDesc(N, V, D, wdtype="bf16", xdtype="bf16")
    W = torch.empty(V, D, dtype=torch.bfloat16, device="cuda")
    for a in range(0, V, 100000):
        W[a:a + 100000] = torch.arange(a, min(V, a + 100000), device="cuda")[:, None] % 251
    out = new(N, D, torch.bfloat16, 0)
    tbe.tbe_token_forward(desc, W, ids, out)
    assert torch.equal(out, W[ids])
    grad = randn(g, N, D).bfloat16()
    W.fill_(float("nan"))
    tbe.tbe_token_backward(desc, grad, ids, W, tbe.token_workspace(desc))
    rows = torch.unique(ids)
    want = torch.zeros(V, D // 64, dtype=F64, device="cuda")
    for d0 in range(0, D, D // 64):
        sl = slice(d0, d0 + D // 64)
        want.zero_().index_add_(0, ids, grad[:, sl].to(F64))
        close(W[rows][:, sl], want[rows], 4 * U32 * 8, "bf16", "backward")
    touched = torch.zeros(V, dtype=torch.bool, device="cuda")
    touched[rows] = True
    for a in range(0, V, 100000):
        part = W[a:a + 100000][~touched[a:a + 100000]]
        assert not part.view(torch.int16).any()


# --- experts ---------------------------------------------------------------------------
def plan_of(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where((flat < 0) | (flat >= E), E, flat)
    order = torch.sort(key, stable=True).indices
    place = torch.empty_like(order)
    place[order] = torch.arange(flat.numel(), device=flat.device)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=flat.device))
    return offsets, order, torch.where(key == E, -1 - place, place)


EXPERT = [  # N, K, E, D, dtype, idx64, dropped, stride padding
    (0, 2, 4, 16, "bf16", True, 0, 0),
    (1, 1, 1, 1, "f32", False, 0, 0),
    (1, 3, 2, 5, "f16", True, 0.4, 0),
    (4, 8, 64, 2048, "bf16", True, 0, 0),
    (33, 2, 8, 1001, "f32", True, 0.1, 0),
    (50, 64, 1023, 70, "bf16", False, 0.2, 3),
    (100, 4, 6, 8, "f16", False, 1.0, 0),
    (1024, 8, 16, 72, "bf16", True, 0.05, 0),
    (1025, 8, 16, 65, "bf16", True, 0.05, 1),
    (3000, 5, 512, 520, "f16", True, 0.0, 0),
    (40000, 8, 100, 40, "bf16", False, 0.1, 0),
    (70, 3, 5, 4100, "bf16", True, 0.1, 0),
    (40, 7, 5, 9001, "f32", True, 0.1, 2),
]


@pytest.mark.parametrize("N,K,E,D,t,idx64,drop,stride", EXPERT)
def test_expert(N, K, E, D, t, idx64, drop, stride):
    say("expert", N, K, E, D, t, drop, stride)
    tbe = lib()
    g = gen(N * K + E + D)
    idx = torch.int64 if idx64 else torch.int32
    M = N * K
    ids = (torch.rand(N, K, generator=g) ** 2 * E).long().clamp(max=E - 1)
    bad = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1])
    ids = torch.where(torch.rand(N, K, generator=g) < drop,
                      bad[torch.randint(0, 4, (N, K), generator=g)], ids).to(idx).cuda()
    desc = tbe.ExpertDesc(N, K, E, D, dtype=t, idx64=idx64)
    plan = tbe.ExpertPlan(desc)
    ws = tbe.expert_workspace(desc)
    ws.fill_(0xFF)
    tbe.tbe_expert_plan(desc, ids, plan, ws)
    offsets, order, slots = plan_of(ids, E)
    assert torch.equal(plan.offsets.long(), offsets)
    assert torch.equal(plan.order.long(), order)
    assert torch.equal(plan.slots.long(), slots)

    ok = (slots >= 0).view(N, K)
    place = torch.where(slots >= 0, slots, -1 - slots)
    x = view_of(randn(g, N, D).to(DT[t]), stride)
    xs = new(M, D, DT[t], stride)
    tbe.tbe_expert_dispatch(desc, x, plan.slots, xs)
    want = torch.zeros(M, D, dtype=DT[t], device="cuda")
    want[place] = torch.where(ok.view(-1, 1), x.repeat_interleave(K, 0), 0)
    assert torch.equal(xs, want)
    around(xs, stride)

    w = torch.rand(N, K, generator=g).cuda()
    w[~ok] = float("nan")               # a dropped assignment's weight is not used
    ys = randn(g, M, D).to(DT[t])
    ys[place[~ok.view(-1)]] = float("nan")   # nor its row
    ys = view_of(ys, stride)
    out = new(N, D, DT[t], stride)
    tbe.tbe_expert_combine(desc, ys, plan.slots, w, out)
    w64 = torch.where(ok, w.to(F64), 0.0)
    y64 = torch.where(ok[:, :, None], ys[place].to(F64).view(N, K, D), 0.0)
    terms = w64[:, :, None] * y64
    close(out, terms.sum(1), (K + 1) * U32 * terms.abs().sum(1), t, "combine")
    around(out, stride)

    dx = new(N, D, DT[t], stride)
    tbe.tbe_expert_dispatch_backward(desc, ys, plan.slots, dx)
    close(dx, y64.sum(1), (K + 1) * U32 * y64.abs().sum(1), t, "dispatch backward")
    around(dx, stride)

    dout = view_of(randn(g, N, D).to(DT[t]), stride)
    dys = new(M, D, DT[t], stride)
    dw = torch.full((N, K), float("nan"), device="cuda")
    tbe.tbe_expert_combine_backward(desc, dout, ys, plan.slots, w, dys, dw)
    d64 = dout.to(F64)
    want = torch.zeros(M, D, dtype=F64, device="cuda")
    want[place] = (w64[:, :, None] * d64[:, None, :]).view(M, D)
    close(dys, want, 2 * U32 * want.abs(), t, "dys")
    around(dys, stride)
    prod = d64[:, None, :] * y64
    close(dw, prod.sum(2), (D + 2) * U32 * prod.abs().sum(2), "f32", "dw")
    # in place
    dw2 = torch.full((N, K), float("nan"), device="cuda")
    tbe.tbe_expert_combine_backward(desc, dout, ys, plan.slots, w, ys, dw2)
    assert torch.equal(ys, dys) and torch.equal(dw, dw2)


def test_expert_slots_out_of_range_are_skipped():
    tbe = lib()
    g = gen(11)
    N, K, D = 6, 2, 24
    M = N * K
    desc = tbe.ExpertDesc(N, K, 4, D, dtype="f32")
    slots = torch.arange(M, dtype=torch.int32)
    slots[3], slots[5], slots[8] = M, 2 ** 31 - 1, -2 ** 31
    bad = torch.zeros(M, dtype=torch.bool)
    bad[[3, 5, 8]] = True
    bad = bad.cuda()
    slots = slots.cuda()
    x, ys = randn(g, N, D), randn(g, M, D)
    xs = new(M, D, torch.float32, 0)
    tbe.tbe_expert_dispatch(desc, x, slots, xs)
    assert torch.isnan(xs[bad]).all()
    assert torch.equal(xs[~bad], x.repeat_interleave(K, 0)[~bad])
    w = torch.ones(N, K, device="cuda")
    out, dys, dw = new(N, D, torch.float32, 0), new(M, D, torch.float32, 0), new(N, K, torch.float32, 0)
    tbe.tbe_expert_combine(desc, ys, slots, w, out)
    kept = torch.where(bad[:, None], 0, ys)
    assert torch.equal(out, kept.view(N, K, D).sum(1))
    tbe.tbe_expert_combine_backward(desc, x, ys, slots, w, dys, dw)
    assert torch.isnan(dys[bad]).all() and (dw.view(-1)[bad] == 0).all()
    assert torch.equal(dys[~bad], x.repeat_interleave(K, 0)[~bad])


def test_expert_gradients_are_adjoints():
    """combine is linear in ys and in w, dispatch in x: inner products agree."""
    tbe = lib()
    g = gen(12)
    N, K, E, D = 200, 3, 7, 130
    desc = tbe.ExpertDesc(N, K, E, D, dtype="f32")
    ids = torch.randint(-1, E, (N, K), generator=g).cuda()
    plan = tbe.ExpertPlan(desc)
    tbe.tbe_expert_plan(desc, ids, plan, tbe.expert_workspace(desc))
    f = torch.float32
    x, ys, dout, w = randn(g, N, D), randn(g, N * K, D), randn(g, N, D), randn(g, N, K)
    xs, out, dys, dx, dw = (new(N * K, D, f, 0), new(N, D, f, 0), new(N * K, D, f, 0),
                            new(N, D, f, 0), new(N, K, f, 0))
    tbe.tbe_expert_dispatch(desc, x, plan.slots, xs)
    tbe.tbe_expert_dispatch_backward(desc, ys, plan.slots, dx)
    tbe.tbe_expert_combine(desc, ys, plan.slots, w, out)
    tbe.tbe_expert_combine_backward(desc, dout, ys, plan.slots, w, dys, dw)

    def agree(a, b, c, d):
        p, q = a.to(F64) * b.to(F64), c.to(F64) * d.to(F64)
        assert (p.sum() - q.sum()).abs() <= (D + 3) * U32 * (p.abs().sum() + q.abs().sum())
    agree(xs, ys, x, dx)
    agree(out, dout, ys, dys)
    agree(out, dout, w, dw)


# --- distillation ------------------------------------------------------------------------
def distill_ref(x, ids, t, tau, gl):
    """Loss, gradient and their bounds in 64 bits."""
    N, V = x.shape
    K = ids.shape[1]
    x, t, gl = x.to(F64), t.to(F64), gl.to(F64)
    ids = ids.long()
    ok = (ids >= 0) & (ids < V) & (t != -math.inf)
    some = ok.any(1, keepdim=True)
    at = torch.where(ok, ids, 0)
    z = torch.where(ok, t / tau, -math.inf)
    zmax = torch.where(some, z.amax(1, keepdim=True), 0.0)
    logp = z - zmax
    logp = logp - torch.log(torch.exp(logp).sum(1, keepdim=True))
    p = torch.where(ok, torch.exp(logp), 0.0)
    m = x.amax(1, keepdim=True)
    y = (x - m) / tau
    s = torch.exp(y).sum(1, keepdim=True)
    logq = y - torch.log(s)
    q = torch.exp(logq)
    lq = logq.gather(1, at)
    terms = torch.where(ok & (p != 0), p * (logp - lq), 0.0)
    loss = tau * tau * terms.sum(1)
    ps = torch.zeros_like(x).scatter_add_(1, at, p)
    gx = (gl * tau)[:, None] * (torch.where(some, q, 0.0) - ps)
    gx = torch.where(some, gx, 0.0)
    # relative error of q and p: three roundings of the scaled difference
    # (twice: in the exponent and through the rescaled sum), the sum's n
    # terms per lane and the steps of its running maximum, exp and division
    span = torch.where(torch.isfinite(y), -y, 0.0).amax(1, keepdim=True)
    rq = U32 * (6 * span + V / 64 + 256)
    tspan = torch.where(ok & torch.isfinite(z), zmax - z, 0.0).amax(1, keepdim=True)
    rp = U32 * (6 * tspan + K + 32)
    el = U32 * 8 * (1 + torch.where(ok, logp.abs() + lq.abs(), 0.0)) + rp + rq
    fine = torch.where(torch.isfinite(terms), terms, 0.0)
    bl = tau * tau * ((rp + (K + 4) * U32) * fine.abs() + torch.where(ok, p * el, 0.0)).sum(1)
    bg = (gl * tau).abs()[:, None] * ((rq + 4 * U32) * q + (rp + (K + 4) * U32) * ps)
    return loss, gx, torch.nan_to_num(bl), torch.nan_to_num(bg)


def distill_case(g, N, V, K, x, t, idx64, prompt, distinct=True):
    xs = (2 * torch.randn(N, V, generator=g)).to(DT[x])
    if distinct and K <= V:
        ids = torch.stack([torch.randperm(V, generator=g)[:K] for _ in range(N)]) if N else torch.zeros(0, K).long()
    else:
        ids = torch.randint(0, V, (N, K), generator=g)
    ts = (3 * torch.randn(N, K, generator=g)).to(DT[t])
    length = torch.randint(0, K + 1, (N,), generator=g)
    length = torch.where(torch.rand(N, generator=g) < 0.5, length, K)
    length = torch.where(torch.rand(N, generator=g) < prompt, 0, length)
    bad = torch.tensor([-1, V, 2 ** 31 - 1, -2 ** 31])
    ids = torch.where(torch.arange(K) < length[:, None], ids,
                      bad[torch.randint(0, 4, (N, K), generator=g)])
    gl = torch.randn(N, generator=g)
    return (xs.cuda(), ids.to(torch.int64 if idx64 else torch.int32).cuda(), ts.cuda(), gl.cuda())


def run_distill(tbe, desc, x, ids, t, gl, stride=0):
    N, V = x.shape
    loss = torch.full((N,), float("nan"), device="cuda")
    stats = torch.full((N, 2), float("nan"), device="cuda")
    gx = new(N, V, x.dtype, stride)
    ws = tbe.distill_workspace(desc)
    ws.fill_(0xFF)
    tbe.tbe_distill_forward(desc, x, ids, t, loss, stats, ws)
    tbe.tbe_distill_backward(desc, x, ids, t, stats, gl, gx)
    around(gx, stride)
    ws.fill_(0xFF)
    loss2 = torch.full((N,), float("nan"), device="cuda")
    gx2 = new(N, V, x.dtype, stride)
    tbe.tbe_distill_step(desc, x, ids, t, gl, loss2, gx2, ws)
    around(gx2, stride)
    return loss, gx, loss2, gx2


DISTILL = [  # N, V, K, x, t, idx64, tau, prompt, distinct, stride padding
    (0, 10, 2, "bf16", "f32", True, 1.0, 0, True, 0),
    (1, 1, 1, "f32", "f32", True, 1.0, 0, True, 0),
    (5, 3, 4, "bf16", "f16", False, 2.0, 0.2, False, 0),
    (7, 8, 3, "f16", "f32", True, 0.7, 0, True, 0),
    (9, 17, 16, "f32", "bf16", True, 1.0, 0.3, True, 3),
    (3, 50021, 20, "f32", "f32", True, 1.0, 0, True, 0),
    (40, 5003, 128, "f16", "f16", False, 2.0, 0.1, True, 0),
    (40, 5003, 200, "bf16", "bf16", True, 1.0, 0.1, False, 1),
    (12, 32000, 1024, "bf16", "f32", True, 0.5, 0.5, True, 0),
    (6, 131072, 64, "bf16", "f32", True, 1.0, 0.1, True, 0),
    (5, 131077, 64, "f16", "f32", True, 1.0, 0.0, True, 0),
    (4, 66000, 256, "f32", "f32", False, 1.0, 0.0, True, 1),
    (5, 65536, 31, "f32", "f16", False, 1.3, 0.0, True, 0),
    (3, 200000, 31, "bf16", "f16", False, 1.0, 0.0, True, 0),
    (2, 200003, 31, "f32", "f16", False, 1.0, 0.0, True, 0),
    (1500, 1000, 9, "bf16", "f32", True, 1.0, 0.2, True, 0),
    (700, 2049, 65, "f32", "f32", True, 1.0, 0.2, True, 0),
]


@pytest.mark.parametrize("N,V,K,x,t,idx64,tau,prompt,distinct,stride", DISTILL)
def test_distill(N, V, K, x, t, idx64, tau, prompt, distinct, stride):
    say("distill", N, V, K, x, t, tau, prompt, distinct, stride)
    tbe = lib()
    desc = tbe.DistillDesc(N, V, K, dtype=x, tdtype=t, idx64=idx64, temperature=tau)
    xs, ids, ts, gl = distill_case(gen(N + V + K), N, V, K, x, t, idx64, prompt, distinct)
    xs = view_of(xs, stride)
    want_l, want_g, bl, bg = distill_ref(xs, ids, ts, tau, gl)
    loss, gx, loss2, gx2 = run_distill(tbe, desc, xs, ids, ts, gl, stride)
    close(loss, want_l, bl, "f32", "loss")
    close(gx, want_g, bg, x, "gradient")
    close(loss2, want_l, bl, "f32", "step: loss")
    close(gx2, want_g, bg, x, "step: gradient")
    # in place, and the same bits again
    both = xs.clone(memory_format=torch.preserve_format) if not stride else view_of(xs, stride)
    ws = tbe.distill_workspace(desc)
    tbe.tbe_distill_step(desc, both, ids, ts, gl, loss, both, ws)
    assert torch.equal(loss, loss2) and torch.equal(both, gx2)
    stats = torch.empty(N, 2, device="cuda")
    tbe.tbe_distill_forward(desc, xs, ids, ts, loss, stats, ws)
    tbe.tbe_distill_backward(desc, xs, ids, ts, stats, gl, xs)
    assert torch.equal(xs, gx)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [600, 20011])
def test_distill_masked_logits(x, V):
    """Rows of -inf and of the type's lowest value, NaN and infinities in rows
    without a teacher, teacher entries of -inf."""
    say("distill masks", x, V)
    tbe = lib()
    N, K, tau = 10, 6, 0.7
    xs, ids, ts, gl = distill_case(gen(V), N, V, K, x, "f32", True, 0.0)
    low = torch.finfo(DT[x]).min
    ids = torch.stack([torch.randperm(V, generator=gen(n))[:K] for n in range(N)]).cuda()
    keep = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, ids, True)
    xs[0] = torch.where(keep[0], xs[0], -math.inf)      # only the teacher's places
    xs[1] = torch.where(keep[1], xs[1], low)
    xs[2] = low                                          # uniform
    xs[3, :V // 2] = -math.inf
    xs[3, ids[3]] = 1.0
    ts[4] = -math.inf                                    # no entry left: not read
    xs[4] = float("nan")
    ids[5] = -1
    xs[5] = math.inf
    ts[6, 1:] = -math.inf                                # one entry left
    xs[7, 5] = float("nan")                              # NaN rows
    xs[8] = -math.inf
    xs[9, ids[9, 0]] = -math.inf                         # q = 0 where p > 0: loss +inf
    desc = tbe.DistillDesc(N, V, K, dtype=x, temperature=tau)
    want_l, want_g, bl, bg = distill_ref(xs, ids, ts, tau, gl)
    nan_rows = torch.zeros(N, dtype=torch.bool, device="cuda")
    nan_rows[7:9] = True
    none = torch.zeros(N, dtype=torch.bool, device="cuda")
    none[4:6] = True
    want_l, want_g = torch.where(none, 0.0, want_l), torch.where(none[:, None], 0.0, want_g)
    # lowest values less a finite maximum: a difference the type holds, or one
    # that overflows; both are exp(-inf) = 0
    for loss, grad in zip(*[iter(run_distill(tbe, desc, xs, ids, ts, gl))] * 2):
        assert torch.isnan(loss[nan_rows]).all() and torch.isnan(grad[nan_rows]).all()
        assert loss[9] == math.inf and want_l[9] == math.inf
        assert (loss[none] == 0).all() and (grad[none] == 0).all()
        fine = ~nan_rows
        close(loss[fine], want_l[fine], bl[fine], "f32", "loss")
        close(grad[fine], want_g[fine], bg[fine], x, "gradient")


def test_distill_gradient_against_differences():
    """Central differences of the 32-bit loss. Its third derivative in one
    logit is tau^2 / tau^3 times a third cumulant of a 0/1 variable (below 0.1)."""
    tbe = lib()
    g = gen(21)
    V, K, tau, h = 300, 8, 1.5, 2.0 ** -5
    x, ids, t, _ = distill_case(g, 1, V, K, "f32", "f32", True, 0.0)
    ids = torch.randperm(V, generator=g)[:K].cuda()[None]
    places = torch.cat([ids[0, :4], x[0].topk(4).indices, torch.tensor([0, V - 1]).cuda()])
    n = len(places)
    rows = x.repeat(2 * n + 1, 1)
    rows[torch.arange(n), places] += h
    rows[torch.arange(n) + n, places] -= h
    R = 2 * n + 1
    desc = tbe.DistillDesc(R, V, K, dtype="f32", temperature=tau)
    gl = torch.ones(R, device="cuda")
    ids, t = ids.repeat(R, 1), t.repeat(R, 1)
    loss, gx, _, _ = run_distill(tbe, desc, rows, ids, t, gl)
    _, _, bl, _ = distill_ref(rows, ids, t, tau, gl)
    step = (rows[:n].to(F64) - rows[n:2 * n].to(F64)).gather(1, places[:, None])[:, 0]
    diff = (loss[:n].to(F64) - loss[n:2 * n].to(F64)) / step
    lim = 0.1 / tau * h * h / 6 + 2 * bl.max() / step.abs() + 1e-6
    assert ((diff - gx[-1, places].to(F64)).abs() <= lim).all()


def test_distill_offsets_beyond_32_bits():
    """2.6e9 logits; the last rows are compared."""
    tbe = lib()
    N, V, K = 20000, 131072, 8
    g = gen(23)
    x = torch.empty(N, V, dtype=torch.bfloat16, device="cuda")
    x.view(torch.int16).zero_()
    x[-3:] = (2 * torch.randn(3, V, generator=g)).cuda().bfloat16()
    ids = torch.full((N, K), -1, dtype=torch.int64, device="cuda")
    ids[-3:] = torch.randint(0, V, (3, K), generator=g).cuda()
    t = torch.randn(N, K, generator=g).cuda()
    gl = torch.ones(N, device="cuda")
    desc = tbe.DistillDesc(N, V, K)
    want_l, want_g, bl, bg = distill_ref(x[-3:], ids[-3:], t[-3:], 1.0, gl[-3:])
    loss, gx, loss2, gx2 = run_distill(tbe, desc, x, ids, t, gl)
    for a, b in ((loss, gx), (loss2, gx2)):
        close(a[-3:], want_l, bl, "f32", "loss")
        close(b[-3:], want_g, bg, "bf16", "gradient")
        assert not a[:-3].any() and not b[:-3].view(torch.int16).any()


# --- streams, graphs, refusals -----------------------------------------------------------
def sequence(tbe, seed):
    """One pass through every call, as a closure over its buffers, and the
    tensors it writes."""
    g = gen(seed)
    N, V, D, K, E, T = 500, 3001, 200, 4, 12, 20
    bf = torch.bfloat16
    td = tbe.TokenDesc(N, V, D, scale=2.0)
    ed = tbe.ExpertDesc(N, K, E, D)
    dd = tbe.DistillDesc(N, V, T)
    W = randn(g, V, D).to(bf)
    ids = token_ids(g, N, V, torch.int64, "square", 0.1)
    eids = torch.randint(-1, E, (N, K), generator=g).cuda()
    w = torch.rand(N, K, generator=g).cuda()
    x, tid, t, gl = distill_case(g, N, V, T, "bf16", "f32", True, 0.2)
    out, gW = new(N, D, bf, 0), new(V, D, bf, 0)
    plan = tbe.ExpertPlan(ed)
    xs, y, dys, dx = new(N * K, D, bf, 0), new(N, D, bf, 0), new(N * K, D, bf, 0), new(N, D, bf, 0)
    dw, loss, stats = new(N, K, torch.float32, 0), torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
    gx, gx2 = new(N, V, bf, 0), new(N, V, bf, 0)
    loss2 = torch.empty(N, device="cuda")
    wt, we, wd = tbe.token_workspace(td), tbe.expert_workspace(ed), tbe.distill_workspace(dd)

    def run(stream=None):
        tbe.tbe_token_forward(td, W, ids, out, stream)
        tbe.tbe_expert_plan(ed, eids, plan, we, stream)
        tbe.tbe_expert_dispatch(ed, out, plan.slots, xs, stream)
        tbe.tbe_expert_combine(ed, xs, plan.slots, w, y, stream)
        tbe.tbe_distill_forward(dd, x, tid, t, loss, stats, wd, stream)
        tbe.tbe_distill_backward(dd, x, tid, t, stats, gl, gx, stream)
        tbe.tbe_distill_step(dd, x, tid, t, gl, loss2, gx2, wd, stream)
        tbe.tbe_expert_combine_backward(ed, y, xs, plan.slots, w, dys, dw, stream)
        tbe.tbe_expert_dispatch_backward(ed, dys, plan.slots, dx, stream)
        tbe.tbe_token_backward(td, dx, ids, gW, wt, stream)
    outs = [out, plan.offsets, plan.order, plan.slots, xs, y, loss, stats, gx, loss2, gx2, dys, dw,
            dx, gW]
    return run, outs


def test_calls_replayed_from_a_graph_match_eager():
    tbe = lib()
    run, outs = sequence(tbe, 31)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    for replay in range(4):
        for o in outs:
            o.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {replay}: output {i} differs"
        run()   # eager work between the replays
        torch.cuda.synchronize()


def test_calls_on_another_stream():
    tbe = lib()
    run, outs = sequence(tbe, 32)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for o in outs:
        o.fill_(3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    side.synchronize()
    for i, (a, b) in enumerate(zip(outs, want)):
        assert torch.equal(a, b), f"output {i} differs"


def test_binding_refuses_wrong_tensors():
    tbe = lib()
    d = tbe.TokenDesc(4, 10, 8)
    W = torch.zeros(10, 8, dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    out = torch.zeros(4, 8, dtype=torch.bfloat16, device="cuda")
    ws = tbe.token_workspace(d)
    tbe.tbe_token_forward(d, W, ids, out)
    for args in [(W.float(), ids, out), (W[:9], ids, out), (W, ids.int(), out), (W, ids[:3], out),
                 (W, ids, out.half()), (W, ids, out.t().contiguous().t()), (W, ids, out[0].expand(4, 8)),
                 (W, ids.cpu(), out), (W, None, out), (W, ids[::1].repeat(2)[::2], out)]:
        with pytest.raises(TypeError):
            tbe.tbe_token_forward(d, *args)
    with pytest.raises(TypeError):
        tbe.tbe_token_backward(d, out, ids, W, None)
    with pytest.raises(tbe.TbeError) as e:
        tbe.tbe_token_backward(d, out, ids, W, ws[:16])
    assert e.value.status == tbe.TBE_ERR_WORKSPACE
    e_ = tbe.ExpertDesc(4, 2, 3, 8)
    with pytest.raises(TypeError):
        tbe.tbe_expert_dispatch(e_, out, torch.zeros(8, dtype=torch.int64, device="cuda"),
                                torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        tbe.tbe_expert_combine(e_, torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda"),
                               torch.zeros(8, dtype=torch.int32, device="cuda"),
                               torch.zeros(4, 2, dtype=torch.bfloat16, device="cuda"), out)
