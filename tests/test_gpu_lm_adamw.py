"""AdamW over many tensors against 64-bit formulas.

Tolerances count roundings, u = 2^-24 each: a moment is one multiply and one
fused multiply-add of two terms, the move about a dozen operations, none of
which cancels; 8-bit moments are off by half a step of e4m3 (2^-4 of the value,
2^-10 of the block's scale for the smallest) and a scale of a few roundings.
"""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, TINY, U32, close, gen, half, say

pytestmark = pytest.mark.gpu
BLOCK = 256


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


def decoded(codes, scales):
    """The values of an 8-bit moment in 64 bits."""
    n = codes.numel()
    return codes.reshape(-1).to(torch.float32).to(F64) * scales.to(F64).repeat_interleave(BLOCK)[:n]


def tensors(g, shapes, dtype, std, gap=0):
    """Tensors of a flat buffer with `gap` elements between them."""
    sizes = [torch.Size(s).numel() for s in shapes]
    flat = torch.full((sum(sizes) + gap * (len(sizes) + 1),), float("nan"), dtype=dtype, device="cuda")
    out, at = [], gap
    for s, n in zip(shapes, sizes):
        flat[at:at + n] = (torch.randn(n, generator=g) * std).to(dtype).cuda()
        out.append(flat[at:at + n].view(s))
        at += n + gap
    return flat, out


def moments(state):
    """(m, v) of each tensor in 64 bits, v as the second moment."""
    if state.bits == 32:
        return [(m.to(F64).reshape(-1), v.to(F64).reshape(-1)) for m, v in zip(state.m, state.v)]
    return [(decoded(m, ms), decoded(v, vs).square())
            for m, v, ms, vs in zip(state.m, state.v, state.ms, state.vs)]


def check_step(desc, kw, params, grads, state, step, lr, scale, copies):
    """One step from the state as it is, against the formula."""
    tbe = lib()
    p0 = [p.to(F64).reshape(-1).clone() for p in params]
    old = moments(state)
    args = (torch.tensor([step], device="cuda"), torch.tensor([lr], device="cuda"),
            None if scale is None else torch.tensor([scale], device="cuda"))
    tbe.tbe_adamw_step(desc, params, grads, state, *args, copies)
    torch.cuda.synchronize()
    b1, b2, eps, wd = kw["beta1"], kw["beta2"], kw["eps"], kw["weight_decay"]
    lr, scale = float(torch.tensor(lr)), 1.0 if scale is None else float(torch.tensor(scale))
    t = max(step, 1)
    for i, (p, g) in enumerate(zip(params, grads)):
        if p.numel() == 0:
            continue
        pt = {v: k for k, v in DT.items()}[p.dtype]
        g = g.to(F64).reshape(-1) * scale
        m = b1 * old[i][0] + (1 - b1) * g
        v = b2 * old[i][1] + (1 - b2) * g * g
        dm = 6 * U32 * (b1 * old[i][0].abs() + (1 - b1) * g.abs()) + TINY["f32"]
        dv = 8 * U32 * v + TINY["f32"]
        root = torch.sqrt(v / (1 - b2 ** t)) + eps
        move = lr / (1 - b1 ** t) * m / root
        x = p0[i] * (1 - lr * wd) - move
        # the move: m's own error and 16 roundings; a second moment too small for float32 is zero
        off = lr / (1 - b1 ** t) * dm / root + 16 * U32 * move.abs() + 3 * U32 * p0[i].abs()
        off = off + move.abs() * torch.sqrt(TINY["f32"] / (1 - b2 ** t) / torch.ones_like(v)) / root
        close(p.reshape(-1), x, off, pt, f"p[{i}]")
        if copies is not None:
            ct = {v: k for k, v in DT.items()}[copies[i].dtype]
            close(copies[i].reshape(-1), x, off + half("f32") * x.abs(), ct, f"copy[{i}]")
        if state.bits == 32:
            close(state.m[i].reshape(-1), m, dm, "f32", f"m[{i}]")
            close(state.v[i].reshape(-1), v, dv, "f32", f"v[{i}]")
            continue
        n = p.numel()
        for codes, scales, want, name in ((state.m[i], state.ms[i], m, "m"),
                                          (state.v[i], state.vs[i], torch.sqrt(v), "v")):
            pad = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=F64, device="cuda")
            pad[:n] = want.abs()
            top = pad.view(-1, BLOCK).amax(1)
            held = top >= 2.0 ** -100
            close(scales, torch.where(held, top / 448, 0.0), 16 * U32 * top / 448, "f32", f"{name} scale[{i}]")
            s = scales.to(F64).repeat_interleave(BLOCK)[:n]
            off = torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -16) + 32 * U32 * want.abs()
            if name == "v":   # what is above zero is held as at least 2^-9 of the scale
                off = torch.where((want > 0) & (want < s * 2.0 ** -9), s * 2.0 ** -9, off)
                assert ((codes.reshape(-1).float() > 0) | (want == 0) | (s == 0)).all()
            off = torch.where(s > 0, off, 2.0 ** -100)
            err = (decoded(codes, scales) - want).abs()
            assert (err <= off).all(), f"{name}[{i}]: {(err / off.clamp_min(1e-300)).max().item():.3g} of the bound"


SHAPES = [(1,), (7,), (255,), (256,), (257, 3), (0,), (4096,), (4097,), (33, 129), (2, 3, 5, 7), (20000,), (5, 4099)]
KINDS = [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", "f16"), ("f32", "bf16", "f16"),
         ("f32", "f16", None), ("bf16", "bf16", None), ("f16", "f16", None), ("bf16", "f32", None), ("f16", "bf16", None)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("p,g,c", KINDS)
def test_steps(p, g, c, bits):
    """Several steps from zero moments; odd sizes, packed at odd starts."""
    say("adamw", p, g, c, bits)
    tbe = lib()
    r = gen(len(p) + bits)
    kw = dict(beta1=0.9, beta2=0.98, eps=1e-8, weight_decay=0.1)
    desc = tbe.AdamWDesc(pdtype=p, gdtype=g, cdtype=c, bits=bits, **kw)
    flat, params = tensors(r, SHAPES, DT[p], 0.5, gap=1)
    edges = torch.isnan(flat)
    state = tbe.AdamWState(desc, params)
    copies = tensors(r, SHAPES, DT[c], 0.0, gap=3)[1] if c else None
    for step in (1, 2, 3, 1000):
        scale = None if step == 2 else 0.25
        grads = tensors(r, SHAPES, DT[g], 0.01, gap=2)[1]
        check_step(desc, kw, params, grads, state, step, 1e-2, scale, copies)
    assert torch.equal(torch.isnan(flat), edges)


def test_more_tensors_than_a_launch_takes():
    tbe = lib()
    r = gen(5)
    kw = dict(beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0)
    desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", **kw)
    shapes = [(1 + 37 * i % 600,) for i in range(211)]
    params, grads = tensors(r, shapes, torch.float32, 1.0)[1], tensors(r, shapes, torch.float32, 1.0)[1]
    order = torch.randperm(211, generator=r).tolist()    # addresses in no order
    params, grads = [params[i] for i in order], [grads[i] for i in order]
    check_step(desc, kw, params, grads, tbe.AdamWState(desc, params), 1, 1e-3, None, None)


@pytest.mark.parametrize("bits", [32, 8])
def test_steps_far_along_and_below_one(bits):
    tbe = lib()
    r = gen(6)
    kw = dict(beta1=0.9, beta2=0.9999, eps=1e-6, weight_decay=0.01)
    desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", bits=bits, **kw)
    params = tensors(r, [(700,)], torch.float32, 1.0)[1]
    state = tbe.AdamWState(desc, params)
    for step in (0, -5, 10 ** 6, 2 ** 40):
        grads = tensors(r, [(700,)], torch.float32, 0.1)[1]
        check_step(desc, kw, params, grads, state, step, 1e-3, 0.5, None)


def test_roots_above_zero_are_not_held_as_zero():
    """An element whose gradient is far below its block's moves by no more than the bound
    of a step with its gradient gone, lr / (1 - beta1) at most, and never by m / eps."""
    tbe = lib()
    desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", bits=8, beta1=0.9, beta2=0.999, eps=1e-12,
                         weight_decay=0.0)
    p = torch.zeros(256, device="cuda")
    state = tbe.AdamWState(desc, [p])
    g = torch.full((256,), 1e-7, device="cuda")
    g[0] = 1.0
    lr = torch.tensor([1e-3], device="cuda")
    tbe.tbe_adamw_step(desc, [p], [g], state, torch.tensor([1], device="cuda"), lr)
    assert (state.v[0].float() > 0).all()
    before = p.clone()
    tbe.tbe_adamw_step(desc, [p], [torch.zeros_like(g)], state, torch.tensor([2], device="cuda"), lr)
    assert (p - before).abs().max().item() <= 1e-2


def test_values_that_are_none():
    """NaN and infinities of a gradient stay with their element; zero gradients from zero
    moments leave the parameters but for their decay; tiny blocks are held as zeros."""
    tbe = lib()
    for bits in (32, 8):
        desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", bits=bits, weight_decay=0.0)
        p = torch.ones(1024, device="cuda")
        state = tbe.AdamWState(desc, [p])
        lr = torch.tensor([1e-2], device="cuda")
        g = torch.randn(1024, generator=gen(1)).cuda()
        g[300], g[301], g[302] = float("nan"), float("inf"), float("-inf")
        g[512:768] = 0.0
        g[768:] = 1e-33
        for step in (1, 2):
            tbe.tbe_adamw_step(desc, [p], [g], state, torch.tensor([step], device="cuda"), lr)
        bad = torch.zeros(1024, dtype=torch.bool, device="cuda")
        bad[300:303] = True
        assert torch.isfinite(p[~bad]).all() and torch.isnan(p[300])
        assert (p[512:768] == 1).all()
        m = state.m[0].float()
        assert torch.isfinite(m[~bad]).all() and torch.isnan(m[300])
        if bits == 8:
            assert torch.isnan(m[300:303]).all() and torch.isnan(state.v[0].float()[300:303]).all()
            assert (state.ms[0][2:] == 0).all() and (m[512:] == 0).all() and torch.isfinite(state.ms[0]).all()


def test_step_and_rate_are_read_on_the_device():
    """A captured step follows the device's step count, rate and scale."""
    tbe = lib()
    for bits in (32, 8):
        desc = tbe.AdamWDesc(pdtype="f32", gdtype="bf16", cdtype="bf16", bits=bits, weight_decay=0.1)
        r = gen(7)
        shapes = [(300,), (4097,), (64, 65)]
        a, b = tensors(r, shapes, torch.float32, 1.0)[1], None
        b = [t.clone() for t in a]
        grads = tensors(r, shapes, torch.bfloat16, 0.1)[1]
        ca, cb = ([torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes] for _ in "ab")
        sa, sb = tbe.AdamWState(desc, a), tbe.AdamWState(desc, b)
        step, lr = torch.zeros(1, dtype=torch.int64, device="cuda"), torch.zeros(1, device="cuda")
        scale = torch.ones(1, device="cuda")
        tbe.tbe_adamw_step(desc, b, grads, sb, step, lr, scale, cb)   # (first use outside the capture)
        b = [t.clone() for t in a]
        sb = tbe.AdamWState(desc, b)
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            tbe.tbe_adamw_step(desc, b, grads, sb, step, lr, scale, cb)
        for t in range(1, 5):
            step.fill_(t)
            lr.fill_(1e-2 / t)
            scale.fill_(0.5 * t)
            for q in grads:
                q.mul_(-1.25)
            tbe.tbe_adamw_step(desc, a, grads, sa, step, lr, scale, ca)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(a + ca, b + cb)), (bits, t)
            assert torch.equal(sa.m_flat.view(torch.uint8), sb.m_flat.view(torch.uint8))
            assert torch.equal(sa.v_flat.view(torch.uint8), sb.v_flat.view(torch.uint8))


def test_refusals():
    tbe = lib()
    desc = tbe.AdamWDesc(pdtype="f32", gdtype="f32", cdtype="bf16")
    p = [torch.zeros(8, device="cuda"), torch.zeros(4, device="cuda")]
    g, c = [torch.zeros_like(t) for t in p], [t.bfloat16() for t in p]
    state = tbe.AdamWState(desc, p)
    step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.ones(1, device="cuda")

    def call(p=p, g=g, c=c, state=state, step=step, lr=lr):
        tbe.tbe_adamw_step(desc, p, g, state, step, lr, None, c)
    call()
    with pytest.raises(TypeError, match="grads: expected 2 tensors, got 1"):
        call(g=g[:1])
    with pytest.raises(TypeError, match="copies: expected a list"):
        call(c=None)
    with pytest.raises(TypeError, match="params: expected 4 elements, got 8"):
        call(p=[p[0], p[0]])
    with pytest.raises(TypeError, match="grads: expected torch.float32"):
        call(g=[t.half() for t in g])
    with pytest.raises(TypeError, match="grads: must be contiguous"):
        call(g=[torch.zeros(16, device="cuda")[::2], g[1]])
    with pytest.raises(TypeError, match="step: expected torch.int64"):
        call(step=lr)
    with pytest.raises(TypeError, match="lr: must be a device tensor"):
        call(lr=torch.ones(1))
    with pytest.raises(TypeError, match="an AdamWState of the description's bits"):
        call(state=tbe.AdamWState(tbe.AdamWDesc(bits=8), p))
    for bad in ([p[0], p[0][2:6]], [p[0], p[0][4:]]):    # the same parameters twice
        with pytest.raises(tbe.TbeError) as e:
            call(p=bad)
        assert e.value.status == tbe.TBE_ERR_ARG
    with pytest.raises(tbe.TbeError):
        call(c=[c[0], c[0][:4]])
