"""8-bit moments of AdamW: the same codes and scales, to the bit, as the formulas in
float32 with every operation rounded by itself.

A code at the border of two neighbours falls to one of them by the last bit of the
value, and the next step's parameter follows it: so the last bit is part of what the
operator does. The formulas are evaluated here on the host, an operation at a time.
"""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, TINY, U32, close, gen, half, say
from tests.test_gpu_lm_adamw import BLOCK, decoded, moments, tensors

pytestmark = pytest.mark.gpu
KW = dict(beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


def encoded(x, least):
    """Codes and scales of x, whole blocks in float32."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top < 2.0 ** -100, torch.zeros(()), top * torch.tensor(1 / 448.0))
    q = torch.where(scale > 0, x / scale, torch.zeros(()))
    if least:
        q = torch.where((q > 0) & (q < 2.0 ** -9), torch.tensor(2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def expected(m, ms, v, vs, g, scale, kw=KW):
    """The moments after a step: (codes of m, scales, codes of v, scales)."""
    n, blocks = g.numel(), ms.numel()

    def whole(x):
        return torch.nn.functional.pad(x.reshape(-1).cpu().float(), (0, blocks * BLOCK - n))

    def decoded(c, s):
        return (whole(c).view(blocks, BLOCK) * s.cpu()[:, None]).view(-1)
    g = whole(g)
    if scale is not None:
        g = g * torch.tensor(scale)
    b1, b2 = torch.tensor(kw["beta1"]), torch.tensor(kw["beta2"])
    g1, g2 = torch.tensor(1 - kw["beta1"]), torch.tensor(1 - kw["beta2"])
    old = decoded(v, vs)
    mm = b1 * decoded(m, ms) + g1 * g
    # (from 64 bits, which rounds to the nearest float32; the host's float32 root need not)
    root = torch.sqrt((b2 * (old * old) + (g2 * g) * g).double()).float()
    return (*encoded(mm, False), *encoded(root, True))


def same_bits(state, i, want):
    for got, ref, what in zip((state.m[i], state.ms[i], state.v[i], state.vs[i]), want, ("m", "ms", "v", "vs")):
        got, ref = got.reshape(-1).cpu(), ref[:got.numel()]
        kind = torch.uint8 if got.dtype == torch.float8_e4m3fn else torch.int32
        off = got.view(kind) != ref.contiguous().view(kind)
        assert not off.any(), f"{what}[{i}]: {int(off.sum())} of {off.numel()} differ"


SMALL = [(1,), (7,), (255,), (256,), (257, 3), (0,), (4097,), (33, 129), (300, 1000)]
LARGE = [(1,), (1027, 2051), (255,), (3, 700001)]   # more than 2^22 elements


@pytest.mark.parametrize("shapes", [SMALL, LARGE], ids=["few", "many"])
@pytest.mark.parametrize("p,g,c", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("f32", "f16", None),
                                   ("bf16", "bf16", None), ("f16", "f16", None)])
def test_codes_and_scales(p, g, c, shapes):
    say("adamw codes", p, g, c, len(shapes))
    tbe = lib()
    r = gen(len(shapes) + len(g))
    desc = tbe.AdamWDesc(pdtype=p, gdtype=g, cdtype=c, bits=8, **KW)
    params = tensors(r, shapes, DT[p], 0.05, gap=1)[1]
    copies = tensors(r, shapes, DT[c], 0.0)[1] if c else None
    state = tbe.AdamWState(desc, params)
    for step in (1, 2, 3):
        grads = tensors(r, shapes, DT[g], 1e-3)[1]
        for q in grads:   # sizes that differ from place to place
            q.mul_(torch.exp(1.5 * torch.randn(q.shape, generator=r)).to(q.dtype).cuda())
        scale = 0.37 if step == 2 else None
        want = [expected(m, ms, v, vs, q, scale) for m, ms, v, vs, q in
                zip(state.m, state.ms, state.v, state.vs, grads)]
        tbe.tbe_adamw_step(desc, params, grads, state, torch.tensor([step], device="cuda"),
                           torch.tensor([1e-3], device="cuda"),
                           None if scale is None else torch.tensor([scale], device="cuda"), copies)
        torch.cuda.synchronize()
        for i, ref in enumerate(want):
            same_bits(state, i, ref)


def test_a_code_is_the_nearest_to_its_value_by_its_scale():
    """beta1 = 0.5 from zero moments: m is half the gradient exactly. Values at the borders of
    neighbouring codes and next to them, by blocks' scales: a code is off by half a step and
    the quotient's one rounding, 2^-24 of it, at most."""
    tbe = lib()
    r = gen(3)
    blocks = 4096
    top = torch.rand(blocks, 1, generator=r) + 0.5
    scale = top * torch.tensor(1 / 448.0)
    codes = torch.arange(1, 126, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    border = (codes[1:] + codes[:-1]) / 2
    at = border[torch.randint(0, border.numel(), (blocks, BLOCK - 1), generator=r)]
    m = (at * scale.double()).float()
    m = (m.view(torch.int32) + torch.randint(-2, 3, m.shape, generator=r, dtype=torch.int32)).view(torch.float32)
    m = torch.cat([top, torch.minimum(m, top)], 1).reshape(-1)
    desc = tbe.AdamWDesc("f32", "f32", bits=8, beta1=0.5, beta2=0.5)
    p = torch.zeros(m.numel(), device="cuda")
    state = tbe.AdamWState(desc, [p])
    tbe.tbe_adamw_step(desc, [p], [(2 * m).cuda()], state, torch.ones(1, dtype=torch.int64, device="cuda"),
                       torch.zeros(1, device="cuda"))
    torch.cuda.synchronize()
    assert torch.equal(state.ms[0].cpu(), scale.view(-1))
    q = m.double().view(blocks, BLOCK) / scale.double()
    got = state.m[0].cpu().float().double().view(blocks, BLOCK)
    step = torch.exp2(torch.floor(torch.log2(q)).clamp(min=-6) - 3)
    # (log2 of a quotient just below a power of two may say the power: its step is the half)
    step = torch.where(q < 8 * step, step / 2, step).clamp(min=2.0 ** -9)
    off = (got - q).abs() - step / 2
    assert (off <= 2.0 ** -24 * q).all(), f"{(off / q).max().item() * 2 ** 24:.3g} roundings beyond half a step"


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("p,g,c", [("f32", "f32", None), ("f32", "bf16", "bf16"), ("bf16", "bf16", None)])
def test_steps_of_many_elements(p, g, c, bits):
    """From 2^22 elements on a thread takes as many vectors as it can: against 64 bits.

    A moment m is two products and a sum, at most three roundings of its terms' sizes (they
    may cancel: the roundings are not relative to m), v and its root eight of their own. An
    8-bit moment is off by those and half a step, 2^-4 of it or 2^-10 of its scale."""
    say("adamw many", p, g, c, bits)
    tbe = lib()
    r = gen(bits + len(g))
    b1, b2 = KW["beta1"], KW["beta2"]
    desc = tbe.AdamWDesc(pdtype=p, gdtype=g, cdtype=c, bits=bits, **KW)
    params = tensors(r, LARGE, DT[p], 0.5, gap=1)[1]
    copies = tensors(r, LARGE, DT[c], 0.0, gap=3)[1] if c else None
    state = tbe.AdamWState(desc, params)
    rate = float(torch.tensor(1e-2))
    for step in (1, 2):
        grads = tensors(r, LARGE, DT[g], 0.01, gap=2)[1]
        old, p0 = moments(state), [x.to(F64).reshape(-1).clone() for x in params]
        tbe.tbe_adamw_step(desc, params, grads, state, torch.tensor([step], device="cuda"),
                           torch.tensor([1e-2], device="cuda"), torch.tensor([0.25], device="cuda"), copies)
        torch.cuda.synchronize()
        for i, q in enumerate(grads):
            q = q.to(F64).reshape(-1) * 0.25
            m = b1 * old[i][0] + (1 - b1) * q
            v = b2 * old[i][1] + (1 - b2) * q * q
            dm = 4 * U32 * (b1 * old[i][0].abs() + (1 - b1) * q.abs()) + TINY["f32"]
            root = torch.sqrt(v / (1 - b2 ** step)) + KW["eps"]
            move = rate / (1 - b1 ** step) * m / root
            x = p0[i] * (1 - rate * KW["weight_decay"]) - move
            off = rate / (1 - b1 ** step) * dm / root + 16 * U32 * move.abs() + 3 * U32 * p0[i].abs()
            close(params[i].reshape(-1), x, off, p, f"p[{i}]")
            if c:
                close(copies[i].reshape(-1), x, off + half("f32") * x.abs(), c, f"copy[{i}]")
            if bits == 32:
                close(state.m[i].reshape(-1), m, dm, "f32", f"m[{i}]")
                close(state.v[i].reshape(-1), v, 8 * U32 * v, "f32", f"v[{i}]")
                continue
            s, t = (k[i].to(F64).repeat_interleave(BLOCK)[:m.numel()] for k in (state.ms, state.vs))
            for got, want, own, by, what in ((decoded(state.m[i], state.ms[i]), m, dm, s, "m"),
                                             (decoded(state.v[i], state.vs[i]), v.sqrt(), 8 * U32 * v.sqrt(), t, "v")):
                size = want.abs() + own
                bound = torch.maximum(size * 2.0 ** -4, by * 2.0 ** -10) * (1 + 4 * U32) + own
                if what == "v":   # a root above zero is held as at least 2^-9 of the scale
                    bound = torch.where(size < by * 2.0 ** -9, by * 2.0 ** -9, bound)
                err = (got - want).abs()
                assert (err <= bound).all(), f"{what}[{i}]: {(err / bound).max().item():.3g} of the bound"
