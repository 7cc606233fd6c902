"""The norm, the experts' products and AdamW where elements lie beyond 2^31 places: the
same bits as the same values close together."""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import gen, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


@pytest.fixture(autouse=True)
def _give_back():
    yield
    torch.cuda.empty_cache()


def far(v, ld, fill=True):
    """v's rows, ld elements apart."""
    base = torch.empty((v.shape[0] - 1) * ld + v.shape[1], dtype=v.dtype, device="cuda")
    w = base.as_strided(v.shape, (ld, 1))
    if fill:
        w.copy_(v)
    return w


def rnd(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


@pytest.mark.parametrize("D,ld", [(512, 1 << 20), (515, (1 << 20) + 3), (20000, 1 << 20)])
def test_norm(D, ld):
    say("norm far", D, ld)
    tbe, g, N = lib(), gen(D), 2100
    x, dy, w, b = rnd(g, N, D), rnd(g, N, D), rnd(g, D, dtype=torch.float32), rnd(g, D, dtype=torch.float32)
    d = tbe.NormDesc(N, D)
    ws, out = tbe.norm_workspace(d), []
    for place in (lambda v, fill: v if fill else torch.empty_like(v), lambda v, fill: far(v, ld, fill)):
        xx, gg, y, dx = place(x, True), place(dy, True), place(x, False), place(x, False)
        stats = torch.empty(N, 2, device="cuda")
        dw, db = torch.empty_like(w), torch.empty_like(b)
        tbe.tbe_norm_forward(d, xx, w, b, y, stats)
        tbe.tbe_norm_backward(d, gg, xx, w, stats, dx, dw, db, ws)
        torch.cuda.synchronize()
        out.append([v.clone() for v in (y, stats, dx, dw, db)])
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("counts,D,F,ld,stride", [
    ([9000, 8000], 64, 96, 1 << 17, (1 << 31) + 64),           # aligned
    ([1100, 1000], 64, 96, (1 << 20) + 8, (1 << 31) + 64),     # rows too far apart for direct loads
    ([3, 5], 64, 96, 1 << 29, (1 << 31) + 64)])                # few rows
def test_ffn(counts, D, F, ld, stride):
    say("ffn far", counts, D, F, ld, stride)
    tbe, g, M = lib(), gen(D + F), sum(counts)
    xs, dys = rnd(g, M, D), rnd(g, M, D)
    gate, up, down = rnd(g, 2, F, D, std=0.1), rnd(g, 2, F, D, std=0.1), rnd(g, 2, D, F, std=0.1)
    offsets = torch.tensor([0, counts[0], M], dtype=torch.int32, device="cuda")
    d = tbe.FfnDesc(M, 2, D, F)
    ws, out = tbe.ffn_workspace(d), []

    def apart(w, fill):   # the second expert's matrix `stride` elements behind the first
        base = torch.empty(stride + w[0].numel(), dtype=w.dtype, device="cuda")
        v = base.as_strided(w.shape, (stride, w.shape[2], 1))
        if fill:
            v.copy_(w)
        return v

    def near(v, fill):
        return v if fill else torch.empty_like(v)
    for rows, mats in ((near, near), (lambda v, fill: far(v, ld, fill), apart)):
        x, dy, ys, dxs = rows(xs, True), rows(dys, True), rows(xs, False), rows(xs, False)
        pre = rows(torch.empty(M, 2 * F, dtype=xs.dtype, device="cuda"), False)
        a, b, c = (mats(w, True) for w in (gate, up, down))
        grads = [mats(w, False) for w in (gate, up, down)]
        tbe.tbe_ffn_forward(d, x, offsets, a, b, c, pre, ys, ws)
        tbe.tbe_ffn_backward(d, dy, x, offsets, a, b, c, pre, dxs, *grads, ws)
        torch.cuda.synchronize()
        out.append([v.clone() for v in (ys, pre, dxs, *grads)])
        del x, dy, ys, dxs, pre, a, b, c, grads
    assert all(torch.equal(p, q) for p, q in zip(*out))


@pytest.mark.parametrize("bits", [8, 32])
def test_adamw(bits):
    """A tensor of more than 2^31 elements: its last ones against a tensor of them alone."""
    say("adamw far", bits)
    tbe, n, tail = lib(), (1 << 31) + 777, 4096 + 777
    d = tbe.AdamWDesc("bf16", "bf16", bits=bits)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros_like(p)
    g = gen(bits)
    for v in (p, q):
        v[-tail:] = rnd(g, tail)
    step, lr = torch.ones(1, dtype=torch.int64, device="cuda"), torch.full((1,), 0.01, device="cuda")
    last, grad = p[-tail:].clone(), q[-tail:].clone()
    state, other = tbe.AdamWState(d, [p]), tbe.AdamWState(d, [last])
    tbe.tbe_adamw_step(d, [p], [q], state, step, lr)
    tbe.tbe_adamw_step(d, [last], [grad], other, step, lr)
    torch.cuda.synchronize()
    assert torch.equal(p[-tail:], last) and not p[:64].any() and not p[n // 2:n // 2 + 64].any()
    for a, b in ((state.m, other.m), (state.v, other.v)):
        assert torch.equal(a[0][-tail:].contiguous().view(torch.uint8), b[0].contiguous().view(torch.uint8))
    if bits == 8:
        blocks = (tail + 255) // 256
        assert torch.equal(state.ms[0][-blocks:], other.ms[0]) and torch.equal(state.vs[0][-blocks:], other.vs[0])
