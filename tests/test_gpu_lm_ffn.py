"""The experts' gated feed-forward products and their gradients against 64-bit
formulas.

Tolerances follow the roundings through the formulas: u = 2^-24 times the sum of
magnitudes for each of a product's n terms, half a step of the type where a value
between two products is rounded to it, and 2^-19 for the activation, whose
exponential is a power of 2 of a rounded exponent (relative to |g| + 1).
"""
import math

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, TINY, U32, around, close, gen, half, new, say, view_of

pytestmark = pytest.mark.gpu
ACT = 2.0 ** -19
SLOPE = 1.13   # of both activations, at most


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


def act(name, g):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    cdf = 0.5 * torch.erfc(-g / math.sqrt(2))
    return g * cdf, cdf + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)


def make(g, counts, D, F, t, tail=0):
    """Inputs for experts with `counts` rows and `tail` rows of nobody."""
    E, M = len(counts), sum(counts) + tail
    offsets = torch.tensor([0] + counts).cumsum(0).to(torch.int32).cuda()

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(DT[t]).cuda()
    s = {"offsets": offsets, "xs": rnd(M, D), "gate": rnd(E, F, D, std=D ** -0.5),
         "up": rnd(E, F, D, std=D ** -0.5), "down": rnd(E, D, F, std=F ** -0.5), "dys": rnd(M, D, std=0.3)}
    for k in ("xs", "dys"):   # nobody's rows are not read
        s[k][sum(counts):] = float("nan")
    return s


def stacked(w, stride):
    """w's matrices with longer rows and a gap between them."""
    if not stride:
        return w
    base = torch.full((w.shape[0], w.shape[1] + 1, w.shape[2] + stride), float("nan"), dtype=w.dtype, device="cuda")
    v = base[:, :w.shape[1], :w.shape[2]]
    v.copy_(w)
    return v


def forward(s, t, name, keep=True, stride=0, desc=None):
    tbe = lib()
    M, D = s["xs"].shape
    E, F, _ = s["gate"].shape
    d = desc or tbe.FfnDesc(M, E, D, F, dtype=t, act=name)
    ws = tbe.ffn_workspace(d)
    ws.fill_(255)
    ys = new(M, D, DT[t], stride)
    pre = new(M, 2 * F, DT[t], stride) if keep else None
    tbe.tbe_ffn_forward(d, view_of(s["xs"], stride), s["offsets"], stacked(s["gate"], stride),
                        stacked(s["up"], stride), stacked(s["down"], stride), pre, ys, ws)
    torch.cuda.synchronize()
    return ys, pre


def backward(s, t, name, pre, stride=0):
    tbe = lib()
    M, D = s["xs"].shape
    E, F, _ = s["gate"].shape
    d = tbe.FfnDesc(M, E, D, F, dtype=t, act=name)
    ws = tbe.ffn_workspace(d)
    ws.fill_(255)
    dxs = new(M, D, DT[t], stride)
    out = [stacked(torch.full_like(s[k], float("nan")), stride) for k in ("gate", "up", "down")]
    tbe.tbe_ffn_backward(d, view_of(s["dys"], stride), view_of(s["xs"], stride), s["offsets"],
                         stacked(s["gate"], stride), stacked(s["up"], stride), stacked(s["down"], stride),
                         view_of(pre, stride), dxs, *out, ws)
    torch.cuda.synchronize()
    return dxs, out


def check(s, t, name, stride=0, keep=True):
    D, F = s["down"].shape[1:]
    h = half(t) if t != "f32" else 0.0
    tiny = TINY[t] if t != "f32" else 0.0
    o = s["offsets"].tolist()
    ys, pre = forward(s, t, name, keep, stride)
    if pre is None:
        pre = forward(s, t, name, True, 0)[1]
    dxs, grads = backward(s, t, name, torch.nan_to_num(pre), stride)
    for e, (a, z) in enumerate(zip(o[:-1], o[1:])):
        x, dy = s["xs"][a:z].to(F64), s["dys"][a:z].to(F64)
        wg, wu, wd = (s[k][e].to(F64) for k in ("gate", "up", "down"))
        g, u = x @ wg.t(), x @ wu.t()
        og, ou = ((D + 2) * U32 * (x.abs() @ w.abs().t()) for w in (wg, wu))
        close(pre[a:z, :F], g, og, t, f"g of expert {e}")
        close(pre[a:z, F:], u, ou, t, f"u of expert {e}")
        v, _ = act(name, g)
        off = (SLOPE * og + ACT * v.abs() * (g.abs() + 1) + 8 * U32 * v.abs()) * (u.abs() + ou) + v.abs() * ou
        off = off + h * (v * u).abs() + tiny + TINY["f32"]
        close(ys[a:z], (v * u) @ wd.t(), off @ wd.abs().t() + (F + 2) * U32 * ((v * u).abs() @ wd.abs().t()), t,
              f"ys of expert {e}")
        # the backward from the products as they are kept
        g, u = pre[a:z, :F].to(F64), pre[a:z, F:].to(F64)
        v, dv = act(name, g)
        dh = dy @ wd
        odh = (D + 2) * U32 * (dy.abs() @ wd.abs())
        av, adv = ACT * (v.abs() + 1) * (g.abs() + 1), ACT * (g.abs() + 1)
        du, dg, hh = dh * v, dh * u * dv, v * u
        odu = odh * (v.abs() + av) + dh.abs() * av + h * du.abs() + tiny
        odg = odh * (u * dv).abs() + (dh * u).abs() * (adv + 8 * U32) + odh * u.abs() * adv + h * dg.abs() + tiny
        ohh = av * u.abs() + (h + 8 * U32) * hh.abs() + tiny
        close(dxs[a:z], dg @ wg + du @ wu, odg @ wg.abs() + odu @ wu.abs() +
              (2 * F + 2) * U32 * (dg.abs() @ wg.abs() + du.abs() @ wu.abs()), t, f"dxs of expert {e}")
        n = (z - a + 2) * U32
        for got, left, lo, right, what in ((grads[0][e], dg, odg, x, "dgate"), (grads[1][e], du, odu, x, "dup"),
                                           (grads[2][e].t(), hh, ohh, dy, "ddown")):
            close(got, left.t() @ right, lo.t() @ right.abs() + n * (left.abs().t() @ right.abs()), t,
                  f"{what} of expert {e}")
    kept = o[-1]
    for v in (ys, dxs):   # rows of nobody are left as they were
        assert torch.isnan(v[kept:]).all()
        around(v, stride) if v.shape[0] else None
    if stride:
        for w in grads:
            assert torch.isnan(w._base[:, -1]).all() and torch.isnan(w._base[:, :, w.shape[2]:]).all()


FFN = [  # rows of each expert, rows of nobody, D, F, type, activation, stride padding
    ([1], 0, 1, 1, "f32", "silu", 0),
    ([3], 0, 8, 8, "bf16", "silu", 0),
    ([1, 0, 2], 1, 64, 64, "bf16", "silu", 0),
    ([0, 0, 0], 4, 64, 32, "bf16", "gelu", 0),
    ([5, 1, 0, 9], 2, 100, 36, "f16", "gelu", 0),
    ([17, 128, 3], 0, 72, 200, "bf16", "silu", 3),
    ([130], 7, 129, 65, "f16", "silu", 0),
    ([200, 60], 0, 257, 131, "f32", "gelu", 1),
    ([40, 300], 0, 96, 520, "f32", "silu", 0),
    ([129, 127, 128, 256, 1], 5, 512, 256, "bf16", "silu", 0),
    ([300, 10, 500], 3, 264, 328, "bf16", "gelu", 8),
    ([700, 900], 0, 640, 384, "f16", "silu", 0),
    ([4] * 33, 0, 192, 160, "bf16", "silu", 0),
    ([2, 1, 0, 3] * 40, 1, 64, 96, "bf16", "silu", 0),
    ([64, 31, 0, 17], 0, 1024, 712, "bf16", "silu", 0),
    ([1000], 0, 320, 1000, "bf16", "gelu", 0),
    # few rows an expert, one to four blocks of 16 at a time, by four waves and by more
    ([1] * 32, 0, 512, 768, "bf16", "silu", 0),
    ([0, 1, 0, 0, 3], 0, 1030, 515, "f16", "gelu", 5),
    ([100, 1, 0, 3] + [0] * 12, 2, 200, 136, "bf16", "silu", 0),
    ([2, 17], 0, 96, 2056, "f32", "silu", 0),
    ([20] * 7 + [31], 0, 264, 1024, "bf16", "silu", 0),
    ([25], 3, 72, 80, "f16", "silu", 1),
    ([40, 63, 0, 90], 1, 136, 2048, "bf16", "gelu", 0),
    ([33], 0, 65, 63, "f32", "silu", 0),
    # enough tiles of 128 x 128
    ([70] * 30 + [1] * 5 + [200] * 5, 9, 1024, 520, "bf16", "silu", 0),
    ([80] * 16, 0, 300, 1030, "f32", "gelu", 0),
    ([150] * 8 + [129] * 8, 0, 1100, 1111, "f16", "silu", 0),
]


@pytest.mark.parametrize("counts,tail,D,F,t,name,stride", FFN)
def test_ffn(counts, tail, D, F, t, name, stride):
    say("ffn", counts if len(counts) < 8 else len(counts), tail, D, F, t, name, stride)
    check(make(gen(sum(counts) + D + F), counts, D, F, t, tail), t, name, stride, keep=D % 2 == 0)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_small_tiles_of_which_a_workgroup_has_several(t):
    # 60 experts' three blocks of 64 rows by eight of columns are more than 1024 workgroups
    counts = [129] * 60
    say("small tiles, several", t)
    check(make(gen(61), counts, 64, 512, t, 3), t, "silu")


@pytest.mark.parametrize("t,name", [("bf16", "silu"), ("f16", "gelu")])
def test_ffn_of_large_tiles(t, name):
    """Products of 256 x 256 tiles, a tile's steps, rows and columns cut at every place."""
    counts = [700, 1, 515, 0, 1030, 256, 255, 1343]
    say("ffn large", counts, t, name)
    check(make(gen(11), counts, 4104, 4168, t, 5), t, name)


def test_same_bits():
    """The same call again and again: no result depends on which workgroup comes first, and
    nothing is read before it has arrived."""
    for counts, D, F in (([700, 1, 515, 0, 1030, 256, 255, 1343], 4096, 4160), ([70] * 30 + [200] * 5, 1024, 520),
                         ([9, 300], 256, 192), ([1] * 32, 512, 768)):
        s = make(gen(sum(counts)), counts, D, F, "bf16")
        ys, pre = forward(s, "bf16", "silu")
        dxs, grads = backward(s, "bf16", "silu", pre)
        for _ in range(4):
            ys2, pre2 = forward(s, "bf16", "silu")
            dxs2, grads2 = backward(s, "bf16", "silu", pre)
            assert torch.equal(ys, ys2) and torch.equal(pre, pre2) and torch.equal(dxs, dxs2)
            assert all(torch.equal(a, b) for a, b in zip(grads, grads2))


def test_no_rows():
    s = make(gen(1), [0, 0], 64, 64, "bf16")
    ys, pre = forward(s, "bf16", "silu")
    dxs, grads = backward(s, "bf16", "silu", pre)
    assert ys.shape == (0, 64) and all(not w.any() for w in grads)


def test_offsets_that_are_none():
    """Offsets outside [0, M], or below their predecessor, are taken for the nearest that are
    neither: nothing is read or written beyond the rows, and the gradients agree with that."""
    counts = [7, 0, 0, 33]
    s = make(gen(2), counts, 64, 96, "bf16")
    want = forward(s, "bf16", "silu")
    grads = backward(s, "bf16", "silu", want[1])
    s["offsets"] = torch.tensor([-2 ** 31, 7, -5, 3, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    got = forward(s, "bf16", "silu")
    other = backward(s, "bf16", "silu", want[1])
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert torch.equal(grads[0], other[0]) and all(torch.equal(a, b) for a, b in zip(grads[1], other[1]))


def test_values_that_are_none_stay_in_their_rows_and_experts():
    s = make(gen(3), [40, 40, 40], 128, 64, "bf16")
    ys, pre = forward(s, "bf16", "silu")
    dxs, grads = backward(s, "bf16", "silu", pre)
    for k in ("xs", "dys"):
        s[k][45] = float("nan")
    ys2, pre2 = forward(s, "bf16", "silu")
    dxs2, grads2 = backward(s, "bf16", "silu", pre2)
    keep = torch.arange(120, device="cuda") != 45
    assert torch.isnan(ys2[45]).all() and torch.isnan(dxs2[45]).all()
    for a, b in ((ys, ys2), (pre, pre2), (dxs, dxs2)):
        assert torch.equal(a[keep], b[keep])
    for a, b in zip(grads, grads2):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2]) and torch.isnan(b[1]).all()


def test_experts_that_share_a_matrix():
    """An expert stride of zero, and gate and up side by side in one tensor."""
    s = make(gen(4), [20, 30], 64, 48, "bf16")
    both = torch.cat([s["gate"], s["up"]], dim=1)
    s["down"] = s["down"][:1].expand(2, 64, 48)
    want = forward({**s, "down": s["down"].contiguous()}, "bf16", "silu")
    got = forward({**s, "gate": both[:, :48], "up": both[:, 48:]}, "bf16", "silu")
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_gradients_against_differences():
    """Along a direction, against a central difference of sum(ys * c) over 2 h = 2^-4 of a
    unit direction: sums of order 10 in float32 leave 10 * 256 u / h, and a third derivative
    of order 100 adds h^2 / 6 of that."""
    g = gen(5)
    for name in ("silu", "gelu"):
        s = make(g, [5, 0, 9], 24, 20, "f32")
        ys, pre = forward(s, "f32", name)
        dxs, (dgate, dup, ddown) = backward(s, "f32", name, pre)
        h = 2.0 ** -5

        def value(s):
            return (forward(s, "f32", name)[0].to(F64) * s["dys"].to(F64)).sum().item()
        for k, grad in (("xs", dxs), ("gate", dgate), ("up", dup), ("down", ddown)):
            for v in (grad, torch.randn(grad.shape, generator=g).cuda()):
                v = v / v.norm()
                got = (value({**s, k: s[k] + h * v}) - value({**s, k: s[k] - h * v})) / (2 * h)
                want = (grad.to(F64) * v.to(F64)).sum().item()
                assert abs(got - want) <= 10 * 256 * U32 / h + 100 * h * h / 6, (name, k)


def test_captured_and_replayed():
    """Two graphs over one workspace, replayed in turn with eager work between, the offsets
    changing on the device."""
    tbe = lib()
    M, E, D, F = 300, 4, 128, 192
    d = tbe.FfnDesc(M, E, D, F)
    ws = tbe.ffn_workspace(d)
    runs = []
    for k in range(2):
        s = make(gen(6 + k), [100, 50, 100, 50], D, F, "bf16")
        out = {"ys": torch.empty_like(s["xs"]), "pre": torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda"),
               "dxs": torch.empty_like(s["xs"]), "dgate": torch.empty_like(s["gate"]),
               "dup": torch.empty_like(s["up"]), "ddown": torch.empty_like(s["down"])}

        def once(s=s, out=out):
            tbe.tbe_ffn_forward(d, s["xs"], s["offsets"], s["gate"], s["up"], s["down"], out["pre"], out["ys"], ws)
            tbe.tbe_ffn_backward(d, s["dys"], s["xs"], s["offsets"], s["gate"], s["up"], s["down"], out["pre"],
                                 out["dxs"], out["dgate"], out["dup"], out["ddown"], ws)
        once()
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
            once()
        runs.append((graph, s, out, once))
    for counts in ([100, 50, 100, 50], [0, 300, 0, 0], [1, 2, 290, 7]):
        for graph, s, out, once in runs:
            s["offsets"].copy_(torch.tensor([0] + counts).cumsum(0))
            once()
            torch.cuda.synchronize()
            want = {k: v.clone() for k, v in out.items()}
            for v in out.values():
                v.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], want[k]) for k in out), counts


def test_with_the_experts_plan():
    """Routed tokens through plan, dispatch, the products, combine, and back: the operators
    together against the products token by token."""
    tbe = lib()
    N, K, E, D, F = 90, 3, 7, 64, 40
    g = gen(8)
    x = torch.randn(N, D, generator=g).cuda()
    s = make(g, [0] * E, D, F, "f32")
    ids = torch.stack([torch.randperm(E, generator=g)[:K] for _ in range(N)]).cuda()
    ids[3, 1] = -1
    w = torch.rand(N, K, generator=g).cuda()
    dout = torch.randn(N, D, generator=g).cuda()
    ed, fd = tbe.ExpertDesc(N, K, E, D, dtype="f32"), tbe.FfnDesc(N * K, E, D, F, dtype="f32")
    plan, ws = tbe.ExpertPlan(ed), tbe.ffn_workspace(fd)
    tbe.tbe_expert_plan(ed, ids, plan, tbe.expert_workspace(ed))
    xs, ys, pre = (torch.empty(N * K, c, device="cuda") for c in (D, D, 2 * F))
    tbe.tbe_expert_dispatch(ed, x, plan.slots, xs)
    tbe.tbe_ffn_forward(fd, xs, plan.offsets, s["gate"], s["up"], s["down"], pre, ys, ws)
    out = torch.empty_like(x)
    tbe.tbe_expert_combine(ed, ys, plan.slots, w, out)
    dys, dw, dxs, dx = torch.empty_like(ys), torch.empty_like(w), torch.empty_like(xs), torch.empty_like(x)
    tbe.tbe_expert_combine_backward(ed, dout, ys, plan.slots, w, dys, dw)
    grads = [torch.empty_like(s[k]) for k in ("gate", "up", "down")]
    tbe.tbe_ffn_backward(fd, dys, xs, plan.offsets, s["gate"], s["up"], s["down"], pre, dxs, *grads, ws)
    tbe.tbe_expert_dispatch_backward(ed, dxs, plan.slots, dx)

    leaf = {k: v.to(F64).requires_grad_() for k, v in
            (("x", x), ("w", w), ("gate", s["gate"]), ("up", s["up"]), ("down", s["down"]))}
    at = ids.clamp(min=0)
    a = torch.einsum("nd,nkfd->nkf", leaf["x"], leaf["gate"][at])
    b = torch.einsum("nd,nkfd->nkf", leaf["x"], leaf["up"][at])
    y = torch.einsum("nkf,nkdf->nkd", torch.nn.functional.silu(a) * b, leaf["down"][at])
    want = (y * (leaf["w"] * (ids >= 0))[:, :, None]).sum(1)
    want.backward(dout.to(F64))
    # values of order 1 to 100 through three products of at most 270 terms
    for got, ref, what in ((out, want.detach(), "out"), (dx, leaf["x"].grad, "dx"), (dw, leaf["w"].grad, "dw"),
                           (grads[0], leaf["gate"].grad, "dgate"), (grads[1], leaf["up"].grad, "dup"),
                           (grads[2], leaf["down"].grad, "ddown")):
        close(got, ref, 2.0 ** -15 * ref.abs().max().item(), "f32", what)
