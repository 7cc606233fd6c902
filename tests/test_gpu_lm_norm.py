"""Layer norm and its gradients against 64-bit formulas.

Tolerances count roundings, u = 2^-24 each. A sum over a row of D columns adds
D / 1024 + 16 values in a lane (a lane has at most 16 columns in registers) and
joins lanes in at most 10 steps, so with the products and the final scaling
n = D / 512 + 64 roundings bound it. The mean's own rounding is corrected from
the row, so no bound grows with the mean.
"""
import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import DT, F64, U32, around, close, gen, new, randn, say, view_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    lib()


def inputs(g, N, D, x, w, mean=1.0):
    rows = randn(g, N, D) * (0.2 + 2 * torch.rand(N, 1, generator=g).cuda()) + mean * randn(g, N, 1)
    return (rows.to(DT[x]), (1 + 0.3 * randn(g, D)).to(DT[w]), (0.3 * randn(g, D)).to(DT[w]),
            (0.1 * randn(g, N, D)).to(DT[x]))


def formula(x, w, b, dy, eps):
    x, dy = x.to(F64), dy.to(F64)
    w = torch.ones(x.shape[1], dtype=F64, device="cuda") if w is None else w.to(F64)
    b = torch.zeros_like(w) if b is None else b.to(F64)
    mean = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)
    xh = (x - mean) * r
    a = dy * w
    m1 = (a * xh).mean(1, keepdim=True)
    return {"mean": mean, "r": r, "xh": xh, "w": w, "y": xh * w + b, "a": a, "dy": dy,
            "dx": r * (a - a.mean(1, keepdim=True) - xh * m1),
            "size": r * (a.abs() + a.abs().mean(1, keepdim=True) + xh.abs() * (a * xh).abs().mean(1, keepdim=True)),
            "dw": (dy * xh).sum(0), "db": dy.sum(0)}


def check(N, D, x, w, xv, wv, bv, dyv, stride=0, eps=1e-5, has_dw=True, has_db=True):
    tbe = lib()
    d = tbe.NormDesc(N, D, dtype=x, wdtype=w, eps=eps)
    X, DY = view_of(xv, stride), view_of(dyv, stride)
    y, dx = new(N, D, DT[x], stride), new(N, D, DT[x], stride)
    stats = torch.full((N, 2), float("nan"), device="cuda")
    tbe.tbe_norm_forward(d, X, wv, bv, y, stats)
    dw = torch.full((D,), float("nan"), dtype=DT[w], device="cuda") if has_dw else None
    db = torch.full((D,), float("nan"), dtype=DT[w], device="cuda") if has_db else None
    ws = tbe.norm_workspace(d)
    ws.fill_(255)
    tbe.tbe_norm_backward(d, DY, X, wv, stats, dx, dw, db, ws)
    torch.cuda.synchronize()
    f = formula(xv, wv, bv, dyv, eps)
    n = D / 512 + 64
    # of xh: its own roundings, and the means' of values of the row's deviation (1 in xh)
    xh_off = n * U32 * (f["xh"].abs() + 1)
    close(stats[:, 0], f["mean"][:, 0], (U32 * f["mean"].abs() + n * U32 / f["r"])[:, 0], "f32", "mean")
    close(stats[:, 1], f["r"][:, 0], n * U32 * f["r"][:, 0], "f32", "rstd")
    close(y, f["y"], xh_off * f["w"].abs() + 2 * U32 * f["y"].abs(), x, "y")
    close(dx, f["dx"], 4 * n * U32 * f["size"], x, "dx")
    rows = N / 256 + 256    # added one after the other: a workgroup's rows, then the workgroups
    if has_dw:
        off = (f["dy"].abs() * (xh_off + rows * U32 * f["xh"].abs())).sum(0)
        close(dw, f["dw"], off, w, "dw")
    if has_db:
        close(db, f["db"], rows * U32 * f["dy"].abs().sum(0), w, "db")
    if N:
        around(y, stride)
        around(dx, stride)
    return y, stats, dx, dw, db


NORM = [  # N, D, x, w, stride padding
    (0, 64, "bf16", "f32", 0), (1, 1, "f32", "f32", 0), (1, 3, "bf16", "bf16", 0), (5, 7, "f16", "f32", 2),
    (3, 8, "bf16", "f32", 0), (17, 100, "f32", "f32", 1), (33, 128, "bf16", "bf16", 0),
    (100, 129, "f16", "f16", 0), (7, 256, "bf16", "f32", 3), (1025, 500, "bf16", "f32", 0),
    (300, 513, "bf16", "bf16", 0), (2000, 1001, "f32", "f32", 0), (16, 2048, "bf16", "bf16", 0),
    (1500, 2040, "bf16", "f32", 0), (777, 1030, "f16", "f32", 0), (1100, 4096, "bf16", "f32", 0),
    (260, 4100, "bf16", "f32", 1), (40, 8191, "f16", "f16", 0), (9, 8200, "f32", "f32", 0),
    (11, 16384, "bf16", "f32", 0), (5, 16390, "bf16", "bf16", 0), (3, 40001, "f32", "f16", 5),
    (20011, 72, "bf16", "bf16", 0),
]


@pytest.mark.parametrize("N,D,x,w,stride", NORM)
def test_norm(N, D, x, w, stride):
    say("norm", N, D, x, w, stride)
    g = gen(N + 3 * D)
    check(N, D, x, w, *inputs(g, N, D, x, w), stride=stride)


@pytest.mark.parametrize("D", [512, 3000, 40000])
def test_rows_far_from_zero(D):
    """A mean 2^13 times the deviation: nothing of the deviation's precision is lost."""
    g = gen(D)
    x, w, b, dy = inputs(g, 37, D, "f32", "f32", mean=0.0)
    check(37, D, "f32", "f32", x + 8192.0, w, b, dy)


def test_without_weight_bias_or_their_gradients():
    g = gen(1)
    x, w, b, dy = inputs(g, 70, 96, "bf16", "f32")
    check(70, 96, "bf16", "f32", x, None, None, dy)
    check(70, 96, "bf16", "f32", x, w, None, dy, has_dw=False)
    check(70, 96, "bf16", "f32", x, None, b, dy, has_db=False)
    check(70, 96, "bf16", "f32", x, w, b, dy, has_dw=False, has_db=False)


def test_no_rows_give_zero_gradients():
    tbe = lib()
    d = tbe.NormDesc(0, 50, dtype="f32")
    e = torch.empty(0, 50, device="cuda")
    dw, db = torch.full((50,), 7.0, device="cuda"), torch.full((50,), 7.0, device="cuda")
    tbe.tbe_norm_backward(d, e, e, None, torch.empty(0, 2, device="cuda"), e, dw, db, tbe.norm_workspace(d))
    assert not dw.any() and not db.any()


def test_equal_values_and_values_that_are_none():
    """A row of equal values has y = b; NaN and infinities stay in their row."""
    tbe = lib()
    N, D = 9, 200
    g = gen(2)
    x, w, b, _ = inputs(g, N, D, "f32", "f32")
    clean = x.clone()
    x[2] = 3.0
    x[4, 7], x[6, 199] = float("nan"), float("inf")
    d = tbe.NormDesc(N, D, dtype="f32")
    y, z = torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty(N, 2, device="cuda")
    tbe.tbe_norm_forward(d, x, w, b, y, stats)
    tbe.tbe_norm_forward(d, clean, w, b, z, torch.empty_like(stats))
    assert torch.equal(y[2], b) and abs(stats[2, 1].item() - 1e-5 ** -0.5) < 1e-4 * 1e-5 ** -0.5
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).all()
    for n in (0, 1, 3, 5, 7, 8):
        assert torch.equal(y[n], z[n])


def test_broadcast_rows():
    """A row stride of zero: one row's values N times."""
    g = gen(3)
    x, w, b, dy = inputs(g, 1, 384, "bf16", "f32")
    a = check(50, 384, "bf16", "f32", x.expand(50, 384).contiguous(), w, b, dy.expand(50, 384).contiguous())
    tbe = lib()
    d = tbe.NormDesc(50, 384)
    y, dx = torch.empty(50, 384, dtype=torch.bfloat16, device="cuda"), None
    stats = torch.empty(50, 2, device="cuda")
    tbe.tbe_norm_forward(d, x.expand(50, 384), w, b, y, stats)
    dx, dw, db = torch.empty_like(y), torch.empty_like(w), torch.empty_like(w)
    tbe.tbe_norm_backward(d, dy.expand(50, 384), x.expand(50, 384), w, stats, dx, dw, db, tbe.norm_workspace(d))
    for one, other in zip(a, (y, stats, dx, dw, db)):
        assert torch.equal(one, other)


def test_gradients_against_differences():
    """The gradient along a direction against the change of sum(y * c): a central difference
    over a step h of a unit direction. Values of order 10 in float32 over 2 h = 2^-5 leave
    10 * 64 u / h, and the third derivative of order 100 adds h^2 / 6 of that."""
    tbe = lib()
    N, D = 6, 48
    g = gen(4)
    x, w, b, c = inputs(g, N, D, "f32", "f32")
    d = tbe.NormDesc(N, D, dtype="f32")
    y, stats = torch.empty_like(x), torch.empty(N, 2, device="cuda")

    def value(x, w, b):
        tbe.tbe_norm_forward(d, x, w, b, y, stats)
        return (y.to(F64) * c.to(F64)).sum().item()

    value(x, w, b)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    tbe.tbe_norm_backward(d, c, x, w, stats, dx, dw, db, tbe.norm_workspace(d))
    h = 2.0 ** -6
    for k, grad in enumerate((dx, dw, db)):
        for v in (grad, randn(g, *grad.shape)):
            v = v / v.norm()
            up, down = [x, w, b], [x, w, b]
            up[k], down[k] = up[k] + h * v, down[k] - h * v
            got = (value(*up) - value(*down)) / (2 * h)
            assert abs(got - (grad.to(F64) * v.to(F64)).sum().item()) <= 10 * 64 * U32 / h + 100 * h * h / 6


def test_captured_and_replayed():
    """Two graphs over one workspace, replayed in turn with eager work between."""
    tbe = lib()
    N, D = 513, 1024
    g = gen(5)
    d = tbe.NormDesc(N, D)
    ws = tbe.norm_workspace(d)
    runs = []
    for _ in range(2):
        x, w, b, dy = inputs(g, N, D, "bf16", "f32")
        out = [torch.empty_like(x), torch.empty(N, 2, device="cuda"), torch.empty_like(x),
               torch.empty_like(w), torch.empty_like(w)]

        def once(x=x, w=w, b=b, dy=dy, out=out):
            tbe.tbe_norm_forward(d, x, w, b, out[0], out[1])
            tbe.tbe_norm_backward(d, dy, x, w, out[1], out[2], out[3], out[4], ws)
        once()
        torch.cuda.synchronize()
        want = [t.clone() for t in out]
        s = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            once()
        runs.append((graph, out, want, once))
    for turn in range(3):
        for graph, out, want, once in runs:
            for t in out:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
            once()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), turn
