"""Language-model operators where a kernel changes its way: sizes around the
borders of its variants, masks and values far from zero, many pieces. Against
the 64-bit implementations and tolerances of test_gpu_lm."""
import math

import pytest
import torch

from tests.gpu_common import lib
from tests.test_gpu_lm import (DT, F64, U32, close, distill_case, distill_ref, gen, new, randn,
                               run_distill, say, token_ids, view_of)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check_distill(tbe, xs, ids, ts, gl, tau, x, t="f32", idx64=True, stride=0):
    N, V = xs.shape
    K = ids.shape[1]
    desc = tbe.DistillDesc(N, V, K, dtype=x, tdtype=t, idx64=idx64, temperature=tau)
    want_l, want_g, bl, bg = distill_ref(xs, ids, ts, tau, gl)
    outs = run_distill(tbe, desc, xs, ids, ts, gl, stride)
    for loss, grad in (outs[:2], outs[2:]):
        close(loss, want_l, bl, "f32", "loss")
        close(grad, want_g, bg, x, "gradient")


# vectors of 16 bytes per row at the borders of the variants: none, 2 and 8 a lane
# of one wave, 8 of 256 threads, 12 and 16 of 1024, and parts beyond; each for
# few rows and for many
BORDERS = [(n, N) for N in (5, 300) for n in (0, 1, 127, 128, 129, 511, 512, 513, 2047, 2048, 2049)] + [
    (n, N) for N in (3, 258) for n in (4095, 4097, 8192, 8193, 12288, 12289)] + [
    (n, N) for N in (3, 257) for n in (16383, 16384)] + [(16385, 3), (32769, 3)]


@pytest.mark.parametrize("vectors,N", BORDERS)
def test_distill_borders(vectors, N):
    tbe = lib()
    for x in ("f32", "bf16"):
        if vectors > 8000 and N > 100 and x == "f32":
            continue  # the same way through the kernel as bf16, at twice the memory
        VE = 4 if x == "f32" else 8
        V = vectors * VE + (vectors + N) % VE + (vectors == 0)
        K = min(V, 11)
        say("distill borders", N, V, x)
        xs, ids, ts, gl = distill_case(gen(vectors + N), N, V, K, x, "f32", True, 0.2, distinct=False)
        check_distill(tbe, xs, ids, ts, gl, 1.0, x)


def test_distill_many_pieces():
    """A vocabulary of two million: 245 pieces of the backward."""
    tbe = lib()
    for V in (2000003, 2002944):
        xs, ids, ts, gl = distill_case(gen(V), 2, V, 40, "bf16", "f32", True, 0.0, distinct=False)
        check_distill(tbe, xs, ids, ts, gl, 1.0, "bf16")


@pytest.mark.parametrize("K", [64, 65, 257, 600, 1024])
@pytest.mark.parametrize("V", [700, 9000, 70001])
def test_distill_long_teachers(K, V):
    """More entries than threads, and places that repeat."""
    say("distill long teachers", K, V)
    tbe = lib()
    for N in (4, 260):
        xs, ids, ts, gl = distill_case(gen(K + V + N), N, V, K, "f16", "bf16", False, 0.2, distinct=False)
        ids[0] = 5
        check_distill(tbe, xs, ids, ts, gl, 2.0, "f16", "bf16", False)


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [37, 3001, 20011, 140003])
def test_distill_far_values(x, V):
    """Rows all negative, far below and above zero, with masks of the lowest
    value in whole parts, and NaN beside such masks."""
    say("distill far values", x, V)
    tbe = lib()
    N, K, tau = 14, 5, 0.7
    xs, ids, ts, gl = distill_case(gen(V), N, V, K, x, "f32", True, 0.0)
    ids = torch.stack([torch.randperm(V, generator=gen(n))[:K] for n in range(N)]).cuda()
    low = torch.finfo(DT[x]).min
    keep = torch.zeros(N, V, dtype=torch.bool, device="cuda").scatter_(1, ids, True)
    at = ids[:, 0]
    xs[0] = xs[0] * 0.1 - 30                       # all negative
    xs[1] = xs[1] * 0.1 - 3000
    xs[2] = xs[2] * 0.1 + 3000
    xs[3, V // 3:] = low                           # masked from a third on
    xs[4, :V // 2] = low
    xs[5] = torch.where(keep[5], -40000.0, low)    # a maximum far below zero
    xs[6] = low
    if x != "f16":
        xs[7] = torch.where(keep[7], 1e30, 0.0)    # far above: only the places count
        xs[8] = -1e30
        # |a max| around 2^23 and 2^24, where a row and a thread become far
        xs[9] = -2.0 ** 24 * tau * math.log(2) * (1 + torch.rand(V, generator=gen(9)).cuda() * 2 ** -8)
        xs[10] = -2.0 ** 23 * tau * math.log(2) * (1 + torch.rand(V, generator=gen(10)).cuda() * 2 ** -8)
    nan_rows = torch.zeros(N, dtype=torch.bool, device="cuda")
    nan_rows[11:14] = True
    xs[11] = low
    xs[11, V // 2] = float("nan")
    xs[12, V - 1] = -float("nan")
    xs[13, 1] = math.inf
    desc = tbe.DistillDesc(N, V, K, dtype=x, temperature=tau)
    want_l, want_g, bl, bg = distill_ref(xs, ids, ts, tau, gl)
    outs = run_distill(tbe, desc, xs, ids, ts, gl)
    fine = ~nan_rows
    for loss, grad in (outs[:2], outs[2:]):
        assert torch.isnan(loss[nan_rows]).all() and torch.isnan(grad[nan_rows]).all()
        close(loss[fine], want_l[fine], bl[fine], "f32", "loss")
        close(grad[fine], want_g[fine], bg[fine], x, "gradient")


def test_distill_rows_without_a_teacher_are_marked_by_their_statistics():
    tbe = lib()
    xs, ids, ts, gl = distill_case(gen(3), 6, 900, 4, "f32", "f32", True, 0.0)
    ids[2] = -1
    ids[4] = 900
    stats = torch.full((6, 2), float("nan"), device="cuda")
    loss = torch.empty(6, device="cuda")
    desc = tbe.DistillDesc(6, 900, 4, dtype="f32")
    tbe.tbe_distill_forward(desc, xs, ids, ts, loss, stats, tbe.distill_workspace(desc))
    assert (stats[[2, 4]] == 0).all() and (loss[[2, 4]] == 0).all()
    rest = [0, 1, 3, 5]
    some = ((ids[rest] >= 0) & (ids[rest] < 900)).any(1)
    assert torch.equal(stats[rest][some][:, 0], xs[rest].amax(1)[some])


@pytest.mark.parametrize("x", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [65, 515, 1027, 9001, 70003])
@pytest.mark.parametrize("first", [0, 1, 2, 3, 7])
def test_distill_alignments(x, V, first):
    """Logits and gradient that start at different elements of 16 bytes, rows of
    an odd and of an aligned length; the elements around them stay. The first and
    last places have a teacher's entry."""
    say("distill alignments", x, V, first)
    tbe = lib()
    for N in (9, 300 if V < 9001 else 20):
        xs, ids, ts, gl = distill_case(gen(V + first), N, V, 6, x, "f32", True, 0.2)
        ids[0, :4] = torch.tensor([0, V - 1, 7, V - 8])
        want_l, want_g, bl, bg = distill_ref(xs, ids, ts, 1.0, gl)
        desc = tbe.DistillDesc(N, V, 6, dtype=x)
        for pad in (1, 16):
            wide = torch.full((N, V + 7 + pad), float("nan"), dtype=DT[x], device="cuda")
            inp = wide[:, first:first + V]
            inp.copy_(xs)
            out = torch.full((N, V + 8), float("nan"), dtype=DT[x], device="cuda")
            grad = out[:, 3:3 + V]
            loss, stats = torch.empty(N, device="cuda"), torch.empty(N, 2, device="cuda")
            ws = tbe.distill_workspace(desc)

            def check():
                close(loss, want_l, bl, "f32", "loss")
                close(grad, want_g, bg, x, "gradient")
                assert torch.isnan(out[:, :3]).all() and torch.isnan(out[:, 3 + V:]).all()
                out.fill_(float("nan"))
            tbe.tbe_distill_step(desc, inp, ids, ts, gl, loss, grad, ws)
            check()
            tbe.tbe_distill_forward(desc, inp, ids, ts, loss, stats, ws)
            tbe.tbe_distill_backward(desc, inp, ids, ts, stats, gl, grad)
            check()
            tbe.tbe_distill_backward(desc, inp, ids, ts, stats, gl, inp)   # in place
            close(inp, want_g, bg, x, "gradient in place")
            rest = torch.ones(V + 7 + pad, dtype=torch.bool, device="cuda")
            rest[first:first + V] = False
            assert torch.isnan(wide[:, rest]).all()


# --- token table -----------------------------------------------------------------------
# few tokens without a sort (up to 2048, fewer of wide rows), one launch's sort
# (up to 4096), three beyond; tables whose rows and spans of 1024 vectors end apart
TOKEN = [(N, V, D, w, x, dist) for N in (1, 2, 512, 513, 1023, 1024, 1025, 2048, 2049) for (V, D, w, x) in
         [(97, 1030, "f32", "f16"), (5000, 8, "bf16", "bf16"), (1, 700, "f16", "f32")]
         for dist in ("same", "square")] + [
    (1024, 50, 4100, "bf16", "f32", "few"),     # 17 segments: over the few tokens' limit
    (737, 50, 4100, "bf16", "f32", "square"),   # just under
    (738, 50, 4100, "bf16", "f32", "square"),
    (4096, 1023 * 1024, 9, "bf16", "bf16", "square"),
    (4097, 1023 * 1024, 9, "f16", "f32", "square"),
    (4096, 700, 260, "f32", "f32", "same"),
    (4097, 700, 260, "f32", "f32", "same"),
    (70000, 1025, 100, "bf16", "bf16", "same"),  # one id: 2188 pieces to join
    (70000, 3000, 520, "bf16", "f16", "few"),
    (33000, 1100, 1, "f32", "bf16", "uniform"),  # runs about as long as a chunk
    (33000, 1100, 513, "f32", "f32", "uniform"),
]


@pytest.mark.parametrize("N,V,D,w,x,dist", TOKEN)
def test_token_borders(N, V, D, w, x, dist):
    say("token borders", N, V, D, w, x, dist)
    tbe = lib()
    g = gen(N + V + D)
    idx = torch.int32
    ids = token_ids(g, N, V, idx, dist, 0.1 if N > 2 else 0)
    desc = tbe.TokenDesc(N, V, D, wdtype=w, xdtype=x, idx64=False, scale=0.5)
    ok = (ids >= 0) & (ids < V)
    at = torch.where(ok, ids.long(), 0)
    grad = randn(g, N, D).to(DT[x])
    grad[~ok] = float("nan")            # a padded token's row is not read
    g64 = torch.where(ok[:, None], grad.to(F64), 0.0)
    want = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, at, g64) * 0.5
    size = torch.zeros(V, D, dtype=F64, device="cuda").index_add_(0, at, g64.abs()) * 0.5
    count = torch.zeros(V, dtype=F64, device="cuda").index_add_(0, at, ok.to(F64))
    for stride in (0, 3):
        gW = new(V, D, DT[w], stride)
        ws = tbe.token_workspace(desc)
        ws.fill_(0xFF)
        tbe.tbe_token_backward(desc, view_of(grad, stride), ids, gW, ws)
        close(gW, want, (count[:, None] + 2) * U32 * size, w, "backward")
        if stride:
            base = gW._base
            assert torch.isnan(base[:, :1]).all() and torch.isnan(base[:, 1 + D:]).all()
