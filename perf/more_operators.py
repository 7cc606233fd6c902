"""Cases that measure the operators a model's training step has between the
token, expert and distillation operators of this library.

  norm    layer norm of rows, and the gradients of rows, weight and bias
  ffn     the experts' gated feed-forward products over rows sorted by expert,
          and the gradients of rows and weights
  adamw   one AdamW step over many tensors, moments in 32 or in 8 bits

`run` computes a case in plain torch operations when `own` is false, and
through the library's entry points when it is true.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5          # of the norm
BLOCK = 256         # elements that share a scale of an 8-bit moment
BETA1, BETA2, ADAM_EPS, DECAY = 0.9, 0.95, 1e-8, 0.1


def _norm(name, kind, N, D, x, w):
    return {"name": name, "op": "norm", "kind": kind, "N": N, "D": D, "x": x, "w": w}


def _ffn(name, kind, N, K, E, D, F, x, act, drop):
    return {"name": name, "op": "ffn", "kind": kind, "N": N, "K": K, "E": E, "D": D, "F": F, "x": x,
            "act": act, "drop": drop}


def _adamw(name, V, D, F, E, L, p, g, c, bits, scaled, tight):
    return {"name": name, "op": "adamw", "V": V, "D": D, "F": F, "E": E, "L": L, "p": p, "g": g, "c": c,
            "bits": bits, "scaled": scaled, "tight": tight}


def listed():
    return [
        # one decoding step of a batch of 16 sequences
        _norm("norm_fwd_decode", "fwd", 16, 2048, "bf16", "bf16"),
        # fine-tuning on a few hundred tokens: odd width, f32 weights of an f16 step
        _norm("norm_step_odd", "fwd_bwd", 777, 1030, "f16", "f32"),
        # a training micro-batch, forward and backward
        _norm("norm_step_batch", "fwd_bwd", 16384, 4096, "bf16", "f32"),
        # the gradient over many narrow rows: the weight's gradient is a long sum
        _norm("norm_bwd_rows", "bwd", 262144, 1024, "bf16", "bf16"),
        # one decoding step of a mixture of experts: every weight is read for a row or two
        _ffn("ffn_infer_decode", "infer", 4, 8, 64, 2048, 768, "bf16", "silu", 0.0),
        # a training batch through many small experts, the products before the activation kept
        _ffn("ffn_fwd_batch", "fwd", 16384, 8, 128, 2048, 768, "bf16", "silu", 0.0),
        # its gradient with fewer, wider experts and assignments dropped at capacity
        _ffn("ffn_bwd_batch", "bwd", 8192, 4, 32, 4096, 1536, "bf16", "silu", 0.05),
        # odd widths in 32 bits: a small model under test
        _ffn("ffn_bwd_odd", "bwd", 333, 2, 8, 1001, 515, "f32", "gelu", 0.1),
        # the parameters of a small model in 32 bits throughout
        _adamw("adamw_small", 2003, 64, 64, 8, 1, "f32", "f32", "none", 32, False, False),
        # adapters: hundreds of small tensors of odd sizes, packed without gaps
        _adamw("adamw_many_8bit", 1009, 129, 33, 2, 48, "f32", "f16", "f16", 8, True, True),
        # a mixture of experts trained with 32-bit parameters beside the 16-bit ones it computes with
        _adamw("adamw_mixed", 32000, 2048, 768, 16, 3, "f32", "bf16", "bf16", 32, False, False),
        # a large vocabulary where memory counts: 16-bit parameters, moments in 8 bits
        _adamw("adamw_8bit", 131072, 2048, 8192, 1, 4, "bf16", "bf16", "none", 8, False, False),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _width(rng, lo, hi):
    """A width, more often a multiple of 64 than not."""
    D = _logint(rng, lo, hi)
    return max(64, D // 64 * 64) if rng.random() < 0.6 else D


def draw(rng):
    op = rng.choice(["norm", "norm", "ffn", "ffn", "ffn", "adamw", "adamw"])
    x = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "norm":
        D = _width(rng, 64, 8192)
        return {"op": op, "kind": rng.choice(["fwd", "bwd", "fwd_bwd"]),
                "N": max(1, min(_logint(rng, 1, 262144), 500000000 // (D * SIZE[x]))), "D": D, "x": x,
                "w": rng.choice([x, "f32"])}
    if op == "ffn":
        kind = rng.choice(["infer", "fwd", "bwd"])
        D, F, E = _width(rng, 64, 4096), _width(rng, 64, 4096), _logint(rng, 1, 128)
        E = max(1, min(E, 3000000000 // (3 * D * F * SIZE[x])))
        K = rng.randint(1, min(E, 8))
        work = D * F * K * (12 if kind == "bwd" else 6) * (8 if x == "f32" else 1)
        N = max(1, min(_logint(rng, 1, 32768), 2200000000000 // work))
        return {"op": op, "kind": kind, "N": N, "K": K, "E": E, "D": D, "F": F, "x": x,
                "act": rng.choice(["silu", "silu", "gelu"]), "drop": rng.choice([0.0, 0.0, 0.1])}
    p = rng.choice(["f32", "f32", "bf16", "f16"])
    g = rng.choice(["f32", "bf16", "f16"]) if p == "f32" else p
    D, E, L = _width(rng, 64, 4096), _logint(rng, 1, 16), _logint(rng, 1, 48)
    F = max(8, _logint(rng, 32, 4096) // E)
    V = _logint(rng, 100, 131072)
    V = max(100, min(V, 150000000 // D))
    L = max(1, min(L, 250000000 // (3 * E * D * F)))
    return {"op": op, "V": V, "D": D, "F": F, "E": E, "L": L, "p": p, "g": g,
            "c": g if p == "f32" and g != "f32" and rng.random() < 0.6 else "none",
            "bits": rng.choice([32, 8]), "scaled": rng.random() < 0.4, "tight": rng.random() < 0.3}


# --- inputs -------------------------------------------------------------------
def _shapes(case):
    """Shapes of the parameters of a small model of L layers of experts."""
    V, D, F, E = case["V"], case["D"], case["F"], case["E"]
    layer = [(D,), (D,), (D, E), (E, F, D), (E, F, D), (E, D, F)]
    return [(V, D)] + layer * case["L"] + [(D, V)]


def _starts(case, unit):
    """Each tensor's first element in a flat buffer whose tensors begin at
    multiples of `unit`, and the buffer's length."""
    starts, at = [], 0
    for s in _shapes(case):
        starts.append(at)
        at += -(-math.prod(s) // unit) * unit
    return starts, at


def _views(flat, case, unit):
    return [flat[a:a + math.prod(s)].view(s) for a, s in zip(_starts(case, unit)[0], _shapes(case))]


def _inputs(case, seed):
    """The case's input tensors on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)

    def rand(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    st = {}
    if case["op"] == "norm":
        N, D, x, w = case["N"], case["D"], DT[case["x"]], DT[case["w"]]
        # rows of a residual stream: each of its own size and offset, a few columns far larger
        col = torch.where(rand(D) < 0.01, 8.0, 1.0)
        rows = randn(N, D) * col * (0.5 + 3.0 * rand(N, 1)) + randn(N, 1)
        st["x"] = rows.to(x)
        st["w"], st["b"] = (1.0 + randn(D, std=0.2)).to(w), randn(D, std=0.2).to(w)
        if case["kind"] != "fwd":
            st["dy"] = randn(N, D, std=0.05, dtype=x)
        return st
    if case["op"] == "ffn":
        N, K, E, D, F, dt = (case[k] for k in "N K E D F x".split())
        dt = DT[dt]
        ids = torch.topk(randn(N, E) + 0.5 * randn(E), K, dim=1).indices
        ids = torch.where(rand(N, K) < case["drop"], E, ids)
        counts = torch.bincount(ids.reshape(-1), minlength=E + 1)
        offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        offsets[1:] = torch.cumsum(counts, 0)[:E]
        st["offsets"] = offsets
        st["xs"] = randn(N * K, D, dtype=dt)
        st["gate"], st["up"] = randn(E, F, D, std=D ** -0.5, dtype=dt), randn(E, F, D, std=D ** -0.5, dtype=dt)
        st["down"] = randn(E, D, F, std=F ** -0.5, dtype=dt)
        if case["kind"] == "bwd":
            # gradients of a mean over the tokens under a loss scale
            st["dys"] = randn(N * K, D, std=0.05, dtype=dt)
        return st
    unit = 1 if case["tight"] else BLOCK
    n = _starts(case, unit)[1]
    blocks = _starts(case, BLOCK)[1]
    p, gt = DT[case["p"]], DT[case["g"]]
    st["p"] = randn(n, std=0.05, dtype=p)
    up = 1024.0 if case["scaled"] else 1.0
    # a gradient: most elements small, their size differing from place to place
    st["g"] = (randn(n, std=1e-3 * up) * torch.exp(1.5 * randn(n))).to(gt)
    m = torch.zeros(blocks, device="cuda")
    v = torch.zeros(blocks, device="cuda")
    for dst, src in zip(_views(m, case, BLOCK), _views(st["g"], case, unit)):
        dst.copy_(src)
    # moments as they are after many steps of gradients of that size
    v.copy_((m / up).square_().mul_(0.3 + rand(blocks)))
    m.mul_(0.3 / up).add_(torch.sqrt(v) * randn(blocks, std=0.2))
    if case["bits"] == 8:
        st["m"], st["ms"] = _quantized(m)
        st["v"], st["vs"] = _quantized(torch.sqrt_(v))
    else:
        st["m"], st["v"] = m, v
    st["step"] = torch.full((1,), 400 + seed % 100, dtype=torch.int64, device="cuda")
    st["lr"] = torch.full((1,), 3e-4, device="cuda")
    st["scale"] = torch.full((1,), 1.0 / up, device="cuda") if case["scaled"] else None
    return st


def _quantized(x, least=False):
    """x (whole blocks) as e4m3 numbers and a scale for each block, whose
    largest magnitude becomes 448. `least`: what is above zero stays above it."""
    x = x.view(-1, BLOCK)
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top < 2.0 ** -100, 0.0, top / 448.0)
    q = torch.where(scale > 0, x / scale, 0.0)
    if least:
        q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    return q.to(torch.float8_e4m3fn).view(-1), scale.view(-1)


def prepare(case, seed):
    st = _inputs(case, seed)
    st["case"] = case

    def new(like):
        return torch.empty_like(like)

    kind = case.get("kind")
    if case["op"] == "norm":
        if kind == "bwd":
            st["stats"] = _norm_stats(st["x"].float())
        else:
            st["y"], st["stats"] = new(st["x"]), torch.empty(case["N"], 2, device="cuda")
        if kind != "fwd":
            st["dx"], st["dw"], st["db"] = new(st["x"]), new(st["w"]), new(st["b"])
    elif case["op"] == "ffn":
        # rows of dropped assignments, behind the last expert's, are left as they are
        if kind == "bwd":
            M, F = case["N"] * case["K"], case["F"]
            st["pre"] = torch.zeros(M, 2 * F, dtype=DT[case["x"]], device="cuda")
            for e, rows in _experts(st["offsets"]):
                x = st["xs"][rows].float()
                st["pre"][rows, :F] = (x @ st["gate"][e].float().t()).to(st["pre"].dtype)
                st["pre"][rows, F:] = (x @ st["up"][e].float().t()).to(st["pre"].dtype)
            st["dxs"] = torch.zeros_like(st["xs"])
            st["dgate"], st["dup"], st["ddown"] = new(st["gate"]), new(st["up"]), new(st["down"])
        else:
            st["ys"] = torch.zeros_like(st["xs"])
            st["pre"] = (torch.zeros(case["N"] * case["K"], 2 * case["F"], dtype=st["xs"].dtype, device="cuda")
                         if kind == "fwd" else None)
    else:
        unit = 1 if case["tight"] else BLOCK
        for k in ("p", "g"):
            st[k + "_list"] = _views(st[k], case, unit)
        st["c"] = None if case["c"] == "none" else torch.zeros(st["p"].shape, dtype=DT[case["c"]], device="cuda")
        st["c_list"] = None if st["c"] is None else _views(st["c"], case, unit)
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """Descriptions, workspaces and the optimizer's state: what a program makes once."""
    import bwd_tbe_pooled_amd as tbe
    case = st["case"]
    if case["op"] == "norm":
        st["desc"] = tbe.NormDesc(case["N"], case["D"], dtype=case["x"], wdtype=case["w"], eps=EPS)
        st["ws"] = tbe.norm_workspace(st["desc"])
    elif case["op"] == "ffn":
        st["desc"] = tbe.FfnDesc(case["N"] * case["K"], case["E"], case["D"], case["F"], dtype=case["x"],
                                 act=case["act"])
        st["ws"] = tbe.ffn_workspace(st["desc"])
    else:
        st["desc"] = tbe.AdamWDesc(pdtype=case["p"], gdtype=case["g"],
                                   cdtype=None if case["c"] == "none" else case["c"], bits=case["bits"],
                                   beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, weight_decay=DECAY)
        st["state"] = tbe.AdamWState(st["desc"], st["p_list"])
        for k in ("m", "v", "ms", "vs"):   # flat buffers, tensors at multiples of the block
            if k in st:
                flat = getattr(st["state"], k + "_flat")
                flat.copy_(st[k])
                st[k] = flat


# --- one pass -----------------------------------------------------------------
def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import bwd_tbe_pooled_amd as tbe
    case, d = st["case"], st["desc"]
    kind = case.get("kind")
    if case["op"] == "norm":
        if kind != "bwd":
            tbe.tbe_norm_forward(d, st["x"], st["w"], st["b"], st["y"], st["stats"])
            if kind == "fwd":
                return st["y"], st["stats"]
        tbe.tbe_norm_backward(d, st["dy"], st["x"], st["w"], st["stats"], st["dx"], st["dw"], st["db"],
                              st["ws"])
        return (st["y"] if kind == "fwd_bwd" else None), st["dx"], st["dw"], st["db"]
    if case["op"] == "ffn":
        if kind == "bwd":
            tbe.tbe_ffn_backward(d, st["dys"], st["xs"], st["offsets"], st["gate"], st["up"], st["down"],
                                 st["pre"], st["dxs"], st["dgate"], st["dup"], st["ddown"], st["ws"])
            return st["dxs"], st["dgate"], st["dup"], st["ddown"]
        tbe.tbe_ffn_forward(d, st["xs"], st["offsets"], st["gate"], st["up"], st["down"], st["pre"],
                            st["ys"], st["ws"])
        return st["ys"], st["pre"]
    tbe.tbe_adamw_step(d, st["p_list"], st["g_list"], st["state"], st["step"], st["lr"], st["scale"],
                       st["c_list"])
    return {k: st[k] for k in ("p", "c", "m", "v", "ms", "vs") if st.get(k) is not None}


def _norm_stats(x):
    mu = x.mean(1)
    var = (x - mu[:, None]).square().mean(1)
    return torch.stack([mu, torch.rsqrt(var + EPS)], 1)


def _experts(offsets):
    """(expert, its rows) of the experts that have rows."""
    o = offsets.tolist()
    return [(e, slice(a, z)) for e, (a, z) in enumerate(zip(o[:-1], o[1:])) if z > a]


def _act(name, g):
    """The activation and its derivative."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1.0 + g * (1.0 - s))
    cdf = 0.5 * (1.0 + torch.erf(g * 2.0 ** -0.5))
    return g * cdf, cdf + g * torch.exp(-0.5 * g * g) * (2.0 * math.pi) ** -0.5


def _run_plain(st):
    case = st["case"]
    kind = case.get("kind")
    if case["op"] == "norm":
        x, w = st["x"].float(), st["w"].float()
        if kind != "bwd":
            st["stats"] = _norm_stats(x)
        mu, r = st["stats"][:, :1], st["stats"][:, 1:]
        xh = (x - mu) * r
        y = (xh * w + st["b"].float()).to(st["x"].dtype) if kind != "bwd" else None
        if kind == "fwd":
            return y, st["stats"]
        dy = st["dy"].float()
        a = dy * w
        s1, s2 = a.mean(1, keepdim=True), (a * xh).mean(1, keepdim=True)
        dx = (r * (a - s1 - xh * s2)).to(st["x"].dtype)
        return y, dx, (dy * xh).sum(0).to(st["w"].dtype), dy.sum(0).to(st["w"].dtype)
    if case["op"] == "ffn":
        return _ffn_plain(st)
    return _adamw_plain(st)


def _ffn_plain(st):
    case, F, dt = st["case"], st["case"]["F"], st["xs"].dtype
    if case["kind"] != "bwd":
        for e, rows in _experts(st["offsets"]):
            x = st["xs"][rows].float()
            g, u = x @ st["gate"][e].float().t(), x @ st["up"][e].float().t()
            st["ys"][rows] = ((_act(case["act"], g)[0] * u) @ st["down"][e].float().t()).to(dt)
            if st["pre"] is not None:
                st["pre"][rows, :F], st["pre"][rows, F:] = g.to(dt), u.to(dt)
        return st["ys"], st["pre"]
    for k in ("dgate", "dup", "ddown"):
        st[k].zero_()
    for e, rows in _experts(st["offsets"]):
        x, dy = st["xs"][rows].float(), st["dys"][rows].float()
        g, u = st["pre"][rows, :F].float(), st["pre"][rows, F:].float()
        a, da = _act(case["act"], g)
        dh = dy @ st["down"][e].float()
        dg, du = dh * u * da, dh * a
        st["dxs"][rows] = (dg @ st["gate"][e].float() + du @ st["up"][e].float()).to(dt)
        st["dgate"][e], st["dup"][e] = (dg.t() @ x).to(dt), (du.t() @ x).to(dt)
        st["ddown"][e] = (dy.t() @ (a * u)).to(dt)
    return st["dxs"], st["dgate"], st["dup"], st["ddown"]


def _adamw_plain(st):
    case = st["case"]
    bits8 = case["bits"] == 8
    t = st["step"].double()
    c1, c2 = (1.0 - BETA1 ** t).float(), (1.0 - BETA2 ** t).float()
    starts = _starts(case, BLOCK)[0]
    for i, (p, g, at) in enumerate(zip(st["p_list"], st["g_list"], starts)):
        n = p.numel()
        pad = -(-n // BLOCK) * BLOCK
        g = g.reshape(-1).float()
        if st["scale"] is not None:
            g = g * st["scale"]
        if bits8:
            blocks = slice(at // BLOCK, (at + pad) // BLOCK)
            m = (st["m"][at:at + pad].float().view(-1, BLOCK) * st["ms"][blocks, None]).view(-1)
            v = (st["v"][at:at + pad].float().view(-1, BLOCK) * st["vs"][blocks, None]).view(-1).square()
            g = torch.nn.functional.pad(g, (0, pad - n))
        else:
            m, v = st["m"][at:at + n], st["v"][at:at + n]
        m = BETA1 * m + (1.0 - BETA1) * g
        v = BETA2 * v + (1.0 - BETA2) * g * g
        root = torch.sqrt(v)
        x = p.reshape(-1).float()
        move = (m / c1) / (root / torch.sqrt(c2) + ADAM_EPS)
        x = x - st["lr"] * DECAY * x - st["lr"] * move[:n]
        p.copy_(x.view(p.shape))
        if st["c"] is not None:
            st["c_list"][i].copy_(x.view(p.shape))
        if bits8:
            st["m"][at:at + pad], st["ms"][blocks] = _quantized(m)
            st["v"][at:at + pad], st["vs"][blocks] = _quantized(root, least=True)
        else:
            st["m"][at:at + n], st["v"][at:at + n] = m, v
    return {k: st[k] for k in ("p", "c", "m", "v", "ms", "vs") if st.get(k) is not None}


# --- cost and exact values ------------------------------------------------------
def work(case):
    if case["op"] == "norm":
        n, b = case["N"] * case["D"], SIZE[case["x"]]
        passes = {"fwd": 2, "bwd": 3, "fwd_bwd": 5}[case["kind"]]
        return {"bytes": passes * n * b + 4 * case["D"] * SIZE[case["w"]] + 8 * case["N"],
                "flops": {"fwd": 8, "bwd": 14, "fwd_bwd": 22}[case["kind"]] * n}
    if case["op"] == "ffn":
        M, E, D, F, b = case["N"] * case["K"], case["E"], case["D"], case["F"], SIZE[case["x"]]
        m = M * (1.0 - case["drop"])
        used = E * (1.0 - (1.0 - min(1.0, case["K"] * (1.0 - case["drop"]) / E)) ** case["N"])
        weights = 3 * D * F * b
        if case["kind"] == "bwd":
            return {"bytes": (used + E) * weights + m * (3 * D + 2 * F) * b, "flops": 12 * m * D * F}
        kept = 2 * F if case["kind"] == "fwd" else 0
        return {"bytes": used * weights + m * (2 * D + kept) * b, "flops": 6 * m * D * F}
    n = sum(math.prod(s) for s in _shapes(case))
    each = 2 * SIZE[case["p"]] + SIZE[case["g"]] + (0 if case["c"] == "none" else SIZE[case["c"]])
    each += 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": n * each, "flops": 16 * n}


def exact(case, seed):
    """The outputs of `run` in 64 bits."""
    st = _inputs(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        x = st["x"].to(f64)
        mean = x.sum(dim=1, keepdim=True) / case["D"]
        x -= mean
        inv = 1.0 / torch.sqrt((x * x).sum(dim=1, keepdim=True) / case["D"] + EPS)
        x *= inv
        y = torch.addcmul(st["b"].to(f64), x, st["w"].to(f64)) if case["kind"] != "bwd" else None
        if case["kind"] == "fwd":
            return y, torch.cat([mean, inv], dim=1)
        dy = st["dy"].to(f64)
        db, dw = dy.sum(dim=0), torch.mul(dy, x).sum(dim=0)
        dy *= st["w"].to(f64)
        along = (dy * x).sum(dim=1, keepdim=True) / case["D"]
        dy -= dy.sum(dim=1, keepdim=True) / case["D"]
        dy -= x * along
        return y, dy * inv, dw, db
    if case["op"] == "ffn":
        return _ffn_exact(case, st)
    return _adamw_exact(case, st)


def _ffn_exact(case, st):
    f64, F, dt = torch.float64, case["F"], DT[case["x"]]
    ends = st["offsets"].cpu().numpy()
    xs, gate, up, down = st["xs"], st["gate"], st["up"], st["down"]

    def phi(z):
        """The factor of the activation: its value is z phi(z)."""
        return 1.0 / (1.0 + torch.exp(-z)) if case["act"] == "silu" else torch.special.ndtr(z)

    def dphi(z):
        if case["act"] == "silu":
            return phi(z) * phi(-z)
        return torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)

    out = {}
    if case["kind"] == "bwd":
        out["dxs"] = torch.zeros(xs.shape, dtype=f64, device="cuda")
        for k, w in (("dgate", gate), ("dup", up), ("ddown", down)):
            out[k] = torch.zeros(w.shape, dtype=f64, device="cuda")
    else:
        out["ys"] = torch.zeros(xs.shape, dtype=f64, device="cuda")
        out["pre"] = (torch.zeros((xs.shape[0], 2 * F), dtype=f64, device="cuda")
                      if case["kind"] == "fwd" else None)
    for e in range(case["E"]):
        a, z = int(ends[e]), int(ends[e + 1])
        if a == z:
            continue
        both = torch.cat([gate[e], up[e]]).to(f64)
        x = xs[a:z].to(f64)
        pre = torch.matmul(x, both.T)
        if case["kind"] != "bwd":
            if out["pre"] is not None:
                out["pre"][a:z] = pre
            h = pre[:, :F] * phi(pre[:, :F]) * pre[:, F:]
            out["ys"][a:z] = torch.matmul(h, down[e].to(f64).T)
            continue
        # the kept products as they are stored: from 32 bits, rounded to the type
        low = torch.cat([(xs[a:z].float() @ w.float().t()).to(dt) for w in (gate[e], up[e])], dim=1).to(f64)
        g, u = low[:, :F], low[:, F:]
        dy = st["dys"][a:z].to(f64)
        dh = torch.matmul(dy, down[e].to(f64))
        value = g * phi(g)
        d = torch.cat([dh * u * (phi(g) + g * dphi(g)), dh * value], dim=1)
        out["dxs"][a:z] = torch.matmul(d, both)
        dboth = torch.matmul(d.T, x)
        out["dgate"][e], out["dup"][e] = dboth[:F], dboth[F:]
        out["ddown"][e] = torch.matmul(dy.T, value * u)
    return tuple(out.values())


def _adamw_exact(case, st):
    f64 = torch.float64
    unit = 1 if case["tight"] else BLOCK
    at_p, n = _starts(case, unit)
    at_m, n_m = _starts(case, BLOCK)
    eight = case["bits"] == 8
    out = {"p": st["p"].to(f64)}
    if case["c"] != "none":
        out["c"] = torch.zeros(n, dtype=f64, device="cuda")
    names = ("ms", "vs") if eight else ("m", "v")
    # what a state holds in 8 bits has no value of its own, its blocks' scales have
    out.update({"m": None, "v": None} if eight else {})
    for k in names:
        out[k] = torch.zeros(n_m // BLOCK if eight else n_m, dtype=f64, device="cuda")
    step, lr = int(st["step"]), float(st["lr"])
    unscale = 1.0 if st["scale"] is None else float(st["scale"])
    for shape, a, b in zip(_shapes(case), at_p, at_m):
        k = math.prod(shape)
        g = st["g"][a:a + k].to(f64) * unscale
        if eight:
            rows = -(-k // BLOCK)
            first = b // BLOCK
            m, r = (torch.mul(st[c][b:b + rows * BLOCK].to(f64).view(rows, BLOCK),
                              st[c + "s"][first:first + rows].to(f64).unsqueeze(1)).flatten()[:k]
                    for c in "mv")
            v = r * r
        else:
            m, v = st["m"][b:b + k].to(f64), st["v"][b:b + k].to(f64)
        m = torch.lerp(g, m, BETA1)
        v = torch.lerp(g * g, v, BETA2)
        x = st["p"][a:a + k].to(f64) * (1.0 - lr * DECAY)
        x -= lr * m / (1.0 - BETA1 ** step) / (torch.sqrt(v / (1.0 - BETA2 ** step)) + ADAM_EPS)
        out["p"][a:a + k] = x
        if "c" in out:
            out["c"][a:a + k] = x
        if eight:
            for name, value in (("ms", m.abs()), ("vs", torch.sqrt(v))):
                whole = torch.zeros(rows * BLOCK, dtype=f64, device="cuda")
                whole[:k] = value
                out[name][first:first + rows] = whole.view(rows, BLOCK).amax(1) / 448.0
        else:
            out["m"][b:b + k], out["v"][b:b + k] = m, v
    return {k: out[k] for k in ("p", "c", "m", "v", "ms", "vs") if k in out}
