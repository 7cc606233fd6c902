"""A small language model distilled from a teacher's top logits, end to end on
the library's token, expert and distillation operators:

    python examples/lm_distill.py [steps] [--gated]

Each token's row is looked up, sent to K of E experts and back with weights,
and projected on the vocabulary; the loss against the teacher's K' logits gives
the gradient of the logits, which goes back through the same operators to the
table, the experts and the router. The products between them are torch's. With
--gated the experts are gated feed-forward blocks on normed rows, and layer norm,
the experts' products and the optimizer's step are the library's too: no step waits
for the host. Then one sequence is continued token by token.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bwd_tbe_pooled_amd as tbe  # noqa: E402


class Model:
    """Embedding, one layer of experts (D x D matrices) and an output matrix."""

    def __init__(self, V, D, E, K, seed=0):
        self.V, self.D, self.E, self.K = V, D, E, K
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def randn(*shape, scale):
            return torch.randn(shape, generator=g, device="cuda") * scale
        self.scale = math.sqrt(D)
        self.params = {"table": randn(V, D, scale=1 / D), "router": randn(D, E, scale=D ** -0.5),
                       "experts": randn(E, D, D, scale=D ** -0.5), "out": randn(D, V, scale=D ** -0.5)}

    def buffers(self, N):
        """Descriptions, plan and workspaces for N tokens: made once, kept by the program."""
        b = {"token": tbe.TokenDesc(N, self.V, self.D, wdtype="f32", xdtype="f32", scale=self.scale),
             "expert": tbe.ExpertDesc(N, self.K, self.E, self.D, dtype="f32")}
        b["plan"] = tbe.ExpertPlan(b["expert"])
        b["token_ws"] = tbe.token_workspace(b["token"])
        b["expert_ws"] = tbe.expert_workspace(b["expert"])
        return b

    def _experts(self, rows, offsets, weights):
        out = torch.zeros_like(rows)
        for e, (a, z) in enumerate(zip(offsets[:-1], offsets[1:])):
            if z > a:
                out[a:z] = rows[a:z] @ weights[e]
        return out

    def forward(self, ids, b):
        """Logits [N, V] and what the backward needs."""
        p, N, M = self.params, ids.numel(), ids.numel() * self.K
        s = {"ids": ids}
        s["h"] = torch.empty(N, self.D, device="cuda")
        tbe.tbe_token_forward(b["token"], p["table"], ids, s["h"])
        top, choice = torch.topk(s["h"] @ p["router"], self.K, dim=1)
        s["choice"], s["w"] = choice, torch.softmax(top, dim=1)
        plan = b["plan"]
        tbe.tbe_expert_plan(b["expert"], choice, plan, b["expert_ws"])
        s["offsets"] = plan.offsets.tolist()
        s["xs"] = torch.empty(M, self.D, device="cuda")
        tbe.tbe_expert_dispatch(b["expert"], s["h"], plan.slots, s["xs"])
        s["ys"] = self._experts(s["xs"], s["offsets"], p["experts"])
        s["y"] = torch.empty(N, self.D, device="cuda")
        tbe.tbe_expert_combine(b["expert"], s["ys"], plan.slots, s["w"], s["y"])
        s["z"] = s["h"] + s["y"]
        return s["z"] @ p["out"], s

    def backward(self, dlogits, s, b):
        """Gradients of all parameters."""
        p, plan, D = self.params, b["plan"], self.D
        grads = {"out": s["z"].t() @ dlogits}
        dz = dlogits @ p["out"].t()
        dys, dw = torch.empty_like(s["ys"]), torch.empty_like(s["w"])
        tbe.tbe_expert_combine_backward(b["expert"], dz, s["ys"], plan.slots, s["w"], dys, dw)
        grads["experts"] = torch.zeros_like(p["experts"])
        dxs = torch.zeros_like(dys)
        for e, (a, z) in enumerate(zip(s["offsets"][:-1], s["offsets"][1:])):
            if z > a:
                grads["experts"][e] = s["xs"][a:z].t() @ dys[a:z]
                dxs[a:z] = dys[a:z] @ p["experts"][e].t()
        dh = torch.empty_like(dz)
        tbe.tbe_expert_dispatch_backward(b["expert"], dxs, plan.slots, dh)
        dh += dz
        dscore = s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True))   # of the softmax over the chosen
        droute = torch.zeros(s["ids"].numel(), self.E, device="cuda").scatter_(1, s["choice"], dscore)
        grads["router"] = s["h"].t() @ droute
        dh += droute @ p["router"].t()
        grads["table"] = torch.empty_like(p["table"])
        tbe.tbe_token_backward(b["token"], dh, s["ids"], grads["table"], b["token_ws"])
        return grads


class GatedModel(Model):
    """The same with a layer norm before the experts, which are gated feed-forward blocks
    of F columns."""

    def __init__(self, V, D, E, K, F, seed=0):
        super().__init__(V, D, E, K, seed)
        self.F = F
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 100)
        del self.params["experts"]
        self.params["norm_w"], self.params["norm_b"] = torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")
        for name, shape in (("gate", (E, F, D)), ("up", (E, F, D)), ("down", (E, D, F))):
            self.params[name] = torch.randn(shape, generator=g, device="cuda") * shape[2] ** -0.5

    def buffers(self, N):
        b = super().buffers(N)
        b["norm"] = tbe.NormDesc(N, self.D, dtype="f32", wdtype="f32")
        b["ffn"] = tbe.FfnDesc(N * self.K, self.E, self.D, self.F, dtype="f32")
        b["norm_ws"], b["ffn_ws"] = tbe.norm_workspace(b["norm"]), tbe.ffn_workspace(b["ffn"])
        return b

    def forward(self, ids, b):
        p, N, M = self.params, ids.numel(), ids.numel() * self.K

        def new(*shape):
            return torch.empty(*shape, device="cuda")
        s = {"ids": ids, "h": new(N, self.D), "x": new(N, self.D), "stats": new(N, 2)}
        tbe.tbe_token_forward(b["token"], p["table"], ids, s["h"])
        tbe.tbe_norm_forward(b["norm"], s["h"], p["norm_w"], p["norm_b"], s["x"], s["stats"])
        top, choice = torch.topk(s["x"] @ p["router"], self.K, dim=1)
        s["choice"], s["w"] = choice, torch.softmax(top, dim=1)
        plan = b["plan"]
        tbe.tbe_expert_plan(b["expert"], choice, plan, b["expert_ws"])
        s["xs"], s["ys"], s["pre"] = new(M, self.D), new(M, self.D), new(M, 2 * self.F)
        tbe.tbe_expert_dispatch(b["expert"], s["x"], plan.slots, s["xs"])
        tbe.tbe_ffn_forward(b["ffn"], s["xs"], plan.offsets, p["gate"], p["up"], p["down"], s["pre"], s["ys"],
                            b["ffn_ws"])
        s["y"] = new(N, self.D)
        tbe.tbe_expert_combine(b["expert"], s["ys"], plan.slots, s["w"], s["y"])
        s["z"] = s["h"] + s["y"]
        return s["z"] @ p["out"], s

    def backward(self, dlogits, s, b):
        p, plan = self.params, b["plan"]
        grads = {k: torch.empty_like(v) for k, v in p.items()}
        grads["out"] = s["z"].t() @ dlogits
        dz = dlogits @ p["out"].t()
        dys, dw, dxs = torch.empty_like(s["ys"]), torch.empty_like(s["w"]), torch.empty_like(s["xs"])
        tbe.tbe_expert_combine_backward(b["expert"], dz, s["ys"], plan.slots, s["w"], dys, dw)
        tbe.tbe_ffn_backward(b["ffn"], dys, s["xs"], plan.offsets, p["gate"], p["up"], p["down"], s["pre"], dxs,
                             grads["gate"], grads["up"], grads["down"], b["ffn_ws"])
        dx, dh = torch.empty_like(dz), torch.empty_like(dz)
        tbe.tbe_expert_dispatch_backward(b["expert"], dxs, plan.slots, dx)
        dscore = s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True))
        droute = torch.zeros(s["ids"].numel(), self.E, device="cuda").scatter_(1, s["choice"], dscore)
        grads["router"] = s["x"].t() @ droute
        dx += droute @ p["router"].t()
        tbe.tbe_norm_backward(b["norm"], dx, s["h"], p["norm_w"], s["stats"], dh, grads["norm_w"], grads["norm_b"],
                              b["norm_ws"])
        dh += dz
        tbe.tbe_token_backward(b["token"], dh, s["ids"], grads["table"], b["token_ws"])
        return grads


def train_gated(steps=60, N=512, V=2003, D=64, E=8, K=2, F=96, top=16, tau=2.0, lr=3e-3, bits=32):
    """Losses of the steps of a gated model under AdamW, moments in `bits` bits."""
    teacher, student = GatedModel(V, D, E, K, F, seed=1), GatedModel(V, D, E, K, F, seed=2)
    teacher.params["out"] *= 4
    b, tb = student.buffers(N), teacher.buffers(N)
    dd = tbe.DistillDesc(N, V, top, dtype="f32", temperature=tau)
    ws = tbe.distill_workspace(dd)
    loss, gl = torch.empty(N, device="cuda"), torch.full((N,), 1.0 / N, device="cuda")
    ad = tbe.AdamWDesc(pdtype="f32", gdtype="f32", bits=bits, weight_decay=0.0)
    params = list(student.params.values())
    state = tbe.AdamWState(ad, params)
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    rate = torch.full((1,), lr, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    losses = []
    for _ in range(steps):
        ids = (torch.rand(N, generator=g, device="cuda") ** 3 * V).long()
        t, places = torch.topk(teacher.forward(ids, tb)[0], top, dim=1)
        logits, saved = student.forward(ids, b)
        tbe.tbe_distill_step(dd, logits, places, t.contiguous(), gl, loss, logits, ws)
        losses.append(loss.mean())
        grads = student.backward(logits, saved, b)
        step += 1
        tbe.tbe_adamw_step(ad, params, [grads[k] for k in student.params], state, step, rate)
    return torch.stack(losses).tolist(), student


def train(steps=60, N=512, V=2003, D=64, E=8, K=2, top=16, tau=2.0, lr=0.05):
    """Losses of the steps. The teacher is a fixed random model."""
    teacher, student = Model(V, D, E, K, seed=1), Model(V, D, E, K, seed=2)
    teacher.params["out"] *= 4
    b, tb = student.buffers(N), teacher.buffers(N)
    dd = tbe.DistillDesc(N, V, top, dtype="f32", temperature=tau)
    ws = tbe.distill_workspace(dd)
    loss = torch.empty(N, device="cuda")
    gl = torch.full((N,), 1.0 / N, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    squares = {k: torch.zeros_like(v) for k, v in student.params.items()}
    losses = []
    for _ in range(steps):
        ids = (torch.rand(N, generator=g, device="cuda") ** 3 * V).long()
        t, places = torch.topk(teacher.forward(ids, tb)[0], top, dim=1)
        logits, state = student.forward(ids, b)
        # loss and gradient in one call; the gradient takes the logits' place
        tbe.tbe_distill_step(dd, logits, places, t.contiguous(), gl, loss, logits, ws)
        losses.append(loss.mean().item())
        for k, grad in student.backward(logits, state, b).items():   # Adagrad
            squares[k].addcmul_(grad, grad)
            student.params[k] -= lr * grad / (squares[k].sqrt() + 1e-8)
    return losses, student


def generate(model, first=1, length=8):
    """Greedy continuation, one token a step."""
    b = model.buffers(1)
    ids = torch.tensor([first], device="cuda")
    out = [first]
    for _ in range(length):
        logits, _ = model.forward(ids, b)
        ids = logits.argmax(1)
        out.append(int(ids))
    return out


if __name__ == "__main__":
    args = [a for a in sys.argv[1:] if a != "--gated"]
    run = train_gated if "--gated" in sys.argv else train
    losses, model = run(int(args[0]) if args else 60)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {len(losses)} steps")
    print("continuation", generate(model))
