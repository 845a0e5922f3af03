"""One training loop of an embedding layer with a sparsely gated expert tower on top.

    python examples/expert_tower.py [--steps 30] [--batch 2048] [--rows small]

The embedding layer (26 one-hot tables of width 128 and their dot interaction) hands a row of
128 + 351 features per sample to the tower: a norm and a projection to the residual stream, one
residual block of experts (each sample goes to the two that its router likes best) with a norm on
either side and a gate, and a linear head.  Matrix products are torch's; everything else of the
tower runs in the library: gated_norm, expert_sort, expert_dispatch, expert_combine, their
gradients, and clip_grads over all of the tower's gradients before its Adagrad step.  The
gradient of the tower's input goes back into the embedding layer, which updates its rows itself.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import recommender_model_embedding_gb300 as E  # noqa: E402


class ExpertTower:
    """Parameters, gradients (both dicts of float32 tensors) and the two directions."""

    def __init__(self, width_in: int, hidden: int = 256, experts: int = 8, k: int = 2, inner: int = 256,
                 seed: int = 0, device: str = "cuda"):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        r = lambda *s: (torch.randn(s, generator=g) / s[-2] ** 0.5).to(device)
        one = lambda n: torch.ones(n, device=device)
        self.k, self.experts = k, experts
        self.p = dict(norm_in=one(width_in), w_in=r(width_in, hidden), norm_block=one(hidden),
                      w_router=r(hidden, experts), w_gate=r(hidden, hidden), w1=r(experts, hidden, inner),
                      w2=r(experts, inner, hidden), norm_post=one(hidden), res_scale=0.5 * one(hidden),
                      norm_out=one(hidden), w_head=r(hidden, 1))
        self.g = {name: torch.zeros_like(v) for name, v in self.p.items()}
        self.acc = {name: torch.full_like(v, 0.1) for name, v in self.p.items()}
        self.norm = torch.zeros(1, device=device)

    def forward(self, feats):
        """Logits [B] of the interaction's rows; keeps what the backward needs."""
        p, k, B = self.p, self.k, feats.shape[0]
        s = self.s = {"feats": feats}
        s["h0"] = torch.empty_like(feats)
        E.gated_norm(feats, None, None, s["h0"], w_pre=p["norm_in"])
        x = s["x"] = s["h0"] @ p["w_in"]
        h = s["h"] = torch.empty_like(x)
        E.gated_norm(x, None, None, h, w_pre=p["norm_block"])
        top = (h @ p["w_router"]).topk(k, dim=1)
        s["ids"], s["w"] = top.indices, top.values.softmax(1)
        i32 = lambda n: torch.empty(n, dtype=torch.int32, device=x.device)
        order, s["pos"], offsets = i32(B * k), i32(B * k), i32(self.experts + 1)
        E.expert_sort(s["ids"], self.experts, order, s["pos"], offsets)
        s["xs"] = torch.empty((B * k, x.shape[1]), device=x.device)
        E.expert_dispatch(h, s["pos"], s["xs"])
        s["cuts"] = offsets.tolist()  # the products' sizes: the one wait for the device
        s["a"] = torch.empty((B * k, p["w1"].shape[2]), device=x.device)
        s["ys"] = torch.empty_like(s["xs"])
        for e, (lo, hi) in enumerate(zip(s["cuts"], s["cuts"][1:])):
            s["a"][lo:hi] = (s["xs"][lo:hi] @ p["w1"][e]).relu()
            s["ys"][lo:hi] = s["a"][lo:hi] @ p["w2"][e]
        y = s["y"] = torch.empty_like(x)
        E.expert_combine(s["ys"], s["pos"], s["w"], y)
        s["gate"] = h @ p["w_gate"]
        s["x_out"], s["h_out"] = torch.empty_like(x), torch.empty_like(x)
        E.gated_norm(x, y, s["x_out"], s["h_out"], gate=s["gate"], w_post=p["norm_post"],
                     res_scale=p["res_scale"], w_pre=p["norm_out"])
        return (s["h_out"] @ p["w_head"])[:, 0]

    def backward(self, dlogit):
        """Fills the gradients from the logits' and returns the input rows'."""
        p, g, s, k = self.p, self.g, self.s, self.k
        d = dlogit[:, None]
        torch.mm(s["h_out"].t(), d, out=g["w_head"])
        x = s["x"]
        dx, dy, dgate = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        E.gated_norm_backward(None, d @ p["w_head"].t(), s["x_out"], s["y"], dx, dy, gate=s["gate"],
                              w_post=p["norm_post"], res_scale=p["res_scale"], w_pre=p["norm_out"],
                              dgate=dgate, dw_post=g["norm_post"], dres_scale=g["res_scale"],
                              dw_pre=g["norm_out"])
        dys, dw = torch.empty_like(s["ys"]), torch.empty_like(s["w"])
        E.expert_combine_backward(dy, s["ys"], s["pos"], s["w"], dys, dw)
        dxs = torch.empty_like(s["xs"])
        for e, (lo, hi) in enumerate(zip(s["cuts"], s["cuts"][1:])):
            a, dyse = s["a"][lo:hi], dys[lo:hi]
            torch.mm(a.t(), dyse, out=g["w2"][e])
            da = (dyse @ p["w2"][e].t()) * (a > 0)
            torch.mm(s["xs"][lo:hi].t(), da, out=g["w1"][e])
            dxs[lo:hi] = da @ p["w1"][e].t()
        dh = torch.empty_like(x)
        E.expert_dispatch_backward(dxs, s["pos"], dh)
        # the router's softmax over the chosen experts, and the gate
        dtop = s["w"] * (dw - (dw * s["w"]).sum(1, keepdim=True))
        dscores = torch.zeros((x.shape[0], self.experts), device=x.device).scatter_(1, s["ids"], dtop)
        torch.mm(s["h"].t(), dscores, out=g["w_router"])
        torch.mm(s["h"].t(), dgate, out=g["w_gate"])
        dh.addmm_(dscores, p["w_router"].t()).addmm_(dgate, p["w_gate"].t())
        E.gated_norm_backward(dx, dh, x, None, dx, None, w_pre=p["norm_block"], dw_pre=g["norm_block"])
        torch.mm(s["h0"].t(), dx, out=g["w_in"])
        dfeats = torch.empty_like(s["feats"])
        E.gated_norm_backward(None, dx @ p["w_in"].t(), s["feats"], None, dfeats, None, w_pre=p["norm_in"],
                              dw_pre=g["norm_in"])
        return dfeats

    def step(self, lr: float = 0.02, max_norm: float = 1.0, eps: float = 1e-8):
        """Clips the gradients by their global norm and takes one Adagrad step."""
        E.clip_grads(self.g.values(), max_norm, self.norm)
        for name, v in self.p.items():
            acc, grad = self.acc[name], self.g[name]
            acc.addcmul_(grad, grad)
            v.addcdiv_(grad, acc.sqrt().add_(eps), value=-lr)


def train(steps: int, batch: int, rows: str = "small", seed: int = 0):
    """Losses of `steps` steps on one synthetic click model (labels from the dense features)."""
    import dataclasses

    import numpy as np

    import synth
    w = dataclasses.replace(synth.workload(2, "small" if rows == "small" else "full"), batch=batch)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    losses = []
    with E.EmbCtx.from_workload(w) as ctx:
        tower = ExpertTower(ctx.out_width, seed=seed)
        feats = torch.empty((batch, ctx.out_width), device="cuda")
        ddense = torch.empty((batch, ctx.D), device="cuda")
        for step in range(steps):
            b = synth.make_batch(w, step)
            ids, dense = dev(b.ids), dev(b.dense)
            label = (dense[:, :16].sum(1) > 0).float()
            ctx.forward_interact(ids, None, batch, dense, feats)
            logit = tower.forward(feats)
            loss = torch.nn.functional.binary_cross_entropy_with_logits(logit, label)
            dfeats = tower.backward((torch.sigmoid(logit) - label) / batch)
            tower.step()
            ctx.backward_interact_adagrad(dfeats, dense, ddense)
            losses.append(loss)
        assert ctx.get_status() == 0
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--batch", type=int, default=2048)
    ap.add_argument("--rows", choices=["small", "full"], default="small",
                    help="small: tables scaled down a thousandfold")
    a = ap.parse_args()
    losses = train(a.steps, a.batch, a.rows)
    for i, v in enumerate(losses):
        if i % 5 == 0 or i == len(losses) - 1:
            print(f"step {i:4d}  loss {v:.4f}")
