"""Cases for the operators of the expert tower that sits on the embedding layer: rows sorted by
expert and brought back with weights, the gated residual with a norm on either side, and the
global gradient norm with clipping.  Each case runs either the plain form (torch operations in
float32) or the framework's kernels (own = True)."""
import math

import numpy as np
import torch

own = False
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one request at serving time: a single sample through two of eight experts
        dict(name="experts_fwd_one", op="experts", n=1, k=2, experts=8, d=128, pad=0, dtype="bf16", drop=0.0),
        # the interaction output of 26 tables of width 128 (128 + 351 columns) as it comes, an odd
        # batch, a few slots dropped
        dict(name="experts_fwd_interaction", op="experts", n=16411, k=3, experts=24, d=479, pad=0, dtype="f32", drop=0.05),
        # the largest training batch, hidden width 512, many experts
        dict(name="experts_fwd_large", op="experts", n=262144, k=4, experts=128, d=512, pad=0, dtype="bf16", drop=0.0),
        # one gradient step of a small batch, rows inside a wider buffer
        dict(name="experts_bwd_small", op="experts_grad", n=1021, k=2, experts=8, d=128, pad=128, dtype="f32", drop=0.1),
        # the gradient of the largest training batch
        dict(name="experts_bwd_large", op="experts_grad", n=262144, k=2, experts=64, d=512, pad=0, dtype="bf16", drop=0.02),
        # a few requests at serving time, one gate a row
        dict(name="norm_fwd_serve", op="norm", n=16, d=1024, pad=0, xtype="bf16", dtype="bf16", gate="row"),
        # the interaction output's odd width, a gate for each element
        dict(name="norm_fwd_interaction", op="norm", n=16411, d=479, pad=0, xtype="f32", dtype="f32", gate="full"),
        # the largest batch, residual stream in 32 bits beside 16-bit blocks
        dict(name="norm_fwd_large", op="norm", n=262144, d=1024, pad=0, xtype="f32", dtype="bf16", gate="full"),
        # an ordinary training batch, no gate, rows inside a wider buffer
        dict(name="norm_bwd_ordinary", op="norm_grad", n=16384, d=512, pad=64, xtype="f32", dtype="f32", gate="none"),
        # the gradient of the largest batch
        dict(name="norm_bwd_large", op="norm_grad", n=262144, d=1024, pad=0, xtype="bf16", dtype="bf16", gate="full"),
        # the dense tensors of a small tower
        dict(name="clip_tower", op="clip", count=16, width=250, dtype="f32", mixed=False, limit=0.5),
        # wide dense layers, 16-bit weights' gradients beside 32-bit biases'
        dict(name="clip_large", op="clip", count=40, width=5001, dtype="bf16", mixed=True, limit=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    while True:
        op = rng.choice(["experts", "experts_grad", "norm", "norm_grad", "clip"])
        if op in ("experts", "experts_grad"):
            e = _log(rng, 2, 256)
            d = _log(rng, 16, 2048)
            c = dict(op=op, n=_log(rng, 1, 262144), k=min(e, rng.choice([1, 2, 3, 4, 6, 8])), experts=e,
                     d=d if rng.random() < 0.4 else -(-d // 8) * 8, pad=rng.choice([0, 0, 8, 33]),
                     dtype=rng.choice(["f32", "bf16"]), drop=round(rng.choice([0.0, rng.random() * 0.5]), 3))
        elif op in ("norm", "norm_grad"):
            d = _log(rng, 16, 8192)
            t = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
            c = dict(op=op, n=_log(rng, 1, 262144), d=d if rng.random() < 0.4 else -(-d // 8) * 8,
                     pad=rng.choice([0, 0, 8, 33]), xtype=t[0], dtype=t[1], gate=rng.choice(["none", "row", "full"]))
        else:
            c = dict(op=op, count=rng.randint(1, 48), width=_log(rng, 8, 5000), dtype=rng.choice(["f32", "bf16"]),
                     mixed=rng.random() < 0.5, limit=rng.choice([0.1, 0.5, 0.9, 2.0]))
        if work(c)["bytes"] <= most:
            return c


def _sizes(c):
    """A tower's tensors: weight matrices, each followed by its bias."""
    return [(c["width"] + i) * c["width"] if i % 2 == 0 else c["width"] + i for i in range(c["count"])]


def _types(c):
    return [torch.float32 if c["mixed"] and i % 2 else DTYPES[c["dtype"]] for i in range(c["count"])]


def _rows(g, n, d, pad, dtype, scale=1.0):
    """n rows of d normal values, inside rows of d + pad."""
    return (torch.randn((n, d + pad), generator=g, device="cuda") * scale).to(dtype)[:, :d]


def _room(n, d, dtype):
    return torch.empty((n, d), dtype=dtype, device="cuda")


def _i32(n):
    return torch.empty(n, dtype=torch.int32, device="cuda")


def _f32(n):
    return torch.empty(n, device="cuda")


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    t = DTYPES[c["dtype"]]
    if c["op"] in ("experts", "experts_grad"):
        n, k, e, d = c["n"], c["k"], c["experts"], c["d"]
        # a router's choice: k different experts a row, some experts far more popular than others
        liking = torch.randn(e, generator=g, device="cuda") * 0.5
        top = (torch.randn((n, e), generator=g, device="cuda") + liking).topk(k, dim=1)
        s["ids"] = top.indices.masked_fill(torch.rand((n, k), generator=g, device="cuda") < c["drop"], -1)
        s["w"] = top.values.softmax(1)
        s["ys"] = _rows(g, n * k, d, c["pad"], t)
        if c["op"] == "experts":
            s["x"] = _rows(g, n, d, c["pad"], t)
            s |= dict(order=_i32(n * k), pos=_i32(n * k), offsets=_i32(e + 1), xs=_room(n * k, d, t), out=_room(n, d, t))
        else:
            s["pos"] = _sort(s["ids"], e)[1]
            s["dout"] = _rows(g, n, d, c["pad"], t)
            s["dxs"] = _rows(g, n * k, d, c["pad"], t)
            s |= dict(dx=_room(n, d, t), dys=_room(n * k, d, t), dw=_f32((n, k)))
    elif c["op"] in ("norm", "norm_grad"):
        n, d, xt = c["n"], c["d"], DTYPES[c["xtype"]]
        s["y"] = _rows(g, n, d, c["pad"], t, 0.7)
        s["gate"] = None if c["gate"] == "none" else _rows(g, n, d if c["gate"] == "full" else 1, c["pad"], t, 1.5)
        for name, mean in (("w_post", 1.0), ("res_scale", 0.3), ("w_pre", 1.0)):
            s[name] = mean + 0.1 * torch.randn(d, generator=g, device="cuda")
        s["x"] = _rows(g, n, d, c["pad"], xt, 2.0)  # the residual stream: before the block, or after it
        if c["op"] == "norm":
            s |= dict(x_out=_room(n, d, xt), h=_room(n, d, t))
        else:
            s["dx_out"] = _rows(g, n, d, c["pad"], xt)
            s["dh"] = _rows(g, n, d, c["pad"], t)
            s |= dict(dx=_room(n, d, xt), dy=_room(n, d, t), dw_post=_f32(d), dres_scale=_f32(d), dw_pre=_f32(d),
                      dgate=None if s["gate"] is None else _room(n, s["gate"].shape[1], t))
    else:
        sizes, types = _sizes(c), _types(c)
        s["grads"] = [(torch.randn(m, generator=g, device="cuda") * 1e-3).to(u) for m, u in zip(sizes, types)]
        s["max_norm"] = c["limit"] * 1e-3 * math.sqrt(sum(sizes))
        s |= dict(out=[torch.empty_like(x) for x in s["grads"]], norm=_f32(1))
    return s


# ---- plain forms ----

def _sort(ids, experts):
    n, k = ids.shape
    key = ids.reshape(-1)
    key = torch.where((key < 0) | (key >= experts), experts, key)
    by, order = key.sort(stable=True)
    place = torch.arange(n * k, device=ids.device)
    pos = torch.empty_like(place).scatter_(0, order, place)
    pos = torch.where(key == experts, -1 - pos, pos)
    offsets = torch.searchsorted(by, torch.arange(experts + 1, device=ids.device))
    return order.to(torch.int32), pos.to(torch.int32), offsets.to(torch.int32)


def _plain_experts(s):
    c, x, ys, w = s["case"], s["x"], s["ys"], s["w"]
    n, k = w.shape
    order, pos, offsets = _sort(s["ids"], c["experts"])
    xs = x[order.long() // k]
    xs = torch.where((torch.arange(n * k, device=x.device) < offsets[-1])[:, None], xs, 0)
    p = pos.long().reshape(n, k)
    back = torch.where((p >= 0)[..., None], ys.float()[p.clamp_min(0)] * w[..., None], 0)
    return dict(order=order, pos=pos, offsets=offsets, xs=xs, out=back.sum(1).to(x.dtype))


def _plain_experts_grad(s):
    dxs, ys, dout, w = s["dxs"], s["ys"], s["dout"], s["w"]
    n, k = w.shape
    pos = s["pos"].long()
    p, kept = pos.clamp_min(0), (pos >= 0)[:, None]
    dx = torch.where(kept, dxs.float()[p], 0).reshape(n, k, -1).sum(1).to(dxs.dtype)
    each = dout.float().repeat_interleave(k, 0)
    dw = torch.where(kept, ys.float()[p] * each, 0).sum(1).reshape(n, k)
    to = torch.where(pos >= 0, pos, -1 - pos)
    rows = torch.where(kept, each * w.reshape(-1, 1), 0).to(ys.dtype)
    dys = torch.empty((n * k, ys.shape[1]), dtype=ys.dtype, device=ys.device)
    dys[to] = rows
    return dict(dx=dx, dys=dys, dw=dw)


def _rms(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _plain_norm(s):
    x, y, gate = s["x"].float(), s["y"].float(), s["gate"]
    p = y * _rms(y) * s["w_post"]
    if gate is not None:
        p = p * torch.sigmoid(gate.float())
    x_out = x + s["res_scale"] * p
    h = x_out * _rms(x_out) * s["w_pre"]
    return dict(x_out=x_out.to(s["x"].dtype), h=h.to(s["y"].dtype))


def _plain_norm_grad(s):
    x, y, dx_out, dh, gate = s["x"].float(), s["y"].float(), s["dx_out"].float(), s["dh"].float(), s["gate"]
    r = _rms(x)
    q = x * r
    dw_pre = (dh * q).sum(0)
    dq = dh * s["w_pre"]
    dx = dx_out + r * (dq - q * (dq * q).mean(1, keepdim=True))
    r = _rms(y)
    a = y * r
    p = a * s["w_post"]
    g = 1.0 if gate is None else torch.sigmoid(gate.float())
    dres_scale = (dx * g * p).sum(0)
    dgp = dx * s["res_scale"]
    dgate = None
    if gate is not None:
        dgate = dgp * p
        if gate.shape[1] < y.shape[1]:
            dgate = dgate.sum(1, keepdim=True)
        dgate = (dgate * g * torch.sigmoid(-gate.float())).to(gate.dtype)
    dp = dgp * g
    dw_post = (dp * a).sum(0)
    da = dp * s["w_post"]
    dy = r * (da - a * (da * a).mean(1, keepdim=True))
    return dict(dx=dx.to(s["x"].dtype), dy=dy.to(s["y"].dtype), dgate=dgate, dw_post=dw_post, dres_scale=dres_scale, dw_pre=dw_pre)


def _plain_clip(s):
    norm = torch.stack([x.float().square().sum() for x in s["grads"]]).sum().sqrt()
    c = torch.clamp(s["max_norm"] / norm, max=1.0)
    return dict(norm=norm.reshape(1), out=[(x.float() * c).to(x.dtype) for x in s["grads"]])


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"experts": _plain_experts, "experts_grad": _plain_experts_grad, "norm": _plain_norm,
                "norm_grad": _plain_norm_grad, "clip": _plain_clip}[op](s)
    import recommender_model_embedding_gb300 as E
    if op == "experts":
        E.expert_sort(s["ids"], s["case"]["experts"], s["order"], s["pos"], s["offsets"])
        E.expert_dispatch(s["x"], s["pos"], s["xs"])
        E.expert_combine(s["ys"], s["pos"], s["w"], s["out"])
        return {name: s[name] for name in ("order", "pos", "offsets", "xs", "out")}
    if op == "experts_grad":
        E.expert_combine_backward(s["dout"], s["ys"], s["pos"], s["w"], s["dys"], s["dw"])
        E.expert_dispatch_backward(s["dxs"], s["pos"], s["dx"])
        return {name: s[name] for name in ("dx", "dys", "dw")}
    if op == "norm":
        E.gated_norm(s["x"], s["y"], s["x_out"], s["h"], gate=s["gate"], w_post=s["w_post"],
                     res_scale=s["res_scale"], w_pre=s["w_pre"], eps=EPS)
        return dict(x_out=s["x_out"], h=s["h"])
    if op == "norm_grad":
        E.gated_norm_backward(s["dx_out"], s["dh"], s["x"], s["y"], s["dx"], s["dy"], gate=s["gate"],
                              w_post=s["w_post"], res_scale=s["res_scale"], w_pre=s["w_pre"], dgate=s["dgate"],
                              dw_post=s["dw_post"], dres_scale=s["dres_scale"], dw_pre=s["dw_pre"], eps=EPS)
        return {name: s[name] for name in ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre")}
    E.clip_grads(s["grads"], s["max_norm"], s["norm"], out=s["out"])
    return dict(norm=s["norm"], out=s["out"])


def work(case):
    c = case
    b = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("experts", "experts_grad"):
        n, k, d = c["n"], c["k"], c["d"]
        slots, kept = n * k, n * k * (1 - c["drop"])
        if c["op"] == "experts":
            # ids and weights in, order, places and offsets out; x and the kept rows of ys in, xs and out out
            return {"bytes": slots * 20 + 4 * (c["experts"] + 1) + (2 * n + slots + kept) * d * b, "flops": 2 * kept * d}
        # places and weights in, dw out; dout and the kept rows of ys and dxs in, dx and dys out
        return {"bytes": slots * 12 + (2 * n + slots + 2 * kept) * d * b, "flops": 4 * kept * d}
    if c["op"] in ("norm", "norm_grad"):
        n, d = c["n"], c["d"]
        xb = 4 if c["xtype"] == "f32" else 2
        gate = {"none": 0, "row": 1, "full": d}[c["gate"]]
        if c["op"] == "norm":
            return {"bytes": n * (d * (2 * xb + 2 * b) + gate * b) + 12 * d, "flops": 12 * n * d}
        return {"bytes": n * (d * (3 * xb + 3 * b) + 2 * gate * b) + 24 * d, "flops": 30 * n * d}
    total = sum(m * (4 if u == torch.float32 else 2) for m, u in zip(_sizes(c), _types(c)))
    return {"bytes": 2 * total + 4, "flops": 3 * sum(_sizes(c))}


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = {name: v.double() for name, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op in ("experts", "experts_grad"):
        ids = s["ids"].cpu().numpy().reshape(-1)
        n, k, e = case["n"], case["k"], case["experts"]
        inside = (ids >= 0) & (ids < e)
        order = np.lexsort((np.arange(n * k), np.where(inside, ids, e)))
        kept = torch.from_numpy(order[:int(inside.sum())]).cuda()  # the slot of each sorted row
        token = torch.div(kept, k, rounding_mode="floor")
        m = kept.numel()
        weight = f64["w"].reshape(-1)[kept][:, None]
        if op == "experts":
            out = torch.zeros((n, case["d"]), dtype=torch.float64, device="cuda")
            out.index_add_(0, token, f64["ys"][:m] * weight)
            return dict(order=None, pos=None, offsets=None, xs=None, out=out)
        dx = torch.zeros((n, case["d"]), dtype=torch.float64, device="cuda").index_add_(0, token, f64["dxs"][:m])
        dys = torch.zeros((n * k, case["d"]), dtype=torch.float64, device="cuda")
        dys[:m] = f64["dout"][token] * weight
        dw = torch.zeros(n * k, dtype=torch.float64, device="cuda")
        dw[kept] = torch.linalg.vecdot(f64["dout"][token], f64["ys"][:m])
        return dict(dx=dx, dys=dys, dw=dw.reshape(n, k))
    if op in ("norm", "norm_grad"):
        y, x, wp, rs, wq = (f64[name] for name in ("y", "x", "w_post", "res_scale", "w_pre"))
        d = case["d"]
        ly = torch.sqrt((y * y).sum(1, keepdim=True) / d + EPS)
        g = 1 / (1 + torch.exp(-f64["gate"])) if s["gate"] is not None else torch.ones((), dtype=torch.float64, device="cuda")
        if op == "norm":
            x_out = x + rs * g * wp * y / ly
            return dict(x_out=x_out, h=wq * x_out / torch.sqrt((x_out * x_out).sum(1, keepdim=True) / d + EPS))
        dh, dx_out = f64["dh"], f64["dx_out"]
        lx = torch.sqrt((x * x).sum(1, keepdim=True) / d + EPS)
        # the derivative of x / lx along dh * w_pre, and so for y
        u = dh * wq
        dx = dx_out + u / lx - x * (u * x).sum(1, keepdim=True) / (d * lx ** 3)
        v = dx * rs * g * wp
        dy = v / ly - y * (v * y).sum(1, keepdim=True) / (d * ly ** 3)
        dgate = None
        if s["gate"] is not None:
            t = dx * rs * wp * y / ly
            dgate = (t if case["gate"] == "full" else t.sum(1, keepdim=True)) * g * (1 - g)
        return dict(dx=dx, dy=dy, dgate=dgate, dw_post=(dx * rs * g * y / ly).sum(0),
                    dres_scale=(dx * g * wp * y / ly).sum(0), dw_pre=(dh * x / lx).sum(0))
    total = math.sqrt(sum(float(torch.linalg.vector_norm(x.double())) ** 2 for x in s["grads"]))
    c = min(1.0, s["max_norm"] / total)
    return dict(norm=torch.tensor([total], dtype=torch.float64), out=[x.double() * c for x in s["grads"]])
