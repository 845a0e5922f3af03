"""Cases for the experts' products of the expert tower: the grouped linear layer and the gated
feed-forward block over rows sorted by expert, with their gradients, dropout with a residual, and
the grouped product from 4-bit weights.  Each case runs either the plain form (torch operations
in float32) or the framework's kernels (own = True)."""
import math

import torch

own = False
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # one request at serving time: a single sample through two of eight experts
        _case("gated", "gated_fwd_one", n=1, k=2, experts=8, d=512, f=1024),
        # the interaction output of 26 tables of width 128 (128 + 351 columns) as it comes, an odd
        # batch, a few slots dropped
        _case("gated", "gated_fwd_interaction", n=4099, k=2, experts=12, d=479, f=640, dtype="f32", drop=0.05, act="gelu"),
        # the largest training batch, what the gradient needs is kept
        _case("gated", "gated_fwd_large", n=262144, k=2, experts=64, d=512, f=1024, keep=True),
        # a gradient step of a small tower, weights laid out [in, out], rows inside a wider buffer
        _case("gated_grad", "gated_bwd_small", n=2048, k=2, experts=8, d=256, f=256, dtype="f32", order="io", pad=64, drop=0.1),
        # the gradient of the largest training batch
        _case("gated_grad", "gated_bwd_large", n=262144, k=2, experts=64, d=512, f=1024, drop=0.02),
        # a few requests at serving time, the block's second product
        _case("linear", "linear_fwd_serve", n=16, k=2, experts=8, d=1024, f=512),
        # the block's second product at the largest training batch
        _case("linear", "linear_fwd_large", n=262144, k=2, experts=64, d=1024, f=512),
        # the gradient of one dense layer on the interaction output's odd width, no experts
        _case("linear_grad", "linear_bwd_dense", n=16411, k=1, experts=0, d=479, f=1000, pad=33),
        # a few rows of a small step, joined to the residual stream
        dict(name="dropout_small", op="dropout", n=16, d=1024, pad=0, xtype="bf16", dtype="bf16", residual=True, p=0.1),
        # the largest training batch, residual stream in 32 bits
        dict(name="dropout_large", op="dropout", n=262144, d=1024, pad=0, xtype="f32", dtype="bf16", residual=True, p=0.2),
        # one request at serving time from 4-bit weights: two of eight experts
        _case("linear4", "linear4_one", n=1, k=2, experts=8, d=1024, f=2048, group=64),
        # a few requests through one dense layer on the interaction output's odd width
        _case("linear4", "linear4_few", n=13, k=1, experts=0, d=479, f=4096, dtype="f32", group=32),
    ]


def _case(op, name=None, n=1, k=1, experts=0, d=1, f=1, dtype="bf16", order="oi", pad=0, drop=0.0, act="silu",
          keep=False, group=0):
    """n rows for k of `experts` each (0: one dense layer) from width d to width f; order: weights
    lie [out, in] or [in, out]."""
    c = dict(op=op, n=n, k=k, experts=experts, d=d, f=f, dtype=dtype, order=order, pad=pad, drop=drop)
    if op.startswith("gated"):
        c["act"] = act
    if op == "gated":
        c["keep"] = keep
    if op == "linear4":
        c["group"] = group
    return dict(name=name, **c) if name else c


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {m: max(work(c)[m] for c in listed()) for m in ("bytes", "flops")}
    while True:
        op = rng.choice(["gated", "gated_grad", "linear", "linear_grad", "dropout", "linear4"])
        if op == "dropout":
            d = _log(rng, 16, 8192)
            t = rng.choice([("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
            c = dict(op=op, n=_log(rng, 1, 262144), d=d if rng.random() < 0.4 else -(-d // 8) * 8, pad=rng.choice([0, 0, 8, 33]),
                     xtype=t[0], dtype=t[1], residual=rng.random() < 0.6, p=round(rng.choice([0.1, 0.5, rng.random()]), 3))
        else:
            e = rng.choice([0, _log(rng, 2, 256)])
            wide = 8192 if op == "linear4" else 2048
            d, f = _log(rng, 16, wide), _log(rng, 16, wide)
            if rng.random() < 0.6:
                d, f = -(-d // 8) * 8, -(-f // 8) * 8
            c = _case(op, n=_log(rng, 1, 32 if op == "linear4" else 262144), k=min(max(e, 1), rng.choice([1, 2, 3, 4])), experts=e,
                      d=d, f=f, dtype=rng.choice(["f32", "bf16", "bf16"]), pad=rng.choice([0, 0, 8, 33]),
                      order="oi" if op == "linear4" else rng.choice(["oi", "io"]),
                      drop=round(rng.choice([0.0, rng.random() * 0.5]), 3) if e else 0.0,
                      act=rng.choice(["silu", "gelu", "relu", "sigmoid"]), keep=rng.random() < 0.5, group=rng.choice([32, 64, 128]))
        w = work(c)
        if all(w[m] <= most[m] for m in most) and c["n"] * c["d"] < 1 << 31:
            return c


def _slots(c):
    """Rows of the products, and how many of them are kept."""
    slots = c["n"] * c["k"]
    return slots, slots - int(slots * c["drop"])


def _outs(c):
    """Rows of a weight matrix: a gated block has two of them, one above the other."""
    return 2 * c["f"] if c["op"].startswith("gated") else c["f"]


def _rows(g, n, d, pad, dtype, scale=1.0):
    """n rows of d normal values, inside rows of d + pad."""
    return (torch.randn((n, d + pad), generator=g, device="cuda") * scale).to(dtype)[:, :d]


def _turned(c, w):
    return w.transpose(1, 2) if c["order"] == "io" else w


def _weights(c, shape, make):
    """[experts, out, in], lying in memory as the case's order says; without experts [out, in]."""
    e, o, i = shape
    w = _turned(c, make((e, i, o) if c["order"] == "io" else (e, o, i)))
    return w if c["experts"] else w[0]


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": c}
    t = DTYPES[c["dtype"]]
    if c["op"] == "dropout":
        s["x"] = _rows(g, c["n"], c["d"], c["pad"], t)
        s["residual"] = _rows(g, c["n"], c["d"], c["pad"], DTYPES[c["xtype"]], 2.0) if c["residual"] else None
        s["rng"] = torch.randint(0, 1 << 40, (2,), generator=g, device="cuda")  # seed and step
        s["site"] = 3
        s["out"] = torch.empty((c["n"], c["d"]), dtype=DTYPES[c["xtype"]] if c["residual"] else t, device="cuda")
        return s
    slots, kept = _slots(c)
    e, d, o = max(c["experts"], 1), c["d"], _outs(c)
    # rows by expert: no expert twice while there are enough of them, some liked better than others
    liking = (torch.randn(e, generator=g, device="cuda") * 0.2).softmax(0)
    if kept <= e:
        count = torch.zeros(e, dtype=torch.int64, device="cuda")
        count[torch.randperm(e, generator=g, device="cuda")[:kept]] = 1
    else:
        count = torch.multinomial(liking, kept, replacement=True, generator=g).bincount(minlength=e)
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    s["offsets"] = offsets.to(torch.int32) if c["experts"] else None
    # for the plain form: the experts in use, and each one's rows in a matrix of the longest's height
    s["used"] = count.nonzero()[:, 0]
    high = max(1, int(count.max()))
    place = torch.arange(high, device="cuda")
    s["valid"] = place < count[s["used"], None]
    s["index"] = torch.where(s["valid"], offsets[s["used"], None] + place, 0)
    s["kept"] = kept
    s["x"] = _rows(g, slots, d, c["pad"], t)
    if c["op"] == "linear4":
        s["q"] = torch.randint(0, 256, (e, o, -(-d // 2)), generator=g, device="cuda", dtype=torch.uint8)
        s["scale"] = (0.5 + torch.rand((e, o, -(-d // c["group"])), generator=g, device="cuda")) / (4.6 * math.sqrt(d))
        if not c["experts"]:
            s["q"], s["scale"] = s["q"][0], s["scale"][0]
    else:
        s["w"] = _weights(c, (e, o, d), lambda m: (torch.randn(m, generator=g, device="cuda") / math.sqrt(d)).to(t))
    room = lambda width: torch.zeros((slots, width), dtype=t, device="cuda")
    if c["op"] == "gated":
        s |= dict(h=room(c["f"]), gu=room(o) if c["keep"] else None)
    elif c["op"] in ("linear", "linear4"):
        s["out"] = room(o)
    else:
        if c["op"] == "gated_grad":
            s["gu"] = _product(s, s["x"], _stack(s)).to(t)  # as the forward left it
            s["dh"] = _rows(g, slots, c["f"], c["pad"], t)
        else:
            s["dout"] = _rows(g, slots, o, c["pad"], t)
        s |= dict(dx=room(d), dw=_weights(c, (e, o, d), lambda m: torch.zeros(m, device="cuda")))
    return s


# ---- plain forms ----

def _stack(s):
    """The weights of the experts in use, in float32."""
    w = s["w"] if s["case"]["experts"] else s["w"][None]
    return w[s["used"]].float()


def _by_expert(s, x):
    return torch.where(s["valid"][..., None], x.float()[s["index"]], 0)


def _back(s, y):
    """Rows in their order again, zero at the dropped places."""
    out = torch.zeros((s["x"].shape[0], y.shape[2]), device=y.device)
    out[:s["kept"]] = y[s["valid"]]
    return out


def _product(s, x, w):
    return _back(s, torch.bmm(_by_expert(s, x), w.transpose(1, 2)))


def _act(name, v):
    if name == "relu":
        return v.clamp_min(0)
    return {"silu": lambda: v / (1 + torch.exp(-v)), "sigmoid": lambda: 1 / (1 + torch.exp(-v)),
            "gelu": lambda: 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))}[name]()


def _act_grad(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    a = 1 / (1 + torch.exp(-v))
    return a * (1 - a) if name == "sigmoid" else a * (1 + v * (1 - a))


def _plain_gated(s):
    c, t = s["case"], s["x"].dtype
    gu = _product(s, s["x"], _stack(s))
    gate, up = gu[:, :c["f"]], gu[:, c["f"]:]
    # (a sigmoid's gate is not zero at zero, but the row's `up` is)
    return dict(h=(_act(c["act"], gate) * up).to(t), gu=gu.to(t) if c["keep"] else None)


def _plain_grad(s):
    c, t = s["case"], s["x"].dtype
    if c["op"] == "gated_grad":
        gate, up, dh = s["gu"][:, :c["f"]].float(), s["gu"][:, c["f"]:].float(), s["dh"].float()
        dout = torch.cat([dh * up * _act_grad(c["act"], gate), dh * _act(c["act"], gate)], 1)
    else:
        dout = s["dout"]
    by = _by_expert(s, dout)
    dx = _back(s, torch.bmm(by, _stack(s))).to(t)
    dw = torch.zeros((max(c["experts"], 1), _outs(c), c["d"]), device=dx.device)
    dw[s["used"]] = torch.bmm(by.transpose(1, 2), _by_expert(s, s["x"]))
    return dict(dx=dx, dw=dw if c["experts"] else dw[0])


def _plain_linear4(s):
    c = s["case"]
    q, scale = (v if c["experts"] else v[None] for v in (s["q"], s["scale"]))
    q = q[s["used"]]
    code = torch.stack([q & 15, q >> 4], -1).flatten(2)[..., :c["d"]].float() - 8
    w = code * scale[s["used"]].repeat_interleave(c["group"], 2)[..., :c["d"]]
    return dict(out=_product(s, s["x"], w).to(s["x"].dtype))


def _bits(rng, site, n, d):
    """16 random bits for each element of an [n, d] matrix: Philox4x32-10 (Salmon, Moraes, Dror and
    Shaw, 2011) of (block of 8 columns, row, step, site) under the seed."""
    low = 0xFFFFFFFF
    blocks = -(-d // 8)
    full = lambda v: v.expand(n, blocks)
    a = full(torch.arange(blocks, device=rng.device)[None, :])
    b = full(torch.arange(n, device=rng.device)[:, None])
    c, e = full(rng[1] & low), full(torch.full_like(rng[0], site))
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, e = ((q >> 32) & low) ^ b ^ k0, q & low, ((p >> 32) & low) ^ e ^ k1, p & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([a, b, c, e], -1)
    return torch.stack([words & 0xFFFF, words >> 16], -1).reshape(n, blocks * 8)[:, :d]


def _plain_dropout(s):
    c = s["case"]
    cut = round(c["p"] * 65536)
    scale = 65536 / (65536 - cut) if cut < 65536 else 0.0
    kept = torch.where(_bits(s["rng"], s["site"], c["n"], c["d"]) >= cut, s["x"].float() * scale, 0)
    return dict(out=(kept if s["residual"] is None else s["residual"].float() + kept).to(s["out"].dtype))


def run(state):
    s = state
    c = s["case"]
    if not own:
        return {"gated": _plain_gated, "gated_grad": _plain_grad, "linear_grad": _plain_grad,
                "linear": lambda s: dict(out=_product(s, s["x"], _stack(s)).to(s["x"].dtype)),
                "linear4": _plain_linear4, "dropout": _plain_dropout}[c["op"]](s)
    import recommender_model_embedding_gb300 as E
    if c["op"] == "gated":
        E.expert_gated(s["x"], s["w"], s["h"], gu=s["gu"], offsets=s["offsets"], act=c["act"])
        return dict(h=s["h"], gu=s["gu"])
    if c["op"] == "gated_grad":
        E.expert_gated_backward(s["dh"], s["gu"], s["x"], s["w"], s["dx"], s["dw"], offsets=s["offsets"], act=c["act"])
        return dict(dx=s["dx"], dw=s["dw"])
    if c["op"] == "linear":
        E.expert_linear(s["x"], s["w"], s["out"], offsets=s["offsets"])
    elif c["op"] == "linear_grad":
        E.expert_linear_backward(s["dout"], s["x"], s["w"], s["dx"], s["dw"], offsets=s["offsets"])
        return dict(dx=s["dx"], dw=s["dw"])
    elif c["op"] == "linear4":
        E.expert_linear4(s["x"], s["q"], s["scale"], s["out"], group=c["group"], offsets=s["offsets"])
    else:
        E.dropout(s["x"], s["out"], c["p"], s["rng"], site=s["site"], residual=s["residual"])
    return dict(out=s["out"])


def work(case):
    c = case
    b = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "dropout":
        xb = 4 if c["xtype"] == "f32" else 2
        each = b + 2 * xb if c["residual"] else 2 * b
        return {"bytes": c["n"] * c["d"] * each + 16, "flops": 3 * c["n"] * c["d"]}
    slots, kept = _slots(c)
    d, f, o, e = c["d"], c["f"], _outs(c), max(c["experts"], 1)
    used = kept if kept <= e else e * (1 - (1 - 1 / e) ** kept)  # experts that have rows, on average
    small = 4 * (e + 1) if c["experts"] else 0
    if c["op"] == "linear4":
        return {"bytes": int(kept * (d + o) * b + used * o * (-(-d // 2) + 4 * -(-d // c["group"]))) + small, "flops": 2 * kept * d * o}
    if c["op"] in ("linear", "gated"):
        out = f * (3 if c.get("keep") else 1)
        return {"bytes": int(kept * (d + out) * b + used * o * d * b) + small, "flops": 2 * kept * d * o}
    # the gradients of the outputs (and what the forward kept), x and the weights in, dx and dw out
    grads = 3 * f if c["op"] == "gated_grad" else f
    return {"bytes": int(kept * (grads + 2 * d) * b + used * o * d * b + 4 * e * o * d) + small, "flops": 4 * kept * d * o}


# ---- from the definitions, in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "dropout":
        return dict(out=_exact_dropout(s))
    x = s["x"].double()
    cuts = s["offsets"].tolist() if c["experts"] else [0, x.shape[0]]
    o = _outs(c)
    if c["op"] == "linear4":
        def weight(e):
            q, scale = (s["q"][e], s["scale"][e]) if c["experts"] else (s["q"], s["scale"])
            column = torch.arange(c["d"], device="cuda")
            code = (q[:, column // 2] >> (4 * (column % 2)).to(torch.uint8)) & 15
            return (code.double() - 8) * scale.double()[:, column // c["group"]]
    else:
        def weight(e):
            return (s["w"][e] if c["experts"] else s["w"]).double()
    spans = [(e, lo, hi) for e, (lo, hi) in enumerate(zip(cuts, cuts[1:])) if hi > lo]
    if c["op"] in ("linear", "linear4", "gated"):
        y = torch.zeros((x.shape[0], o), dtype=torch.float64, device="cuda")
        for e, lo, hi in spans:
            y[lo:hi] = x[lo:hi] @ weight(e).T
        if c["op"] != "gated":
            return dict(out=y)
        return dict(h=_exact_act(c["act"], y[:, :c["f"]])[0] * y[:, c["f"]:], gu=y if c["keep"] else None)
    if c["op"] == "gated_grad":
        act, slope = _exact_act(c["act"], s["gu"][:, :c["f"]].double())
        dh = s["dh"].double()
        dout = torch.cat([dh * s["gu"][:, c["f"]:].double() * slope, dh * act], 1)
    else:
        dout = s["dout"].double()
    dx = torch.zeros((x.shape[0], c["d"]), dtype=torch.float64, device="cuda")
    dw = torch.zeros((max(c["experts"], 1), o, c["d"]), dtype=torch.float64, device="cuda")
    for e, lo, hi in spans:
        dx[lo:hi] = dout[lo:hi] @ weight(e)
        dw[e] = dout[lo:hi].T @ x[lo:hi]
    return dict(dx=dx, dw=dw if c["experts"] else dw[0])


def _exact_act(name, v):
    """An activation and its slope."""
    if name == "relu":
        return torch.where(v > 0, v, 0), (v > 0).double()
    if name == "gelu":
        normal = 0.5 * torch.erfc(-v / math.sqrt(2))  # the normal distribution function
        return v * normal, normal + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    a = torch.sigmoid(v)
    return (a, a * torch.sigmoid(-v)) if name == "sigmoid" else (v * a, a + v * a * torch.sigmoid(-v))


def _exact_dropout(s):
    c = s["case"]
    seed, step = (int(v) for v in s["rng"])
    n, d = c["n"], c["d"]
    cell = torch.arange(n * -(-d // 8), device="cuda")
    low = (1 << 32) - 1
    wide = -(-d // 8)
    word = [cell % wide, torch.div(cell, wide, rounding_mode="floor"), torch.full_like(cell, step & low), torch.full_like(cell, s["site"])]

    def high_low(v, m):  # of a 64-bit product, by halves of the factor
        lower, upper = v * (m & 0xFFFF), v * (m >> 16)
        total = lower + ((upper & 0xFFFF) << 16)
        return (upper >> 16) + (total >> 32), total & low

    for i in range(10):
        keys = (seed + i * 0x9E3779B9) & low, ((seed >> 32) + i * 0xBB67AE85) & low
        (h0, l0), (h1, l1) = high_low(word[0], 0xD2511F53), high_low(word[2], 0xCD9E8D57)
        word = [h1 ^ word[1] ^ keys[0], l1, h0 ^ word[3] ^ keys[1], l0]
    out = torch.zeros((n, d), dtype=torch.float64, device="cuda") if s["residual"] is None else s["residual"].double()
    cut = round(c["p"] * 65536)
    for t in range(min(8, d)):
        keep = ((word[t // 2] >> (16 * (t % 2))) & 0xFFFF).reshape(n, wide)[:, :len(range(t, d, 8))] >= cut
        out[:, t::8] += torch.where(keep, s["x"][:, t::8].double() * (65536 / max(65536 - cut, 1)), 0)
    return out
