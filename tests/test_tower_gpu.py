"""The expert tower's operators against plain implementations in 64 bits.

Tolerances: with u = 2^-24, a sum of m products in fp32, in any order, is within (m + 2) u of
the sum of the terms' sizes; every expression below carries its bound through from that, plus
one rounding of the output (u for fp32, 2^-8 for bf16 with its 8 significant bits, relative).
The constant 40 u covers the few elementary operations between sums (rsqrt, exp, divisions and
products, each within a few u)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from helpers import build_lib
    build_lib()
    import recommender_model_embedding_gb300 as E
    return E


def within(got, ref, err, what):
    """|got - ref| <= err + the rounding of got's type, with equal infinities and NaNs."""
    r = 2.0 ** -8 if got.dtype == torch.bfloat16 else U32
    got = got.double()
    fin = ref.isfinite()
    assert torch.equal(got.isnan(), ref.isnan()), what
    assert torch.equal(got[~fin & ~ref.isnan()], ref[~fin & ~ref.isnan()]), what
    bound = err * (1 + r) + r * ref.abs() + 1e-38
    bad = fin & ((got - ref).abs() > bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()}; first {i}: got {got[i].item()!r} "
                             f"ref {ref[i].item()!r} bound {bound[i].item()!r}")


def rows(g, n, d, dtype, pad=0, skip=0, scale=1.0):
    """[n, d] normal values inside rows of skip + d + pad."""
    return (torch.randn((n, skip + d + pad), generator=g, device="cuda") * scale).to(dtype)[:, skip:skip + d]


def room(n, d, dtype, pad=0, skip=0):
    """[n, d] output inside a buffer of sentinels, and that buffer."""
    full = torch.full((n, skip + d + pad), 77.0, dtype=dtype, device="cuda")
    return full[:, skip:skip + d], full


def outside_untouched(full, d, skip):
    assert bool((full[:, :skip] == 77.0).all()) and bool((full[:, skip + d:] == 77.0).all())


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---- sort ----

def sort_ref(ids, e):
    key = ids.reshape(-1).cpu().numpy()
    key = np.where((key < 0) | (key >= e), e, key)
    order = np.argsort(key, kind="stable")
    pos = np.empty(order.size, np.int64)
    pos[order] = np.arange(order.size)
    pos = np.where(key == e, -1 - pos, pos)
    return order, pos, np.searchsorted(key[order], np.arange(e + 1))


def sort(E, ids, e, **kw):
    S = ids.numel()
    order, pos = (torch.full((S,), -77, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.full((e + 1,), -77, dtype=torch.int32, device="cuda")
    E.expert_sort(ids, e, order, pos, off, **kw)
    return order, pos, off


def check_sort(E, ids, e):
    got = sort(E, ids, e)
    for a, r, what in zip(got, sort_ref(ids, e), ("order", "pos", "offsets")):
        np.testing.assert_array_equal(a.cpu().numpy(), r, err_msg=what)
    return got


@pytest.mark.parametrize("n,k,e,drop", [
    (0, 2, 8, 0), (1, 1, 1, 0), (1, 2, 8, 0), (3, 16, 1024, 0.3), (31, 3, 5, 0.5), (2048, 2, 7, 0.1),
    (2049, 2, 8, 0), (4095, 1, 1024, 0.2), (4097, 3, 33, 0.05), (70001, 4, 128, 0.02),
    (300007, 2, 3, 0), (262144, 8, 1024, 0.3), (5000, 1, 1, 0)])
def test_sort_matches_stable_sort(E, n, k, e, drop):
    g = gen(n + k)
    ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
    ids = (ids.float() ** 2 / max(1, e)).long()  # skewed to the low experts
    ids = ids.masked_fill(torch.rand((n, k), generator=g, device="cuda") < drop, -1)
    check_sort(E, ids, e)


def test_sort_odd_ids(E):
    """Ids far outside the range drop their slots, and one expert may take every slot or none."""
    ids = torch.tensor([[0, 7], [8, -1], [2 ** 40, -2 ** 63], [2 ** 63 - 1, 2 ** 32], [7, 7]], device="cuda")
    check_sort(E, ids, 8)
    check_sort(E, torch.full((9000, 2), 3, device="cuda"), 8)
    check_sort(E, torch.full((9000, 2), -1, device="cuda"), 8)


# ---- dispatch, combine and their gradients ----

SHAPES = [  # n, k, d, e, drop, pad, skip
    (1, 1, 1, 2, 0, 0, 0), (1, 2, 128, 8, 0, 0, 0), (5, 3, 7, 4, 0.4, 0, 0), (33, 4, 8, 5, 0.2, 8, 0),
    (100, 2, 479, 6, 0.1, 1, 0), (64, 5, 512, 9, 0.1, 0, 0), (17, 8, 130, 70, 0.5, 3, 1),
    (9, 16, 2056, 40, 0.3, 0, 0), (257, 1, 64, 3, 0.9, 64, 64), (40, 3, 5000, 8, 0.1, 0, 0),
    (12, 6, 1000, 3, 1.0, 0, 0)]


def routed(E, n, k, e, drop, g):
    ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
    ids = ids.masked_fill(torch.rand((n, k), generator=g, device="cuda") < drop, -1)
    if n > 2:
        ids[n // 2] = -1  # a row that no expert takes
    return ids, sort(E, ids, e)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,d,e,drop,pad,skip", SHAPES)
def test_dispatch_and_gradient(E, n, k, d, e, drop, pad, skip, dtype):
    g, t = gen(n * 7 + d), TYPES[dtype]
    ids, (order, pos, off) = routed(E, n, k, e, drop, g)
    x = rows(g, n, d, t, pad, skip)
    xs, full = room(n * k, d, t, pad, skip)
    E.expert_dispatch(x, pos, xs)
    ref = x[order.long() // k].clone()
    ref[int(off[-1]):] = 0
    assert torch.equal(xs, ref)
    outside_untouched(full, d, skip)

    dxs = rows(g, n * k, d, t, pad, skip)
    dxs[int(off[-1]):] = float("nan")  # what dropped places hold is not read
    dx, full = room(n, d, t, pad, skip)
    E.expert_dispatch_backward(dxs, pos, dx)
    p = pos.long().reshape(n, k)
    each = torch.where((p >= 0)[..., None], dxs.double()[p.clamp_min(0)], 0.0)
    within(dx, each.sum(1), (k + 2) * U32 * each.abs().sum(1), "dx")
    outside_untouched(full, d, skip)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,k,d,e,drop,pad,skip", SHAPES)
def test_combine_and_gradient(E, n, k, d, e, drop, pad, skip, dtype):
    g, t = gen(n * 5 + d), TYPES[dtype]
    ids, (order, pos, off) = routed(E, n, k, e, drop, g)
    kept = int(off[-1])
    p = pos.long().reshape(n, k)
    ys = rows(g, n * k, d, t, pad, skip)
    w = torch.rand((n, k), generator=g, device="cuda")
    ys[kept:] = float("inf")
    w[p < 0] = float("nan")
    out, full = room(n, d, t, pad, skip)
    E.expert_combine(ys, pos, w, out)
    on = (p >= 0)[..., None]
    each = torch.where(on, ys.double()[p.clamp_min(0)] * w.double()[..., None], 0.0)
    within(out, each.sum(1), (k + 2) * U32 * each.abs().sum(1), "out")
    outside_untouched(full, d, skip)

    dout = rows(g, n, d, t, pad, skip)
    dys, full = room(n * k, d, t, pad, skip)
    dw = torch.full((n, k), 77.0, device="cuda")
    E.expert_combine_backward(dout, ys, pos, w, dys, dw)
    ref = torch.zeros((n * k, d), dtype=torch.float64, device="cuda")
    tok = order[:kept].long() // k
    ref[:kept] = dout.double()[tok] * w.double().reshape(-1)[order[:kept].long()][:, None]
    within(dys, ref, U32 * ref.abs(), "dys")
    outside_untouched(full, d, skip)
    prod = torch.where(on, ys.double()[p.clamp_min(0)] * dout.double()[:, None], 0.0)
    within(dw, prod.sum(2), (d + 2) * U32 * prod.abs().sum(2), "dw")
    assert bool((dw[p < 0] == 0).all())


def test_expert_gradients_against_differences(E):
    """L = sum(c * combine(dispatch(x) * a)) is linear in x and in w: a step's difference is the
    gradient's product with it, up to the roundings of the two fp32 forwards."""
    n, k, d, e = 37, 3, 24, 5
    g = gen(3)
    ids, (order, pos, off) = routed(E, n, k, e, 0.2, g)
    x, vx = rows(g, n, d, torch.float32), rows(g, n, d, torch.float32)
    w, vw = torch.rand((n, k), generator=g, device="cuda"), torch.rand((n, k), generator=g, device="cuda")
    a, c = rows(g, n * k, d, torch.float32), rows(g, n, d, torch.float32)

    def forward(x, w):
        xs, out = torch.empty((n * k, d), device="cuda"), torch.empty((n, d), device="cuda")
        E.expert_dispatch(x, pos, xs)
        ys = xs * a
        E.expert_combine(ys, pos, w, out)
        return ys, (out.double() * c.double()).sum().item(), (out.double() * c.double()).abs().sum().item()

    ys, l0, mag = forward(x, w)
    dys, dw, dx = torch.empty_like(ys), torch.empty_like(w), torch.empty_like(x)
    E.expert_combine_backward(c, ys, pos, w, dys, dw)
    E.expert_dispatch_backward(dys * a, pos, dx)
    up, _, mu = 1, 0, 0
    lx, lw = forward(x + vx, w), forward(x, w + vw)
    # roundings: step, product, k sums and output of each forward, d-term and n-term gradients
    tol = (d + n + 4 * k + 20) * U32
    sx = (dx.double() * vx.double()).sum().item()
    assert abs(lx[1] - l0 - sx) <= tol * (lx[2] + mag + (dx.double() * vx.double()).abs().sum().item()) * k
    sw = (dw.double() * vw.double()).sum().item()
    assert abs(lw[1] - l0 - sw) <= tol * (lw[2] + mag + (dw.double() * vw.double()).abs().sum().item()) * k


def test_expert_rows_past_32_bit_offsets(E):
    """Rows 2^20 elements apart and more than 2^31 elements in all."""
    n, k, d, step = 1100, 2, 64, 1 << 20
    g = gen(8)
    ids, (order, pos, off) = routed(E, n, k, 4, 0.1, g)
    big = torch.empty((n * k, step), dtype=torch.bfloat16, device="cuda")
    x, xs = rows(g, n, d, torch.bfloat16), big[:, step - d:]
    E.expert_dispatch(x, pos, xs)
    ref = x[order.long() // k].clone()
    ref[int(off[-1]):] = 0
    assert torch.equal(xs, ref)
    out, w = torch.empty_like(x), torch.ones((n, k), device="cuda")
    E.expert_combine(xs, pos, w, out)
    p = pos.long().reshape(n, k)
    within(out, x.double() * (p >= 0).sum(1, keepdim=True), 4 * U32 * x.double().abs(), "out")
    E.expert_combine_backward(x, xs, pos, w, xs.new_empty((n * k, d)), dw := torch.empty_like(w))
    ref = torch.where(p >= 0, (x.double() ** 2).sum(1, keepdim=True), 0.0)
    within(dw, ref, (d + 2) * U32 * ref, "dw")


def test_broadcast_input_rows(E):
    """An expanded gradient (row step 0) is an ordinary input."""
    n, k, d = 50, 2, 40
    g = gen(9)
    ids, (order, pos, off) = routed(E, n, k, 4, 0.1, g)
    one = rows(g, 1, d, torch.float32)
    w, ys = torch.rand((n, k), generator=g, device="cuda"), rows(g, n * k, d, torch.float32)
    a, b = torch.empty((n * k, d), device="cuda"), torch.empty((n * k, d), device="cuda")
    da, db = torch.empty_like(w), torch.empty_like(w)
    E.expert_combine_backward(one.expand(n, d), ys, pos, w, a, da)
    E.expert_combine_backward(one.repeat(n, 1), ys, pos, w, b, db)
    assert torch.equal(a, b) and torch.equal(da, db)


# ---- gated norm ----

NORMS = [  # n, d, gate, pad, skip
    (1, 1, "full", 0, 0), (3, 2, "row", 0, 0), (7, 3, "none", 0, 0), (19, 8, "full", 0, 0),
    (33, 17, "row", 5, 1), (40, 64, "full", 0, 0), (700, 128, "none", 8, 0), (300, 479, "full", 0, 0),
    (65, 480, "row", 32, 32), (50, 512, "full", 0, 0), (2, 1000, "row", 0, 0), (1300, 1024, "full", 0, 0),
    (21, 2047, "full", 0, 0), (20, 2048, "none", 0, 0), (9, 2056, "row", 0, 0), (6, 4096, "full", 0, 0),
    (5, 4100, "full", 4, 0), (4, 8191, "row", 0, 0), (11, 8192, "full", 0, 0)]


def norm_case(n, d, gate, xt, bt, pad, skip, seed):
    g = gen(seed)
    s = dict(x=rows(g, n, d, xt, pad, skip, 2.0), y=rows(g, n, d, bt, pad, skip, 0.7),
             dx_out=rows(g, n, d, xt, pad, skip), dh=rows(g, n, d, bt, pad, skip))
    s["gate"] = None if gate == "none" else rows(g, n, d if gate == "full" else 1, bt, pad, skip, 2.0)
    for name, mean in (("w_post", 1.0), ("res_scale", 0.3), ("w_pre", 1.0)):
        s[name] = mean + 0.2 * torch.randn(d, generator=g, device="cuda")
    return s


def norm_ref(s, eps):
    """x_out and h with their error bounds."""
    d = s["x"].shape[1]
    c = (d / 2 + 40) * U32
    x, y = s["x"].double(), s["y"].double()
    ones = torch.ones(d, dtype=torch.float64, device="cuda")
    wp, rs, wq = (ones if s[k] is None else s[k].double() for k in ("w_post", "res_scale", "w_pre"))
    g = 1.0 if s["gate"] is None else torch.sigmoid(s["gate"].double())
    term = rs * g * y * torch.rsqrt((y * y).mean(1, keepdim=True) + eps) * wp
    xo = x + term
    ex = c * (x.abs() + term.abs())
    r = torch.rsqrt((xo * xo).mean(1, keepdim=True) + eps)
    h = xo * r * wq
    rel = (ex * ex).sum(1, keepdim=True).sqrt() / (xo * xo).sum(1, keepdim=True).sqrt().clamp_min(1e-300)
    return xo, ex, h, wq.abs() * r * ex + h.abs() * (c + rel)


@pytest.mark.parametrize("xt,bt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,d,gate,pad,skip", NORMS)
def test_gated_norm(E, n, d, gate, pad, skip, xt, bt):
    xt, bt = TYPES[xt], TYPES[bt]
    s = norm_case(n, d, gate, xt, bt, pad, skip, n + d)
    vec = {k: s[k] for k in ("gate", "w_post", "res_scale", "w_pre")}
    xo, fx = room(n, d, xt, pad, skip)
    h, fh = room(n, d, bt, pad, skip)
    E.gated_norm(s["x"], s["y"], xo, h, eps=1e-5, **vec)
    rx, ex, rh, eh = norm_ref(s, 1e-5)
    within(xo, rx, ex, "x_out")
    within(h, rh, eh, "h")
    outside_untouched(fx, d, skip)
    outside_untouched(fh, d, skip)
    # in place, and x_out alone
    again = s["x"].clone()
    E.gated_norm(again, s["y"], again, None, eps=1e-5, **vec)
    assert torch.equal(again, xo)
    # h alone, from the residual stream as it is
    E.gated_norm(s["x"], None, None, h, w_pre=s["w_pre"], eps=1e-5)
    x = s["x"].double()
    ref = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * s["w_pre"].double()
    within(h, ref, (d / 2 + 40) * U32 * ref.abs(), "h alone")


def norm_grad_ref(s, eps):
    """The gradients in 64 bits with their error bounds: {name: (value, bound)}."""
    n, d = s["x"].shape
    c = (d + 60) * U32
    x, y = s["x"].double(), s["y"].double()
    zero = torch.zeros((), dtype=torch.float64, device="cuda")
    dxo = zero if s["dx_out"] is None else s["dx_out"].double()
    dh = zero if s["dh"] is None else s["dh"].double()
    ones = torch.ones(d, dtype=torch.float64, device="cuda")
    wp, rs, wq = (ones if s[k] is None else s[k].double() for k in ("w_post", "res_scale", "w_pre"))
    mean = lambda v: v.mean(1, keepdim=True)
    rx, ry = torch.rsqrt(mean(x * x) + eps), torch.rsqrt(mean(y * y) + eps)
    q, a = x * rx, y * ry
    g = torch.ones_like(x[:, :1]) if s["gate"] is None else torch.sigmoid(s["gate"].double())
    rest = 1 - g if s["gate"] is None else torch.sigmoid(-s["gate"].double())
    dq = (dh * wq).expand_as(x)
    t = dxo + rx * (dq - q * mean(dq * q))
    mt = dxo.abs() + rx * (dq.abs() + q.abs() * mean((dq * q).abs()))
    et = c * mt
    f = (rs * wp).abs() * g
    u, eu = t * rs * wp * g, f * et
    um = mean(u * a)
    eum = mean(a.abs() * eu) + c * mean(f * mt * a.abs())
    dy = ry * (u - a * um)
    edy = ry * (eu + a.abs() * eum + c * (f * mt + a.abs() * mean(f * mt * a.abs())))
    dg, edg = u * a * rest, 2 * f * et * a.abs() * rest
    if s["gate"] is not None and s["gate"].shape[1] < d:
        dg, edg = dg.sum(1, keepdim=True), edg.sum(1, keepdim=True) + c * (f * mt * a.abs() * rest).sum(1, keepdim=True)
    many = (n + 4) * U32 + c
    T, eT = (t * g * a).sum(0), many * (mt * g * a.abs()).sum(0) + (et * g * a.abs()).sum(0)
    dpre = (dh * q).expand_as(x)
    return dict(dx=(t, et), dy=(dy, edy), dgate=(dg, edg), dw_post=(rs * T, rs.abs() * eT),
                dres_scale=(wp * T, wp.abs() * eT), dw_pre=(dpre.sum(0), many * dpre.abs().sum(0)))


def norm_grad(E, s, eps, pad=0, skip=0, names=("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre"), **kw):
    n, d = s["x"].shape
    xt, bt = s["x"].dtype, s["y"].dtype
    made = dict(dx=lambda: room(n, d, xt, pad, skip), dy=lambda: room(n, d, bt, pad, skip),
                dgate=lambda: room(n, s["gate"].shape[1], bt, pad, skip))
    out, full = {}, {}
    for k in ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre"):
        out[k] = None
        if k in names and not (k == "dgate" and s["gate"] is None):
            out[k], full[k] = made[k]() if k in made else (torch.full((d,), 77.0, device="cuda"), None)
    E.gated_norm_backward(s["dx_out"], s["dh"], s["x"], s["y"], out["dx"], out["dy"], gate=s["gate"],
                          w_post=s["w_post"], res_scale=s["res_scale"], w_pre=s["w_pre"], dgate=out["dgate"],
                          dw_post=out["dw_post"], dres_scale=out["dres_scale"], dw_pre=out["dw_pre"], eps=eps, **kw)
    for k in ("dx", "dy", "dgate"):
        if out[k] is not None:
            outside_untouched(full[k], out[k].shape[1], skip)
    return out


@pytest.mark.parametrize("xt,bt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("n,d,gate,pad,skip", NORMS)
def test_gated_norm_backward(E, n, d, gate, pad, skip, xt, bt):
    s = norm_case(n, d, gate, TYPES[xt], TYPES[bt], pad, skip, n * 3 + d)
    ref = norm_grad_ref(s, 1e-5)
    got = norm_grad(E, s, 1e-5, pad, skip)
    for k, v in got.items():
        if v is not None:
            within(v, *ref[k], k)
    again = norm_grad(E, s, 1e-5, pad, skip)
    for k, v in got.items():  # sums in a fixed order
        assert v is None or torch.equal(v, again[k]), k


@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("d", [24, 130, 1024])
def test_gated_norm_backward_parts(E, d, gate):
    """Missing inputs count as zeros or ones, missing outputs change no other, dx may be dx_out."""
    s = norm_case(45, d, gate, torch.float32, torch.float32, 0, 0, d)
    full = norm_grad(E, s, 1e-6)
    for names in (("dx",), ("dy", "dw_pre"), ("dw_post",), ("dgate", "dres_scale")):
        if gate == "none" and "dgate" in names:
            continue
        for k, v in norm_grad(E, s, 1e-6, names=names).items():
            assert v is None or torch.equal(v, full[k]), k
    dx = s["dx_out"].clone()
    E.gated_norm_backward(dx, s["dh"], s["x"], s["y"], dx, None, gate=s["gate"], w_post=s["w_post"],
                          res_scale=s["res_scale"], w_pre=s["w_pre"], eps=1e-6)
    assert torch.equal(dx, full["dx"])
    for missing in ("dx_out", "dh", "w_post", "res_scale", "w_pre"):
        m = {**s, missing: None}
        names = ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre")
        names = names[:-1] if missing == "dh" else names
        ref = norm_grad_ref(m, 1e-6)
        for k, v in norm_grad(E, m, 1e-6, names=names).items():
            if v is not None:
                within(v, *ref[k], f"{k} without {missing}")
    # no block: the norm before the next block alone
    dx, dpre = torch.empty_like(s["x"]), torch.empty(d, device="cuda")
    E.gated_norm_backward(s["dx_out"], s["dh"], s["x"], None, dx, None, w_pre=s["w_pre"], dw_pre=dpre, eps=1e-6)
    assert torch.equal(dx, full["dx"])
    within(dpre, *norm_grad_ref(s, 1e-6)["dw_pre"], "dw_pre")


@pytest.mark.parametrize("gate", ["none", "row", "full"])
def test_gated_norm_against_differences(E, gate):
    """Central differences of L = sum(c1 x_out) + sum(c2 h) along random directions.  With steps
    of size e = 2^-6 the error is e^2/6 of the third derivative (taken as at most 40 of the
    scale below) plus two forwards' roundings over 2 e."""
    n, d, e = 11, 48, 2.0 ** -6
    s = norm_case(n, d, gate, torch.float32, torch.float32, 0, 0, 5)
    s["dx_out"], s["dh"] = rows(gen(6), n, d, torch.float32), rows(gen(7), n, d, torch.float32)

    def loss(s):
        xo, h = torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda")
        E.gated_norm(s["x"], s["y"], xo, h, gate=s["gate"], w_post=s["w_post"], res_scale=s["res_scale"],
                     w_pre=s["w_pre"], eps=1e-2)
        a, b = xo.double() * s["dx_out"].double(), h.double() * s["dh"].double()
        return (a.sum() + b.sum()).item(), (a.abs().sum() + b.abs().sum()).item(), xo

    _, mag, xo = loss(s)
    got = norm_grad(E, {**s, "x": xo}, 1e-2)
    for name, grad in (("x", "dx"), ("y", "dy"), ("gate", "dgate"), ("w_post", "dw_post"),
                       ("res_scale", "dres_scale"), ("w_pre", "dw_pre")):
        if s[name] is None:
            continue
        v = torch.randn(s[name].shape, generator=gen(len(name)), device="cuda")
        up, down = {**s, name: s[name] + e * v}, {**s, name: s[name] - e * v}
        slope = (loss(up)[0] - loss(down)[0]) / (2 * e)
        dot = got[grad].double() * v.double()
        tol = e * e / 6 * 40 * mag + (d + 40) * U32 * mag / e
        assert abs(slope - dot.sum().item()) <= tol, (name, slope, dot.sum().item(), tol)


def test_gated_norm_odd_values(E):
    """Zero rows, saturated gates, and rows with infinities or NaN that touch no other row."""
    n, d = 24, 96
    s = norm_case(n, d, "full", torch.float32, torch.float32, 0, 0, 1)
    s["x"][0], s["y"][0], s["y"][1] = 0, 0, 0
    s["gate"][2], s["gate"][3] = float("inf"), float("-inf")
    s["gate"][4], s["gate"][5] = 200.0, -200.0
    clean = norm_ref(s, 1e-6)
    xo, h = torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda")
    vec = {k: s[k] for k in ("w_post", "res_scale", "w_pre")}
    E.gated_norm(s["x"], s["y"], xo, h, gate=s["gate"], **vec)
    within(xo, clean[0], clean[1], "x_out")
    within(h, clean[2], clean[3], "h")
    ref, got = norm_grad_ref(s, 1e-6), norm_grad(E, s, 1e-6)
    for k, v in got.items():
        within(v, *ref[k], k)
    s["x"][7, 5], s["y"][9, 50], s["gate"][11, 95] = float("nan"), float("inf"), float("nan")
    xo2, h2 = torch.empty_like(xo), torch.empty_like(h)
    E.gated_norm(s["x"], s["y"], xo2, h2, gate=s["gate"], **vec)
    keep = [i for i in range(n) if i not in (7, 9, 11)]
    assert torch.equal(xo2[keep], xo[keep]) and torch.equal(h2[keep], h[keep])
    assert h2[7].isnan().all() and h2[9].isnan().any() and h2[11].isnan().all()


def test_gated_norm_empty_batch(E):
    z = torch.empty((0, 40), device="cuda")
    E.gated_norm(z, z, z, z)
    dw = [torch.full((40,), 3.0, device="cuda") for _ in range(3)]
    E.gated_norm_backward(z, z, z, z, z, z, dw_post=dw[0], dres_scale=dw[1], dw_pre=dw[2])
    assert not any(bool(v.any()) for v in dw)


def test_gated_norm_rows_past_32_bit_offsets(E):
    n, d, step = 2200, 64, 1 << 20
    s = norm_case(n, d, "none", torch.bfloat16, torch.bfloat16, 0, 0, 4)
    big = torch.empty((n, step), dtype=torch.bfloat16, device="cuda")
    far = big[:, step - d:]
    far.copy_(s["y"])
    a, b = torch.empty_like(s["x"]), torch.empty_like(s["x"])
    E.gated_norm(s["x"], s["y"], a, None)
    E.gated_norm(s["x"], far, b, None)
    assert torch.equal(a, b)
    E.gated_norm(s["x"], s["y"], far, None)
    assert torch.equal(a, far)


# ---- gradient norm and clipping ----

def clip_ref(grads, m):
    norm = float(np.sqrt(sum(float((g.double() ** 2).sum()) for g in grads)))
    return norm, min(1.0, m / norm) if norm > 0 else 1.0


@pytest.mark.parametrize("sizes", [
    [1], [0], [], [3, 0, 5], [64, 64 * 64, 1], [16384, 16385, 2047], [1 << 20, 7, 250 * 250],
    [i % 37 for i in range(700)], [5_000_001, 3_333_333]])
@pytest.mark.parametrize("types", ["f32", "bf16", "mixed"])
def test_clip(E, sizes, types):
    g = gen(len(sizes))
    dt = lambda i: torch.bfloat16 if types == "bf16" or (types == "mixed" and i % 2) else torch.float32
    grads = [torch.randn(m, generator=g, device="cuda").to(dt(i)) for i, m in enumerate(sizes)]
    norm = torch.full((1,), 77.0, device="cuda")
    for limit in (0.3, 1.5):
        full, _ = clip_ref(grads, 1.0)
        m = float(np.float32(limit * full)) if full else 1.0
        ref, c = clip_ref(grads, m)
        out = [torch.full_like(x, 77.0) for x in grads]
        E.clip_grads(grads, m, norm, out=out)
        # at most 32 squares a group in fp32, fp64 beyond: 34 u, half of it after the root
        assert abs(norm.item() - ref) <= 20 * U32 * ref
        for x, o in zip(grads, out):
            within(o, x.double() * c, 24 * U32 * c * x.double().abs(), "out")
            assert c < 1 or torch.equal(o, x)
        here = [x.clone() for x in grads]
        n2 = torch.empty(1, device="cuda")
        E.clip_grads(here, m, n2)
        assert torch.equal(n2, norm) and all(torch.equal(a, b) for a, b in zip(here, out))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1e30, 1e-30, 1e18, 1e-20, 1e-38])
def test_clip_scales_far_from_one(E, scale, dtype):
    """Squares that leave fp32's range do not cost the norm."""
    g = gen(2)
    grads = [(torch.randn(m, generator=g, device="cuda", dtype=torch.float64) * scale).to(TYPES[dtype])
             for m in (1000, 33333, 5)]
    grads.append(torch.zeros(4096, dtype=TYPES[dtype], device="cuda"))
    norm = torch.empty(1, device="cuda")
    full, _ = clip_ref(grads, 1.0)
    m = float(np.float32(full / 4))
    ref, c = clip_ref(grads, m)
    out = [torch.empty_like(x) for x in grads]
    E.clip_grads(grads, m, norm, out=out)
    assert abs(norm.item() - ref) <= 20 * U32 * ref
    for x, o in zip(grads, out):
        within(o, x.double() * c, 24 * U32 * c * x.double().abs(), "out")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_clip_leaves_bad_gradients(E, bad):
    grads = [torch.randn(5000, device="cuda"), torch.randn(70, device="cuda")]
    grads[0][4321] = bad
    keep = [x.clone() for x in grads]
    norm = torch.zeros(1, device="cuda")
    E.clip_grads(grads, 1.0, norm)
    assert not norm.isfinite().any() and (norm.isnan().item() if bad != bad else norm.isinf().item())
    for a, b in zip(grads, keep):
        assert torch.equal(a.view(torch.int32), b.view(torch.int32))
    big = [torch.full((100,), 3e38, device="cuda")]  # finite, but its norm is not in fp32
    E.clip_grads(big, 1.0, norm)
    assert norm.isinf().item() and bool((big[0] == 3e38).all())


def test_clip_limits_and_alignment(E):
    flat = torch.randn(100_003, device="cuda")
    half = flat.bfloat16()
    grads = [flat[1:50_001], flat[50_002:], half[3:40_004], half[40_005:]]
    keep = [x.clone() for x in grads]
    norm = torch.empty(1, device="cuda")
    E.clip_grads(grads, float("inf"), norm)
    ref, _ = clip_ref(keep, 1.0)
    assert abs(norm.item() - ref) <= 20 * U32 * ref
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    e = [flat[0].item(), half[40_004].item()]
    E.clip_grads(grads, 1.0, norm)
    _, c = clip_ref(keep, 1.0)
    for a, b in zip(grads, keep):
        within(a, b.double() * c, 24 * U32 * c * b.double().abs(), "in place")
    assert [flat[0].item(), half[40_004].item()] == e  # between the tensors
    E.clip_grads(grads, 0.0, norm)
    assert not any(bool(a.any()) for a in grads)


# ---- streams and repeatability ----

def test_calls_on_another_stream(E):
    """Calls on a side stream, with their own workspaces, behind work queued on it."""
    g = gen(12)
    n, k, e, d = 9000, 4, 16, 64
    ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
    s = norm_case(n, d, "full", torch.float32, torch.float32, 0, 0, 3)
    grads = [torch.randn(300_000, generator=g, device="cuda")]
    a_sort, a_norm = sort(E, ids, e), norm_grad(E, s, 1e-6)
    a_clip, a_n = [torch.empty_like(grads[0])], torch.empty(1, device="cuda")
    E.clip_grads(grads, 1.0, a_n, out=a_clip)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        filler = torch.randn((4096, 4096), device="cuda")
        for _ in range(4):
            filler = filler @ filler * 1e-3
        late_ids, late_dh, late_g = ids + 0, s["dh"] * 1, [grads[0] * 1]
        b_sort = sort(E, late_ids, e, stream=side)
        b_norm = norm_grad(E, {**s, "dh": late_dh}, 1e-6, stream=side)
        b_clip, b_n = [torch.empty_like(grads[0])], torch.empty(1, device="cuda")
        E.clip_grads(late_g, 1.0, b_n, out=b_clip, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a_sort, b_sort))
    assert all(v is None or torch.equal(v, b_norm[k]) for k, v in a_norm.items())
    assert torch.equal(a_clip[0], b_clip[0]) and torch.equal(a_n, b_n)


def test_calls_in_a_graph(E):
    """Captured once, replayed on new contents of the same buffers."""
    g = gen(13)
    n, k, e, d = 5000, 2, 8, 128
    ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
    x, w = rows(g, n, d, torch.bfloat16), torch.rand((n, k), generator=g, device="cuda")
    order, pos = (torch.empty(n * k, dtype=torch.int32, device="cuda") for _ in range(2))
    off = torch.empty(e + 1, dtype=torch.int32, device="cuda")
    xs, out, norm = torch.empty((n * k, d), dtype=x.dtype, device="cuda"), torch.empty_like(x), torch.empty(1, device="cuda")
    ws = [torch.empty(max(16, b), dtype=torch.uint8, device="cuda")
          for b in (E.expert_sort_workspace(n, k, e), E.clip_grads_workspace(1))]

    def step():
        E.expert_sort(ids, e, order, pos, off, workspace=ws[0])
        E.expert_dispatch(x, pos, xs)
        E.expert_combine(xs, pos, w, out)
        E.clip_grads([out], 1.0, norm, workspace=ws[1])

    step()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step()
    ids.copy_(torch.randint(-1, e, (n, k), generator=g, device="cuda"))
    x.copy_(rows(g, n, d, torch.bfloat16))
    graph.replay()
    got = [v.clone() for v in (order, pos, off, xs, out, norm)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (order, pos, off, xs, out, norm)))


def test_workspace_contents_do_not_matter(E):
    g = gen(14)
    ids = torch.randint(0, 9, (9000, 3), generator=g, device="cuda")
    s = norm_case(500, 256, "row", torch.bfloat16, torch.bfloat16, 0, 0, 3)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda")
    for a, b in zip(sort(E, ids, 9, workspace=ws), sort(E, ids, 9)):
        assert torch.equal(a, b)
    a, b = norm_grad(E, s, 1e-6, workspace=ws), norm_grad(E, s, 1e-6)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_calls_between_other_work(E):
    """Calls queued back to back with torch's kernels and copies before, between and after them, on
    buffers that are written again every round, give what the same work gives with a wait after
    every step."""
    n, k, e, d = 700, 3, 9, 96
    g = gen(21)
    ids0 = torch.randint(-1, e, (n, k), generator=g, device="cuda")
    base = rows(g, n, d, torch.float32)
    host = torch.randn(n, d).pin_memory()

    def run(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        x, h, xs = torch.empty_like(base), torch.empty_like(base), torch.empty((n * k, d), device="cuda")
        ids, y, out = torch.empty_like(ids0), torch.empty_like(base), []
        w = torch.full((n, k), 1.0 / k, device="cuda")
        order, pos = (torch.empty(n * k, dtype=torch.int32, device="cuda") for _ in range(2))
        off, norm = torch.empty(e + 1, dtype=torch.int32, device="cuda"), torch.empty(1, device="cuda")
        dw = torch.empty(d, device="cuda")
        for r in range(12):
            steps = [
                lambda: x.copy_(host, non_blocking=True),
                lambda: x.add_(base * r),
                lambda: E.gated_norm(x, None, None, h),
                lambda: ids.copy_((ids0 + r) % (e + 1) - 1),
                lambda: E.expert_sort(ids, e, order, pos, off),
                lambda: E.expert_dispatch(h, pos, xs),
                lambda: xs.mul_(1.5),
                lambda: E.expert_combine(xs, pos, w, y),
                lambda: E.gated_norm(x, y, x, h),
                lambda: E.gated_norm_backward(x, h, x, y, x, y, dw_post=dw),
                lambda: E.clip_grads([x, y, dw], 3.0, norm),
                lambda: out.append(torch.cat([x.flatten(), y.flatten(), h.flatten(), dw, norm])),
                lambda: x.zero_(),
            ]
            for s in steps:
                s()
                pause()
        torch.cuda.synchronize()
        return out

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_graph_with_other_work_and_streams(E):
    """A captured step with copies, fills, torch kernels and a forked stream between the calls."""
    g = gen(22)
    n, d = 513, 120
    src, x, h = rows(g, n, d, torch.bfloat16), torch.empty((n, d), dtype=torch.bfloat16, device="cuda"), torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    z, dw, norm = torch.empty_like(h), torch.empty(d, device="cuda"), torch.empty(1, device="cuda")
    side = torch.cuda.Stream()

    def step():
        x.copy_(src)
        E.gated_norm(x, None, None, h)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            z.copy_(h)
            E.gated_norm(z, src, z, None)
        dw.zero_()
        E.gated_norm_backward(x, h, x, None, x, None, dw_pre=dw)
        torch.cuda.current_stream().wait_stream(side)
        E.clip_grads([x, z, dw], 0.5, norm)
        x.add_(z)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    src.copy_(rows(g, n, d, torch.bfloat16))
    graph.replay()
    got = [v.clone() for v in (x, z, h, dw, norm)]
    step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, (x, z, h, dw, norm)))


@pytest.mark.parametrize("n,k,e", [
    (2048, 1, 9), (2049, 1, 9), (4096, 1, 1024), (4097, 1, 1024), (1025, 16, 300), (32768, 2, 64),
    (32769, 2, 64), (20000, 16, 128), (155648, 8, 255), (155649, 8, 256), (1_100_000, 8, 40),
    (1_100_000, 8, 900)])
def test_sort_where_its_launches_change(E, n, k, e):
    """Sizes on either side of one CTA of few warps, one CTA, two launches and three, and chunks too
    large for registers."""
    g = gen(n + e)
    ids = torch.randint(0, e, (n, k), generator=g, device="cuda")
    ids = ids.masked_fill(torch.rand((n, k), generator=g, device="cuda") < 0.1, -1)
    ids[: n // 3] = ids[: n // 3] % 3  # a few crowded experts
    check_sort(E, ids, e)


@pytest.mark.parametrize("n,d", [(1, 64), (95 * 32, 64), (97 * 32, 64), (16 * 6 * 2, 1024), (16 * 6 * 2 + 1, 1024),
                                 (96, 8192), (97, 8192)])
def test_gated_norm_backward_where_its_launches_change(E, n, d):
    """Rows that take one CTA, one CTA an SM and more, with and without the vectors' gradients."""
    s = norm_case(n, d, "full", torch.float32, torch.bfloat16, 0, 0, n)
    ref, got = norm_grad_ref(s, 1e-6), norm_grad(E, s, 1e-6)
    for k, v in got.items():
        within(v, *ref[k], k)
    for k, v in norm_grad(E, s, 1e-6, names=("dx", "dy")).items():
        assert v is None or torch.equal(v, got[k]), k
    ws = torch.empty(max(16, E.gated_norm_backward_workspace(n, d)), dtype=torch.uint8, device="cuda")
    for k, v in norm_grad(E, s, 1e-6, workspace=ws).items():
        assert torch.equal(v, got[k]), k


@pytest.mark.parametrize("total,count", [(1048576, 3), (1048577, 3), (5000, 256), (5000, 257)])
def test_clip_where_its_launches_change(E, total, count):
    """Lists that cut a tensor range at random places, on either side of what one launch takes."""
    g = gen(count)
    cut = sorted(torch.randint(0, total + 1, (count - 1,), generator=g, device="cuda").tolist())
    sizes = [b - a for a, b in zip([0] + cut, cut + [total])]
    grads = [torch.randn(m, generator=g, device="cuda") for m in sizes]
    norm, out = torch.empty(1, device="cuda"), [torch.empty_like(x) for x in grads]
    E.clip_grads(grads, 2.0, norm, out=out)
    ref, c = clip_ref(grads, 2.0)
    assert abs(norm.item() - ref) <= 20 * U32 * ref
    for x, o in zip(grads, out):
        within(o, x.double() * c, 24 * U32 * c * x.double().abs(), "out")
