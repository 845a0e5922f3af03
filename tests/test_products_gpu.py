"""The experts' products on the GPU against their definitions in 64 bits: the grouped linear layer and
the gated block in both directions, over types, layouts, odd widths, empty and one-row experts, rows
of no expert, and NaN in rows that a call has no business with.

Tolerances.  A result in type t is rounded once: eps(t) / 2 of its value.  Before that, a sum of K
products is off by at most K 2^-23 of the sum of their magnitudes, in whatever order and however each
addition is rounded (2^-23 is a whole step of fp32).  fp32 operands are split so that what is left out of
a product is below 2^-22 of it (two pairs of parts below 2^-8 2^-16 times at most two, and the third part's
rounding).  The gated backward rounds [dg, du] to bf16 for bf16 calls: eps / 2 of each product's magnitude.
Beside the bound of each element, fp32 results' distance in the 2-norm is held to 2^-20 of the
magnitudes': single elements' worst cases do not add up."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
NAMES = {F32: "f32", BF16: "bf16"}


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def rows(n, d, dtype, g, pad=0, shift=0, scale=1.0):
    """n rows of normal values in rows of d + pad, starting `shift` elements into the storage."""
    flat = torch.full((n * (d + pad) + shift,), float("nan"), device="cuda").to(dtype)
    m = flat[shift:].view(n, d + pad)[:, :d]
    m.copy_(torch.randn((n, d), generator=g, device="cuda") * scale)
    return m


def weights(e, o, i, dtype, g, order="oi", pad=0):
    w = torch.randn((e, o, i), generator=g, device="cuda") / math.sqrt(i)
    if order == "io":  # [e, in, out + pad], turned
        store = torch.full((e, i, o + pad), float("nan"), device="cuda", dtype=dtype)
        store[:, :, :o] = w.transpose(1, 2)
        return store[:, :, :o].transpose(1, 2)
    if order == "among":  # rows of all experts in turn
        store = torch.full((o, e, i + pad), float("nan"), device="cuda", dtype=dtype)
        store[:, :, :i] = w.transpose(0, 1)
        return store[:, :, :i].transpose(0, 1)
    store = torch.full((e, o, i + pad), float("nan"), device="cuda", dtype=dtype)
    store[:, :, :i] = w
    return store[:, :, :i]


def offsets_of(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def close(got, want, mag, K, extra=0.0, split=False):
    """Every element within its bound, and for fp32 the whole within 2^-20 of the magnitudes."""
    got, t = got.double(), got.dtype
    bound = torch.finfo(t).eps / 2 * want.abs() + (K * 2.0 ** -23 + (2.0 ** -22 if split else 0.0) + extra) * mag + 1e-30
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {((got - want).abs() / bound).max().item():.3g} of its bound"
    if t == F32 and extra == 0.0:
        assert (got - want).norm() <= 2.0 ** -20 * mag.norm() + 1e-30


def by_expert(x, w, counts):
    """x W_e^T for each expert's rows, and the sums of magnitudes (64 bits)."""
    y = torch.zeros((x.shape[0], w.shape[1]), dtype=torch.float64, device="cuda")
    m = torch.zeros_like(y)
    lo = 0
    for e, c in enumerate(counts):
        a, b = x[lo:lo + c].double(), w[e].double()
        y[lo:lo + c], m[lo:lo + c] = a @ b.T, a.abs() @ b.abs().T
        lo += c
    return y, m


def by_rows(a, b, counts):
    """a[rows]^T b[rows] of each expert, and the sums of magnitudes."""
    y = torch.zeros((len(counts), a.shape[1], b.shape[1]), dtype=torch.float64, device="cuda")
    m = torch.zeros_like(y)
    lo = 0
    for e, c in enumerate(counts):
        p, q = a[lo:lo + c].double(), b[lo:lo + c].double()
        y[e], m[e] = p.T @ q, p.abs().T @ q.abs()
        lo += c
    return y, m


# counts of rows, rows of no expert behind them, in, out, weight layout, padding of rows, start in the storage
SHAPES = [
    ([1], 0, 64, 64, "oi", 0, 0),
    ([128], 0, 128, 256, "oi", 0, 0),
    ([3, 0, 1, 5], 2, 64, 96, "oi", 0, 0),
    ([3, 0, 1, 5], 2, 64, 96, "io", 0, 0),
    ([0, 0, 7], 0, 8, 8, "io", 0, 0),
    ([257, 255, 256, 0, 1], 40, 200, 264, "oi", 8, 0),
    ([257, 255, 256, 0, 1], 40, 200, 264, "io", 8, 0),
    ([300, 500], 3, 479, 351, "oi", 33, 1),
    ([300, 500], 3, 479, 351, "io", 33, 1),
    ([70, 65, 64, 63], 0, 1, 1, "oi", 0, 0),
    ([70, 65, 64, 63], 0, 3, 130, "io", 0, 3),
    ([511], 0, 1030, 17, "oi", 0, 0),
    ([40] * 30, 9, 72, 520, "among", 0, 0),
    ([2049, 30], 1, 320, 384, "oi", 0, 0),
    ([20, 30, 0, 14], 2, 72, 40, "oi", 0, 0),
    ([20, 30, 0, 14], 2, 72, 40, "io", 0, 0),
    ([0, 60, 0, 3], 1, 479, 33, "io", 5, 1),
    ([31], 0, 1030, 130, "io", 0, 0),
    ([31], 0, 1030, 130, "oi", 0, 0),
    ([1, 0, 2] * 15, 4, 256, 72, "oi", 0, 0),
    ([9000, 11003], 5, 136, 640, "oi", 0, 0),
    ([7000, 13003], 5, 640, 136, "io", 8, 0),
]
IDS = [f"{len(s[0])}x{sum(s[0])}+{s[1]}-{s[2]}-{s[3]}-{s[4]}" for s in SHAPES]


def setup(shape, dtype, seed, halves=1):
    counts, rest, i, o, order, pad, shift = shape
    g = gen(seed)
    S = sum(counts) + rest
    x = rows(S, i, dtype, g, pad, shift)
    w = weights(len(counts), halves * o, i, dtype, g, order, pad)
    x[sum(counts):] = float("nan")  # what rows of no expert hold is nobody's business
    return counts, S, x, w, offsets_of(counts), g


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear(E, shape, dtype):
    counts, S, x, w, off, g = setup(shape, dtype, 1)
    out = rows(S, shape[3], dtype, g, shape[5], shape[6])
    before = out.clone()
    E.expert_linear(x, w, out, offsets=off)
    n = sum(counts)
    y, m = by_expert(x, w, counts)
    close(out[:n], y[:n], m[:n], shape[2], split=dtype == F32)
    assert torch.equal(out[n:], before[n:])


@pytest.mark.parametrize("dw_type", ["f32", "same"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear_backward(E, shape, dtype, dw_type):
    if dtype == F32 and dw_type == "same":
        pytest.skip("the same")
    counts, S, x, w, off, g = setup(shape, dtype, 2)
    n, i, o = sum(counts), shape[2], shape[3]
    dout = rows(S, o, dtype, g, shape[5], shape[6])
    dout[n:] = float("nan")
    dx = rows(S, i, dtype, g, shape[5])
    before = dx.clone()
    dw = torch.empty_like(weights(len(counts), o, i, dtype, g, shape[4]), dtype=F32 if dw_type == "f32" else dtype).fill_(float("nan"))
    E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
    y, m = by_expert(dout, w.transpose(1, 2), counts)
    close(dx[:n], y[:n], m[:n], o, split=dtype == F32)
    assert torch.equal(dx[n:], before[n:])
    y, m = by_rows(dout, x, counts)
    close(dw, y, m, max(counts), split=dtype == F32)
    # one of them alone is the same
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    E.expert_linear_backward(dout, x, w, dx2, None, offsets=off)
    E.expert_linear_backward(dout, x, w, None, dw2, offsets=off)
    assert torch.equal(dx2[:n], dx[:n]) and torch.equal(dw2, dw)


def act64(name, v):
    if name == "relu":
        return torch.where(v > 0, v, 0), (v > 0).double()
    if name == "gelu":
        p = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    s = torch.sigmoid(v)
    return (s, s * torch.sigmoid(-v)) if name == "sigmoid" else (v * s, s + v * s * torch.sigmoid(-v))


ACTS = ["silu", "gelu", "relu", "sigmoid"]


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated(E, shape, dtype, act):
    """h's bound: |act'| <= 1.13 and |act(v)| <= max(1, |v|) for all four, so an error of dg in g and du in u makes at
    most 1.13 |u| dg + max(1, |g|) du, and the fast exponential's 2^-17 (fp32: 2^-21) of the value more."""
    counts, S, x, w, off, g = setup(shape, dtype, 3, 2)
    n, f = sum(counts), shape[3]
    h, gu = rows(S, f, dtype, g, shape[5], shape[6]), rows(S, 2 * f, dtype, g, shape[5])
    before = h.clone(), gu.clone()
    E.expert_gated(x, w, h, gu=gu, offsets=off, act=act)
    y, m = by_expert(x, w, counts)
    y, m = y[:n], m[:n]
    close(gu[:n], y, m, shape[2], split=dtype == F32)
    a, u = act64(act, y[:, :f])[0], y[:, f:]
    off_by = shape[2] * 2.0 ** -23 + (2.0 ** -22 if dtype == F32 else 0)
    mag = 1.13 * u.abs() * m[:, :f] + y[:, :f].abs().clamp_min(1) * m[:, f:] + off_by * m[:, :f] * m[:, f:]
    fast = 2.0 ** -17 if dtype == BF16 else 2.0 ** -21
    bound = torch.finfo(dtype).eps / 2 * (a * u).abs() + off_by * mag + fast * u.abs() * (a.abs() + 1e-3) + 1e-30
    assert ((h[:n].double() - a * u).abs() <= bound).all()
    assert torch.equal(h[n:], before[0][n:]) and torch.equal(gu[n:], before[1][n:])
    h2 = torch.empty_like(h)
    E.expert_gated(x, w, h2, offsets=off, act=act)
    assert torch.equal(h2[:n], h[:n])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated_backward(E, shape, dtype, act):
    counts, S, x, w, off, g = setup(shape, dtype, 4, 2)
    n, i, f = sum(counts), shape[2], shape[3]
    dh, gu = rows(S, f, dtype, g, shape[5], shape[6]), rows(S, 2 * f, dtype, g, shape[5], scale=2.0)
    dh[n:], gu[n:] = float("nan"), float("nan")
    dx = rows(S, i, dtype, g)
    before = dx.clone()
    dw = torch.empty_like(w, dtype=F32).fill_(float("nan"))
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, act=act)
    a, slope = act64(act, gu[:, :f].double())
    d, u = dh.double(), gu[:, f:].double()
    dgu = torch.cat([d * u * slope, d * a], 1)
    # act and its slope are off by 2^-17 of max(1, |value|) (fp32: 2^-21), and the pair is rounded once for bf16
    rough = torch.cat([(d * u).abs(), d.abs() * gu[:, :f].double().abs().clamp_min(1)], 1)
    extra, fast = (2.0 ** -8, 2.0 ** -16) if dtype == BF16 else (0.0, 2.0 ** -20)
    y, m = by_expert(dgu, w.transpose(1, 2), counts)
    mr = by_expert(rough, w.transpose(1, 2), counts)[1]
    bound = lambda y, m, mr, K, t: (torch.finfo(t).eps / 2 * y.abs() + (K * 2.0 ** -23 + 2.0 ** -22 + extra) * m + fast * mr + 1e-30)
    assert ((dx[:n].double() - y[:n]).abs() <= bound(y, m, mr, 2 * f, dtype)[:n]).all()
    assert torch.equal(dx[n:], before[n:])
    y, m = by_rows(dgu, x, counts)
    mr = by_rows(rough, x, counts)[1]
    assert ((dw.double() - y).abs() <= bound(y, m, mr, max(counts), F32)).all()


@pytest.mark.parametrize("order", ["oi", "io"])
def test_gated_backward_in_parts(E, order):
    """Gradients in the weights' own type, rounded once more (of [dg, du] rounded to bf16: 2^-8 of each
    product), and dx and dw each alone."""
    g, counts = gen(12), [40, 0, 130]
    off, f, i = offsets_of(counts), 36, 50
    x, dh, gu = rows(170, i, BF16, g), rows(170, f, BF16, g), rows(170, 2 * f, BF16, g)
    w = weights(3, 2 * f, i, BF16, g, order)
    a, slope = act64("silu", gu[:, :f].double())
    dgu = torch.cat([dh.double() * gu[:, f:].double() * slope, dh.double() * a], 1)
    y, m = by_rows(dgu, x, counts)
    dw = torch.empty_like(w).fill_(float("nan"))
    dx = torch.empty_like(x)
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off)
    assert ((dw.double() - y).abs() <= 2.0 ** -8 * y.abs() + (2.0 ** -8 + 2.0 ** -15) * m + 1e-30).all()
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    E.expert_gated_backward(dh, gu, x, w, dx2, None, offsets=off)
    E.expert_gated_backward(dh, gu, x, w, None, dw2, offsets=off)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_most_experts(E, dtype):
    """1024 experts of no, one and a few rows, in both directions."""
    g = gen(13)
    counts = [(7 * i) % 5 for i in range(1024)]
    n, off = sum(counts), offsets_of(counts)
    x, dout, w = rows(n, 40, dtype, g), rows(n, 24, dtype, g), weights(1024, 24, 40, dtype, g)
    out, dx, dw = torch.empty_like(dout), torch.empty_like(x), torch.empty((1024, 24, 40), device="cuda")
    E.expert_linear(x, w, out, offsets=off)
    E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
    y, m = by_expert(x, w, counts)
    close(out, y, m, 40, split=dtype == F32)
    y, m = by_expert(dout, w.transpose(1, 2), counts)
    close(dx, y, m, 24, split=dtype == F32)
    y, m = by_rows(dout, x, counts)
    close(dw, y, m, 4, split=dtype == F32)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_calls_in_a_row_and_on_two_streams(E, dtype):
    """Calls that follow one another on one workspace, each kernel started early, and calls on two streams
    at once: the bits of calls by themselves."""
    g, counts = gen(14), [300, 0, 211, 77]
    off, f, i = offsets_of(counts), 48, 72
    sets = []
    for _ in range(3):
        x, dh, w = rows(588, i, dtype, g), rows(588, f, dtype, g), weights(4, 2 * f, i, dtype, g)
        room = [torch.zeros(s, device="cuda", dtype=t) for s, t in (((588, f), dtype), ((588, 2 * f), dtype), ((588, i), dtype), ((4, 2 * f, i), F32))]
        sets.append((x, dh, w, *room))

    def run(s, ws):
        x, dh, w, h, gu, dx, dw = s
        E.expert_gated(x, w, h, gu=gu, offsets=off, workspace=ws)
        E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, workspace=ws)

    alone = []
    for s in sets:
        run(s, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in s[3:]])
        for t in s[3:]:
            t.zero_()
    need = E.expert_gated_backward_workspace(sets[0][1], sets[0][4], sets[0][0], sets[0][2], sets[0][5], sets[0][6], offsets=off)
    spaces = [torch.empty(max(need, 1 << 20), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for s in sets:
            run(s, spaces[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for s, w in zip(sets, alone) for a, b in zip(s[3:], w))
    for s in sets:
        for t in s[3:]:
            t.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for k, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                run(sets[k], spaces[k])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for k in range(2) for a, b in zip(sets[k][3:], alone[k]))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_other_experts_rows_do_not_leak(E, dtype):
    """An expert whose rows, gradients and weights are NaN or infinite changes no other's results by a bit."""
    counts = [70, 33, 200]
    g = gen(5)
    x, dout = rows(303, 96, dtype, g), rows(303, 80, dtype, g)
    w, off = weights(3, 80, 96, dtype, g), offsets_of(counts)
    out, dx = rows(303, 80, dtype, g), rows(303, 96, dtype, g)
    dw = torch.empty((3, 80, 96), device="cuda")
    keep = torch.ones(303, dtype=torch.bool, device="cuda")
    keep[70:103] = False

    def all_of():
        E.expert_linear(x, w, out, offsets=off)
        E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
        return out[keep].clone(), dx[keep].clone(), dw[[0, 2]].clone()

    clean = all_of()
    assert all(v.isfinite().all() for v in clean)
    for bad in (float("nan"), float("inf")):
        x[70:103], dout[70:103], w[1] = bad, bad, bad
        dirty = all_of()
        assert all(torch.equal(p, q) for p, q in zip(clean, dirty))
        assert not out[70:103].isfinite().any() and not dx[70:103].isfinite().any() and not dw[1].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_no_rows(E, dtype):
    """No rows at all, or none kept: nothing is written but zero weight gradients."""
    w = torch.randn((3, 32, 16), device="cuda").to(dtype)
    w2 = torch.randn((3, 32, 16), device="cuda").to(dtype)
    for S in (0, 300):
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        x, out = torch.full((S, 16), float("nan"), device="cuda", dtype=dtype), torch.ones((S, 32), device="cuda", dtype=dtype)
        h, gu = torch.ones((S, 16), device="cuda", dtype=dtype), torch.ones((S, 32), device="cuda", dtype=dtype)
        E.expert_linear(x, w, out, offsets=off)
        E.expert_gated(x, w2, h, gu=gu, offsets=off)
        assert (out == 1).all() and (h == 1).all() and (gu == 1).all()
        dx, dw = torch.ones_like(x), torch.ones((3, 32, 16), device="cuda")
        E.expert_linear_backward(out, x, w, dx, dw, offsets=off)
        assert (dx == 1).all() and (dw == 0).all()
        dw = torch.ones((3, 32, 16), device="cuda", dtype=dtype)
        E.expert_gated_backward(h, gu, x, w2, dx, dw, offsets=off)
        assert (dx == 1).all() and (dw == 0).all()
        q, scale = torch.zeros((3, 32, 8), dtype=torch.uint8, device="cuda"), torch.ones((3, 32, 1), device="cuda")
        E.expert_linear4(x, q, scale, out, group=32, offsets=off)
        assert (out == 1).all()


def test_bad_offsets_stay_inside(E):
    """Offsets out of order or range: some results, inside the buffers (the neighbours' stay)."""
    g = gen(6)
    big = torch.zeros((900, 64), device="cuda", dtype=BF16)
    out = big[300:600]
    x, w = rows(300, 32, BF16, g), weights(4, 64, 32, BF16, g)
    dw = torch.empty((4, 64, 32), device="cuda")
    for off in ([0, 500, 100, 9000, 200], [-5, 100, 50, 300, 301], [400, 300, 200, 100, 0], [0, 2 ** 31 - 1, -2 ** 31, 7, 9]):
        o = torch.tensor(off, dtype=torch.int32, device="cuda")
        E.expert_linear(x, w, out, offsets=o)
        E.expert_linear_backward(out, x, w, None, dw, offsets=o)
        torch.cuda.synchronize()
        assert (big[:300] == 0).all() and (big[600:] == 0).all()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_dense_layer_split_over_rows(E, dtype):
    """One dense layer with few tiles of dw and many rows: its parts are summed in a fixed order."""
    g = gen(7)
    x, dout = rows(20011, 479, dtype, g, 33), rows(20011, 70, dtype, g)
    w = weights(1, 70, 479, dtype, g)[0]
    dw = torch.empty((70, 479), device="cuda")
    E.expert_linear_backward(dout, x, w, None, dw)
    y, m = by_rows(dout, x, [20011])
    close(dw[None], y, m, 20011, split=dtype == F32)
    again = torch.empty_like(dw)
    E.expert_linear_backward(dout, x, w, None, again)
    assert torch.equal(dw, again)


def test_broadcast_rows_and_weights(E):
    """Row step 0 (one row for all), and one matrix for every expert."""
    g = gen(8)
    x = rows(1, 40, BF16, g).expand(300, 40)
    w = weights(1, 24, 40, BF16, g).expand(3, 24, 40)
    off, out = offsets_of([100, 0, 200]), torch.empty((300, 24), device="cuda", dtype=BF16)
    E.expert_linear(x, w, out, offsets=off)
    y, m = by_expert(x, w, [100, 0, 200])
    close(out, y, m, 40)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
def test_elements_past_2_31(E, dtype):
    """Rows whose elements lie beyond 2^31 of the storage's start."""
    step, S = 1 << 20, 2100
    g = gen(9)
    store = torch.empty(step * S, device="cuda", dtype=dtype)
    x = store.view(S, step)[:, 128:192]
    out = store.view(S, step)[:, 1024:1056]
    x.copy_(torch.randn((S, 64), generator=g, device="cuda"))
    w = weights(2, 32, 64, dtype, g)
    counts = [50, 2050]
    E.expert_linear(x, w, out, offsets=offsets_of(counts))
    y, m = by_expert(x, w, counts)
    close(out, y, m, 64, split=dtype == F32)
    dw = torch.empty((2, 32, 64), device="cuda")
    E.expert_linear_backward(out, x, w, None, dw, offsets=offsets_of(counts))
    y, m = by_rows(out, x, counts)
    close(dw, y, m, 2050, split=dtype == F32)


def test_graph_streams_and_workspace(E):
    """Captured and replayed with other offsets, on a stream of its own, with the caller's workspace; the
    replays give a direct call's bits."""
    g = gen(10)
    x, w = rows(400, 100, BF16, g), weights(4, 2 * 60, 100, BF16, g)
    off = offsets_of([100, 100, 100, 100])
    h, gu, dx, dw = (torch.zeros(s, device="cuda", dtype=t) for s, t in
                     (((400, 60), BF16), ((400, 120), BF16), ((400, 100), BF16), ((4, 120, 100), F32)))
    dh = rows(400, 60, BF16, g)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        E.expert_gated(x, w, h, gu=gu, offsets=off, workspace=ws)
        E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for counts in ([400, 0, 0, 0], [1, 2, 3, 300], [0, 0, 0, 0], [17, 200, 83, 100]):
        off.copy_(offsets_of(counts))
        for t in (h, gu, dx, dw):
            t.fill_(7)
        graph.replay()
        got = [t.clone() for t in (h, gu, dx, dw)]
        for t in (h, gu, dx, dw):
            t.fill_(7)
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, (h, gu, dx, dw)))
        y, m = by_expert(x, w, counts)
        n = sum(counts)
        if n:
            close(gu[:n], y[:n], m[:n], 100)


def test_gradients_against_differences(E):
    """The gated block's and the linear layer's gradients against central differences of their own
    forward in fp32: a step of 2^-7 in one direction leaves an error of about 2^-14 (cube of the step, halved
    twice) and the forward's rounding over the step, about 2^-20 2^7; 2^-9 of the gradient's size holds both."""
    g = gen(11)
    counts, i, f, o = [9, 0, 14], 24, 20, 16
    off = offsets_of(counts)
    x, w1, w2 = rows(23, i, F32, g), weights(3, 2 * f, i, F32, g), weights(3, o, f, F32, g)
    pull = torch.randn((23, o), generator=g, device="cuda")

    def loss(x, w1, w2, act):
        h, out = torch.empty((23, f), device="cuda"), torch.empty((23, o), device="cuda")
        E.expert_gated(x, w1, h, offsets=off, act=act)
        E.expert_linear(h, w2, out, offsets=off)
        return (out.double() * pull.double()).sum()

    for act in ("silu", "gelu", "sigmoid"):
        h, gu, out = torch.empty((23, f), device="cuda"), torch.empty((23, 2 * f), device="cuda"), torch.empty((23, o), device="cuda")
        E.expert_gated(x, w1, h, gu=gu, offsets=off, act=act)
        E.expert_linear(h, w2, out, offsets=off)
        dh, dx, dw1, dw2 = torch.empty_like(h), torch.empty_like(x), torch.empty_like(w1), torch.empty_like(w2)
        E.expert_linear_backward(pull, h, w2, dh, dw2, offsets=off)
        E.expert_gated_backward(dh, gu, x, w1, dx, dw1, offsets=off, act=act)
        for which, grad in enumerate((dx, dw1, dw2)):
            args = [x, w1, w2]
            way = torch.randn(grad.shape, generator=g, device="cuda")
            way /= way.norm()
            step = 2.0 ** -7
            ends = []
            for sign in (1, -1):
                moved = list(args)
                moved[which] = (args[which] + sign * step * way).contiguous()
                ends.append(loss(*moved, act))
            slope = (ends[0] - ends[1]) / (2 * step)
            assert abs(slope - (grad.double() * way.double()).sum()) <= 2.0 ** -9 * grad.double().norm()
