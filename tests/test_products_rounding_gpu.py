"""How far the experts' products are from their definitions as a whole: distances in the 2-norm, which a
rounding too many shows in and an element's worst case does not.

Let y be the definition's result, z what a kernel has before its last rounding, d = z - y.  The rounded z is at least
as near to z as the rounded y, so |round(z) - y| <= |round(y) - y| + 2 |d|, and so are the 2-norms.  In |d| the errors of a
sum's products, which weights of either sign multiply, add up as independent ones: a relative error of at most r
of each product makes at most r |q|, q the root of the sum of the products' squares."""
import math

import pytest
import torch

from test_products_gpu import ACTS, BF16, F32, NAMES, act64, by_expert, by_rows, gen, offsets_of, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def off_by(got, y):
    """Distance of `got` beyond that of y rounded to its type."""
    return ((got.double() - y).norm() - (y.to(got.dtype).double() - y).norm()).item()


def gated_case(counts, i, f, dtype, seed, act):
    g = gen(seed)
    n = sum(counts)
    x, dh, gu = rows(n, i, dtype, g), rows(n, f, dtype, g), rows(n, 2 * f, dtype, g)
    w = weights(len(counts), 2 * f, i, dtype, g)
    a, slope = act64(act, gu[:, :f].double())
    d, u = dh.double(), gu[:, f:].double()
    return x, dh, gu, w, torch.cat([d * u * slope, d * a], 1)


@pytest.mark.parametrize("dw_type", ["none", "f32", "same"])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,i,f", [([300, 0, 412], 96, 8), ([1000, 24], 64, 128), ([257, 0, 255], 520, 1024)])
def test_gated_backward_of_bf16_rows(E, counts, i, f, act, dw_type):
    """[dg, du] are not rounded to bf16 on their way into dx and dw: two parts of eight bits leave at most
    2^-14 of each, act and its slope 2^-16 (the approximate power of two and reciprocal), three parts for an
    fp32 dw 2^-21.  Sums: 2^-23 of the result for each 16 products that the tensor core adds, of two (three) parts."""
    x, dh, gu, w, dgu = gated_case(counts, i, f, BF16, 21, act)
    off = offsets_of(counts)
    dx = torch.empty_like(x)
    dw = None if dw_type == "none" else torch.empty_like(w, dtype=F32 if dw_type == "f32" else BF16)
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, act=act)
    y = by_expert(dgu, w.transpose(1, 2), counts)[0]
    q = by_expert(dgu ** 2, w.transpose(1, 2).double() ** 2, counts)[0].sqrt().norm().item()
    r = 2.0 ** -14 + 2.0 ** -16 + 2 * 2 * f / 16 * 2.0 ** -23
    assert off_by(dx, y) <= 2 * r * q
    if dw is None:
        return
    y = by_rows(dgu, x, counts)[0]
    q = by_rows(dgu ** 2, x.double() ** 2, counts)[0].sqrt().norm().item()
    # (parts of 512 rows, of 256 where the result is fp32)
    sums = 48 * 2.0 ** -23 if dw.dtype == F32 else 64 * 2.0 ** -23
    r = sums + (2.0 ** -20 if dw.dtype == F32 else 2.0 ** -14 + 2.0 ** -16)
    assert off_by(dw, y) <= 2 * r * q


@pytest.mark.parametrize("dw_type", [F32, BF16], ids=NAMES.get)
def test_infinities_of_the_gated_backward(E, dw_type):
    """An infinite weight makes its input's dx infinite, with the sign of what it is multiplied by, and an infinite x
    its column of dw; values that bf16 holds as they are (products of powers of two) among what they meet."""
    counts = [40, 30]
    x, dh, gu, w, _ = gated_case(counts, 64, 32, BF16, 22, "relu")
    for t in (dh, gu):  # powers of two of either sign: dg and du have one part that is not small
        t.copy_(torch.ldexp(t.sign(), torch.frexp(t.float()).exponent))
    x, w = x.contiguous(), w.contiguous()
    w[0, 5, 7], w[1, 40, 9], x[3, 11], x[50, 12] = math.inf, -math.inf, math.inf, -math.inf
    a, slope = act64("relu", gu[:, :32].double())
    dgu = torch.cat([dh.double() * gu[:, 32:].double() * slope, dh.double() * a], 1)
    dx, dw = torch.empty_like(x), torch.empty_like(w, dtype=dw_type)
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=offsets_of(counts), act="relu")
    same = lambda got, want: torch.equal(got.double().nan_to_num(nan=5e307), want.nan_to_num(nan=5e307))
    for got, want in ((dx[:40, 7], dgu[:40, 5] * math.inf), (dx[40:, 9], dgu[40:, 40] * -math.inf),
                      (dw[0, :, 11], dgu[3] * math.inf), (dw[1, :, 12], dgu[50] * -math.inf)):
        assert same(got, want)
    dx[:40, 7] = 0
    dx[40:, 9] = 0
    dw[0, :, 11] = 0
    dw[1, :, 12] = 0
    assert dx.isfinite().all() and dw.isfinite().all()


def rms(a, b, counts, by):
    """Norm of the roots of the sums of the products' squares."""
    return by(a.double() ** 2, b.double() ** 2, counts)[0].sqrt()


def of_fp32(K):
    """What a sum of K fp32 products is off by, of the root of their squares' sum: 2^-22 of each product left out; parts of
    512, to which the tensor core adds 16 products at a time and cuts off up to a step of 2^-23 of the sum so far, half of
    one on average (its own rounding a step at most); each part's and the last rounding, 2^-24."""
    return 2.0 ** -22 + 32 * 2.0 ** -24 + (-(-K // 512) + 1) * 2.0 ** -24


def of_bf16(K):
    """One sum of K exact products: half a step of 2^-23 for each 16."""
    return -(-K // 16) * 2.0 ** -24


LONG = [([300, 0, 412], 96, 64), ([700], 8192, 72), ([257, 300], 2056, 8), ([8192], 64, 136), ([5000, 11000], 520, 40), ([2], 8192, 64), ([20, 9], 2056, 40)]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("counts,i,o", LONG)
def test_linear(E, counts, i, o, dtype):
    """Both directions, an fp32 dw of bf16 rows among them (its parts are of 512 rows as well)."""
    g, n, off = gen(23), sum(counts), offsets_of(counts)
    of = of_fp32 if dtype == F32 else of_bf16
    x, dout, w = rows(n, i, dtype, g), rows(n, o, dtype, g), weights(len(counts), o, i, dtype, g)
    out, dx, dw = torch.empty_like(dout), torch.empty_like(x), torch.empty((len(counts), o, i), device="cuda")
    E.expert_linear(x, w, out, offsets=off)
    E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
    wt = w.transpose(1, 2)
    assert off_by(out, by_expert(x, w, counts)[0]) <= 2 * of(i) * rms(x, w, counts, by_expert).norm()
    assert off_by(dx, by_expert(dout, wt, counts)[0]) <= 2 * of(o) * rms(dout, wt, counts, by_expert).norm()
    assert off_by(dw, by_rows(dout, x, counts)[0]) <= 2 * of_fp32(max(counts)) * rms(dout, x, counts, by_rows).norm()


@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("counts", [[2], [300]], ids=["few", "many"])
def test_longest_rows(E, counts, dtype):
    """65536 inputs, as many as there can be: in bf16 the one sum's error, 2^-12, is still inside the result's rounding."""
    test_linear(E, counts, 65536, 40, dtype)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("counts,i,f", [([300, 0, 412], 96, 64), ([700], 4096, 72), ([8192], 64, 136), ([20, 9], 2056, 40)])
def test_gated_in_fp32(E, counts, i, f, act):
    """h from g and u as they are (errors times |act'| |u| <= 1.13 |u| and |act|), the exponential's 2^-21; the gradients'
    [dg, du] 2^-20 off."""
    x, dh, gu, w, dgu = gated_case(counts, i, f, F32, 24, act)
    off, h = offsets_of(counts), torch.empty_like(dh)
    E.expert_gated(x, w, h, offsets=off, act=act)
    y, q = by_expert(x, w, counts)[0], rms(x, w, counts, by_expert)
    a, u = act64(act, y[:, :f])[0], y[:, f:]
    d = of_fp32(i) * (1.13 * u.abs() * q[:, :f] + a.abs() * q[:, f:]) + 2.0 ** -21 * u.abs() * (a.abs() + 1e-3)
    assert off_by(h, a * u) <= 2 * d.norm()
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, act=act)
    wt = w.transpose(1, 2)
    assert off_by(dx, by_expert(dgu, wt, counts)[0]) <= 2 * (of_fp32(2 * f) + 2.0 ** -20) * rms(dgu, wt, counts, by_expert).norm()
    assert off_by(dw, by_rows(dgu, x, counts)[0]) <= 2 * (of_fp32(max(counts)) + 2.0 ** -20) * rms(dgu, x, counts, by_rows).norm()
