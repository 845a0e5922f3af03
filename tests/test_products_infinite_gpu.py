"""Infinite and NaN elements in fp32 products give what the definition gives, in one row of few and in many: an
infinity times what is not zero is an infinity of its sign (whatever parts either is split into; a weight that
bf16 holds has parts of zero), times zero NaN, and so is the sum of infinities of two signs."""
import math

import pytest
import torch

from test_products_gpu import F32, act64, by_expert, by_rows, gen, offsets_of, rows, weights

pytestmark = pytest.mark.gpu

SHAPES = [([3, 0, 2], 72, 40), ([9, 30], 100, 130), ([300, 500], 479, 351), ([2049, 30], 320, 384), ([700], 1100, 64)]
IDS = [f"{len(s[0])}x{sum(s[0])}-{s[1]}-{s[2]}" for s in SHAPES]


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def same(got, want):
    got = got.double()
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(got.isinf(), want.isinf()) and torch.equal(got[want.isinf()], want[want.isinf()])


def plain(t, g):
    """Some of the elements zero, one, or a half of the other sign, which have one part."""
    r = torch.rand(t.shape, generator=g, device="cuda")
    t[r < 0.1], t[(r >= 0.1) & (r < 0.4)], t[(r >= 0.4) & (r < 0.6)] = 0, 1, -0.5
    return t


def spoil(t, g, share=64):
    """A few infinities and a NaN in some of the rows of a matrix."""
    n = t.shape[0]
    r = torch.randperm(n, generator=g, device="cuda")[:max(1, n // share)]
    c = torch.randint(t.shape[1], (len(r), 2), generator=g, device="cuda")
    t[r, c[:, 0]] = math.inf
    t[r[::2], c[::2, 1]] = -math.inf
    if len(r) > 4:
        t[r[1], c[1, 1]] = math.nan
    return t


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear(E, shape, order):
    counts, i, o = shape
    g, n, off = gen(31), sum(counts), offsets_of(counts)
    x, dout = spoil(plain(rows(n, i, F32, g), g), g), plain(rows(n, o, F32, g), g)
    w = weights(len(counts), o, i, F32, g, order)
    plain(w, g)
    out, dx, dw = torch.empty_like(dout), torch.empty_like(x), torch.empty((len(counts), o, i), device="cuda")
    E.expert_linear(x, w, out, offsets=off)
    want = by_expert(x, w, counts)[0]
    assert want.isinf().any()
    same(out, want)
    E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
    same(dx, by_expert(dout, w.transpose(1, 2), counts)[0])
    same(dw, by_rows(dout, x, counts)[0])
    x = plain(rows(n, i, F32, g), g)
    for e in range(len(counts)):
        spoil(w[e], g, 16)
    E.expert_linear(x, w, out, offsets=off)
    same(out, by_expert(x, w, counts)[0])
    E.expert_linear_backward(dout, x, w, dx, dw, offsets=off)
    same(dx, by_expert(dout, w.transpose(1, 2), counts)[0])


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated(E, shape):
    counts, i, f = shape
    g, n, off = gen(32), sum(counts), offsets_of(counts)
    x, w = spoil(plain(rows(n, i, F32, g), g), g), weights(len(counts), 2 * f, i, F32, g)
    plain(w, g)
    h, gu = torch.empty((n, f), device="cuda"), torch.empty((n, 2 * f), device="cuda")
    E.expert_gated(x, w, h, gu=gu, offsets=off)
    want = by_expert(x, w, counts)[0]
    same(gu, want)
    same(h, act64("silu", want[:, :f])[0] * want[:, f:])
    # and the gradients, of finite g and u
    x, gu = plain(rows(n, i, F32, g), g), plain(rows(n, 2 * f, F32, g), g)
    dh = spoil(plain(rows(n, f, F32, g), g), g)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    E.expert_gated_backward(dh, gu, x, w, dx, dw, offsets=off, act="silu")
    a, slope = act64("silu", gu[:, :f].double())
    dgu = torch.cat([dh.double() * gu[:, f:].double() * slope, dh.double() * a], 1)
    same(dx, by_expert(dgu, w.transpose(1, 2), counts)[0])
    same(dw, by_rows(dgu, x, counts)[0])
