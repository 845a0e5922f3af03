"""A sparsely gated block as it is used: rows sorted by expert, through each expert's gated block and second layer, a
dropout, and back with weights; forward and backward against automatic differentiation of the same
block in 64 bits, written with dense masks; and the same served from 4-bit weights."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def i32(n):
    return torch.empty(n, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,n,k,e,d,f", [(torch.float32, 333, 2, 5, 48, 40), (torch.float32, 3, 2, 8, 479, 64),
                                             (torch.bfloat16, 700, 2, 6, 96, 72), (torch.bfloat16, 1, 2, 8, 128, 64)])
def test_block(E, dtype, n, k, e, d, f):
    """fp32: four products in a row, each within 2^-20 of the magnitudes, which the sums along 479 columns leave
    about 30 times the results: 2^-13 of each result's size holds it.  bf16: inputs and six intermediates are
    rounded to 2^-8 each, and errors add up as squares: 4 2^-8 holds it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, res, pull = (r(n, d).to(dtype) for _ in range(3))
    w1, w2 = (r(e, 2 * f, d) / math.sqrt(d)).to(dtype), (r(e, d, f) / math.sqrt(f)).to(dtype)
    ids = torch.rand((n, e), generator=g, device="cuda").topk(k, 1).indices
    ids[torch.rand((n, k), generator=g, device="cuda") < 0.2] = -1
    w = torch.rand((n, k), generator=g, device="cuda")
    rng, p = torch.tensor([77, 5], device="cuda"), 0.3
    S = n * k
    order, pos, off = i32(S), i32(S), i32(e + 1)
    room = lambda *s: torch.empty(s, device="cuda", dtype=dtype)
    xs, h, gu, ys, y, out = room(S, d), room(S, f), room(S, 2 * f), room(S, d), room(n, d), room(n, d)
    E.expert_sort(ids, e, order, pos, off)
    E.expert_dispatch(x, pos, xs)
    E.expert_gated(xs, w1, h, gu=gu, offsets=off)
    E.expert_linear(h, w2, ys, offsets=off)
    E.expert_combine(ys, pos, w, y)
    E.dropout(y, out, p, rng, site=1, residual=res)
    dy, dys, dw = room(n, d), room(S, d), torch.empty((n, k), device="cuda")
    dh, dxs, dx = room(S, f), room(S, d), room(n, d)
    dw1, dw2 = torch.empty((e, 2 * f, d), device="cuda"), torch.empty((e, d, f), device="cuda")
    E.dropout_backward(pull, dy, p, rng, site=1)
    E.expert_combine_backward(dy, ys, pos, w, dys, dw)
    E.expert_linear_backward(dys, h, w2, dh, dw2, offsets=off)
    E.expert_gated_backward(dh, gu, xs, w1, dxs, dw1, offsets=off)
    E.expert_dispatch_backward(dxs, pos, dx)

    leaf = lambda v: v.double().requires_grad_()
    x64, res64, w164, w264, ww = leaf(x), leaf(res), leaf(w1), leaf(w2), leaf(w)
    every = torch.stack([(torch.nn.functional.silu(x64 @ w164[i, :f].T) * (x64 @ w164[i, f:].T)) @ w264[i].T for i in range(e)], 1)
    kept = ids >= 0
    mixed = (torch.where(kept, ww, 0)[..., None] * every.gather(1, ids.clamp_min(0)[..., None].expand(n, k, d))).sum(1)
    mask = torch.empty((n, d), device="cuda")
    E.dropout(torch.ones((n, d), device="cuda"), mask, p, rng, site=1)
    want = res64 + mixed * mask.double()
    want.backward(pull.double())
    tol = 2.0 ** -13 if dtype == torch.float32 else 4 * 2.0 ** -8
    for got, ref in ((out, want), (dx, x64.grad), (dw1, w164.grad), (dw2, w264.grad), (dw, ww.grad)):
        assert (got.double() - ref).norm() <= tol * ref.norm() + 1e-30


def test_served_from_4_bits(E):
    """Weights packed and served: the block of the dequantised weights in 64 bits; bf16 rounds twice on the way, 2^-8
    each, and once at the end."""
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    n, k, e, d, f, group = 3, 2, 8, 256, 96, 64
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, w1, w2 = r(n, d).bfloat16(), r(e, f, d) / math.sqrt(d), r(e, d, f) / math.sqrt(f)

    def pack(w):
        q = torch.empty((*w.shape[:2], w.shape[2] // 2), dtype=torch.uint8, device="cuda")
        s = torch.empty((*w.shape[:2], -(-w.shape[2] // group)), device="cuda")
        E.quantize_rows4(w, q, s, group)
        column = torch.arange(w.shape[2], device="cuda")
        return q, s, (((q[..., column // 2].long() >> (4 * (column % 2))) & 15) - 8).double() * s.double()[..., column // group]

    (q1, s1, v1), (q2, s2, v2) = pack(w1), pack(w2)
    ids = torch.rand((n, e), generator=g, device="cuda").topk(k, 1).indices
    S = n * k
    order, pos, off = i32(S), i32(S), i32(e + 1)
    room = lambda *s: torch.empty(s, device="cuda", dtype=torch.bfloat16)
    xs, a, ys, y = room(S, d), room(S, f), room(S, d), room(n, d)
    w = torch.rand((n, k), generator=g, device="cuda")
    E.expert_sort(ids, e, order, pos, off)
    E.expert_dispatch(x, pos, xs)
    E.expert_linear4(xs, q1, s1, a, group=group, offsets=off)
    a.relu_()
    E.expert_linear4(a, q2, s2, ys, group=group, offsets=off)
    E.expert_combine(ys, pos, w, y)
    every = torch.stack([(x.double() @ v1[i].T).relu() @ v2[i].T for i in range(e)], 1)
    want = (w.double()[..., None] * every.gather(1, ids[..., None].expand(n, k, d))).sum(1)
    assert (y.double() - want).norm() <= 3 * 2.0 ** -8 * want.norm()
