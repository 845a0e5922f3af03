"""One weight matrix for every expert (step 0): read where it lies, or copied once, however many experts there
are, in both directions and by either kernel."""
import pytest
import torch

from test_products_gpu import BF16, F32, NAMES, by_expert, by_rows, close, gen, offsets_of, rows, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("i,o", [(136, 264), (41, 33)])
def test_workspace(E, i, o, dtype, order):
    g = gen(41)
    x, dout, gu = rows(2000, i, dtype, g), rows(2000, o, dtype, g), rows(2000, 2 * o, dtype, g)
    one = weights(1, 2 * o, i, dtype, g, order)
    need = []
    for experts in (2, 15):  # (by the kernel for many rows)
        off = torch.linspace(0, 2000, experts + 1, device="cuda").int()
        w = one.expand(experts, 2 * o, i)
        dx = torch.empty_like(x)
        need.append((E.expert_linear_workspace(x, w[:, :o], dout, offsets=off), E.expert_gated_workspace(x, w, dout, offsets=off),
                     E.expert_linear_backward_workspace(dout, x, w[:, :o], dx, None, offsets=off),
                     E.expert_gated_backward_workspace(dout, gu, x, w, dx, None, offsets=off)))
    assert need[0] == need[1]


@pytest.mark.parametrize("order", ["oi", "io"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("counts", [[3, 0, 2, 1], [400, 0, 300, 1, 211]], ids=["few", "many"])
@pytest.mark.parametrize("i,o", [(136, 264), (41, 33)])
def test_products(E, i, o, counts, dtype, order):
    g, n, e, off = gen(42), sum(counts), len(counts), offsets_of(counts)
    x, dout = rows(n, i, dtype, g), rows(n, o, dtype, g)
    w = weights(1, 2 * o, i, dtype, g, order).expand(e, 2 * o, i)
    out, gu, h = torch.empty_like(dout), rows(n, 2 * o, dtype, g), torch.empty_like(dout)
    dx, dw = torch.empty_like(x), torch.empty((e, o, i), device="cuda")
    E.expert_linear(x, w[:, :o], out, offsets=off)
    y, m = by_expert(x, w[:, :o], counts)
    close(out, y, m, i, split=dtype == F32)
    E.expert_gated(x, w, h, gu=gu, offsets=off)
    y, m = by_expert(x, w, counts)
    close(gu, y, m, i, split=dtype == F32)
    E.expert_linear_backward(dout, x, w[:, :o], dx, dw, offsets=off)
    y, m = by_expert(dout, w[:, :o].transpose(1, 2), counts)
    close(dx, y, m, o, split=dtype == F32)
    y, m = by_rows(dout, x, counts)
    close(dw, y, m, max(counts), split=dtype == F32)
    again, own = torch.empty_like(x), torch.empty_like(x)
    E.expert_gated_backward(dout, gu, x, w, again, None, offsets=off)
    E.expert_gated_backward(dout, gu, x, w.contiguous(), own, None, offsets=off)
    assert torch.equal(again, own)
