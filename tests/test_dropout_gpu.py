"""Dropout on the GPU against a plain Philox4x32-10 in Python: the known answers of the generator,
every element's choice, rounding, and what a dropped element may hold."""
import numpy as np
import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16
LOW = 0xFFFFFFFF


def philox(counter, key):
    """Philox4x32-10 of arrays of four 32-bit counter words under two key words (numpy, uint64)."""
    c = [np.asarray(v, dtype=np.uint64) & np.uint64(LOW) for v in counter]
    k = list(key)
    for _ in range(10):
        p, q = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        hi = lambda v: v >> np.uint64(32)
        lo = lambda v: v & np.uint64(LOW)
        c = [hi(q) ^ c[1] ^ np.uint64(k[0]), lo(q), hi(p) ^ c[3] ^ np.uint64(k[1]), lo(p)]
        k = [(k[0] + 0x9E3779B9) & LOW, (k[1] + 0xBB67AE85) & LOW]
    return c


def draws(n, d, seed, step, site):
    """16 bits of each element."""
    b = -(-d // 8)
    col, row = np.meshgrid(np.arange(b), np.arange(n))
    w = philox([col, row, np.full_like(col, step & LOW), np.full_like(col, site)], [seed & LOW, seed >> 32 & LOW])
    out = np.empty((n, b, 8), dtype=np.int64)
    for i in range(8):
        out[:, :, i] = (w[i // 2] >> np.uint64(16 * (i % 2))) & np.uint64(0xFFFF)
    return torch.from_numpy(out.reshape(n, b * 8)[:, :d])


def test_known_answers():
    """The generator's published test vectors (counter and key all zero, all ones)."""
    assert [int(v) for v in philox([0, 0, 0, 0], [0, 0])] == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert [int(v) for v in philox([LOW] * 4, [LOW] * 2)] == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def expected(x, residual, p, seed, step, site, out_type):
    cut = round(p * 65536)
    keep = draws(x.shape[0], x.shape[1], seed, step, site).cuda() >= cut
    v = torch.where(keep, x.double() * (65536 / max(65536 - cut, 1)), 0)
    if residual is not None:
        v = v + residual.double()
    return keep, v


CASES = [(1, 1), (1, 7), (3, 8), (5, 16), (300, 479), (17, 1024), (2, 8192), (1, 65536), (5000, 24), (70000, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("types", [(F32, F32), (BF16, F32), (BF16, BF16)], ids=["f32", "bf16+f32", "bf16"])
@pytest.mark.parametrize("n,d", CASES)
@pytest.mark.parametrize("pad", [0, 5])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_dropout(E, n, d, pad, types, p):
    """Off by one rounding to the output's type and two of fp32 (the scale, the product)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(n * d)
    t, o = types
    x = torch.randn((n, d + pad), generator=g, device="cuda").to(t)[:, :d]
    res = torch.randn((n, d + pad), generator=g, device="cuda").to(o)[:, :d]
    seed, step, site = 0x0123456789ABCDEF, (5 << 32) + 77, 4000000000
    rng = torch.tensor([seed, step], device="cuda")
    for residual in (None, res):
        ot = o if residual is not None else t
        out = torch.empty((n, d + pad), dtype=ot, device="cuda")[:, :d]
        E.dropout(x, out, p, rng, site=site, residual=residual)
        keep, want = expected(x, residual, p, seed, step, site, ot)
        bound = torch.finfo(ot).eps / 2 * want.abs() + 2.0 ** -22 * (want.abs() + (0 if residual is None else residual.double().abs()))
        assert ((out.double() - want).abs() <= bound).all()
        if residual is None:
            assert torch.equal(out != 0, keep & (x != 0))
    dx = torch.empty((n, d), dtype=t, device="cuda")
    E.dropout_backward(x, dx, p, rng, site=site)
    assert torch.equal(dx, expected(x, None, p, seed, step, site, t)[1].to(t)) or t == F32


@pytest.mark.gpu
def test_backward_is_the_forwards_mask(E):
    """The gradient of sum(pull * out) to x, against differences: out is linear in x, so exact up to rounding."""
    x = torch.randn((33, 50), device="cuda")
    rng = torch.tensor([11, 3], device="cuda")
    pull, dx = torch.randn_like(x), torch.empty_like(x)
    E.dropout_backward(pull, dx, 0.3, rng, site=9)
    a, b = torch.empty_like(x), torch.empty_like(x)
    E.dropout(x + 1, a, 0.3, rng, site=9)
    E.dropout(x - 1, b, 0.3, rng, site=9)
    assert torch.allclose(pull * (a - b) / 2, dx, rtol=2e-6, atol=2e-6)


@pytest.mark.gpu
def test_dropped_elements_hold_anything_and_in_place(E):
    rng = torch.tensor([1, 2], device="cuda")
    keep = draws(40, 100, 1, 2, 0).cuda() >= round(0.4 * 65536)
    x = torch.randn((40, 100), device="cuda")
    x[~keep] = float("nan")
    res = torch.randn((40, 100), device="cuda")
    out, plain = torch.empty_like(x), torch.empty_like(x)
    E.dropout(x, out, 0.4, rng, residual=res)
    E.dropout(x, plain, 0.4, rng)
    assert out.isfinite().all() and torch.equal(out[~keep], res[~keep]) and (plain[~keep] == 0).all()
    y, r = x.clone(), res.clone()
    E.dropout(y, y, 0.4, rng)
    E.dropout(x, r, 0.4, rng, residual=r)
    assert torch.equal(y, plain) and torch.equal(r, out)


@pytest.mark.gpu
def test_graph_draws_anew(E):
    """Seed and step are read when the call runs."""
    x, out = torch.ones((64, 64), device="cuda"), torch.empty((64, 64), device="cuda")
    rng = torch.tensor([5, 0], device="cuda")
    E.dropout(x, out, 0.5, rng)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.dropout(x, out, 0.5, rng)
        rng[1].add_(1)
    for step in range(3):
        graph.replay()
        assert torch.equal(out.cpu() != 0, draws(64, 64, 5, step, 0) >= 32768)
    assert rng[1].item() == 3


@pytest.mark.gpu
def test_share_of_dropped(E):
    """4M draws at p = 0.25: the share is within five standard deviations, 5 sqrt(p (1 - p) / n) = 0.0011."""
    x, out = torch.ones((4096, 1024), device="cuda"), torch.empty((4096, 1024), device="cuda")
    E.dropout(x, out, 0.25, torch.tensor([123, 456], device="cuda"))
    assert abs((out == 0).double().mean().item() - 0.25) < 0.0011
    assert torch.equal(out[out != 0], torch.full_like(out[out != 0], 65536 / 49152))


@pytest.mark.gpu
def test_elements_past_2_31(E):
    n = 2100
    store = torch.zeros((n, 1 << 20), device="cuda")
    x = store[:, 64:128]
    x.fill_(1)
    out = store[:, 512:576]
    E.dropout(x, out, 0.5, torch.tensor([9, 9], device="cuda"))
    assert torch.equal(out.cpu() != 0, draws(n, 64, 9, 9, 0) >= 32768)
