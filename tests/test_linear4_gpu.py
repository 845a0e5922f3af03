"""4-bit weights on the GPU: packing against its rule step by step, and the grouped product against its
definition in 64 bits (a result is rounded once, eps / 2; before that a sum of K terms is off by at most
K 2^-23 of the sum of magnitudes, and each scale's product by 2^-24)."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def unpack(q, scale, d, group):
    column = torch.arange(d, device=q.device)
    code = (q[..., column // 2].long() >> (4 * (column % 2))) & 15
    return (code.double() - 8) * scale.double()[..., column // group]


@pytest.mark.parametrize("group", [32, 64, 128, 96])
@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (3, 31, 2), (5, 64, 0), (17, 479, 33), (200, 1024, 0)])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_packing(E, n, d, pad, group, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    w = torch.randn((n, d + pad), generator=g, device="cuda").to(dtype)[:, :d]
    w[0] = 0
    q = torch.empty((n, -(-d // 2)), dtype=torch.uint8, device="cuda")
    scale = torch.empty((n, -(-d // group)), device="cuda")
    E.quantize_rows4(w, q, scale, group)
    v = np.zeros((n, -(-d // group) * group), np.float32)
    v[:, :d] = w.float().cpu().numpy()
    s = np.abs(v.reshape(n, -1, group)).max(2) / np.float32(7)
    with np.errstate(invalid="ignore", divide="ignore"):
        c = np.where(s[..., None] > 0, np.rint(v.reshape(n, -1, group) / s[..., None]), 0)
    c = (np.clip(c, -7, 7).astype(int) + 8).reshape(n, -1)
    c = np.concatenate([c, np.full((n, 1), 8)], 1)
    c[:, d:] = 8
    want = (c[:, 0:2 * q.shape[1]:2] | c[:, 1:2 * q.shape[1]:2] << 4).astype(np.uint8)
    assert np.array_equal(scale.cpu().numpy(), s.astype(np.float32)) and np.array_equal(q.cpu().numpy(), want)
    back = unpack(q, scale, d, group)
    assert ((back - w.double()).abs() <= scale.double().repeat_interleave(group, 1)[:, :d] * (0.5 + 2.0 ** -20)).all()


SHAPES = [([1], 0, 32, 16), ([1], 0, 1, 1), ([2], 1, 128, 40), ([1, 0, 1, 3], 2, 256, 33), ([8], 0, 479, 100), ([9], 0, 1024, 64),
          ([13, 0, 20], 5, 1030, 17), ([33], 0, 96, 48), ([100, 3], 0, 200, 130), ([1] * 40, 3, 4096, 16), ([0, 0], 7, 64, 64)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 96, 256])
@pytest.mark.parametrize("shape", SHAPES, ids=[f"{len(s[0])}x{sum(s[0])}-{s[2]}-{s[3]}" for s in SHAPES])
@pytest.mark.parametrize("pad", [0, 3])
def test_product(E, shape, group, dtype, pad):
    counts, rest, d, o = shape
    e, n = len(counts), sum(counts)
    g = torch.Generator(device="cuda")
    g.manual_seed(d + o)
    x = torch.randn((n + rest, d + pad), generator=g, device="cuda").to(dtype)[:, :d]
    x[n:] = float("nan")
    q = torch.randint(0, 256, (e, o, -(-d // 2)), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand((e, o, -(-d // group)), generator=g, device="cuda") / math.sqrt(d)
    out = torch.full((n + rest, o + pad), 7.0, device="cuda", dtype=dtype)[:, :o]
    off = torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)
    E.expert_linear4(x, q, scale, out, group=group, offsets=off)
    lo = 0
    for i, c in enumerate(counts):
        a, w = x[lo:lo + c].double(), unpack(q[i], scale[i], d, group)
        want, mag = a @ w.T, a.abs() @ w.abs().T
        bound = torch.finfo(dtype).eps / 2 * want.abs() + (d + 2) * 2.0 ** -23 * mag + 1e-30
        assert ((out[lo:lo + c].double() - want).abs() <= bound).all()
        if dtype == F32 and c:
            assert (out[lo:lo + c].double() - want).norm() <= 2.0 ** -20 * mag.norm()
        lo += c
    assert (out[n:] == 7).all()
    if e == 1 and not rest:
        alone = torch.empty_like(out)
        E.expert_linear4(x, q[0], scale[0], alone, group=group)
        assert torch.equal(alone, out)


# outputs so many that each warp has its own: rows of codes on 16 bytes, 4 bytes, and any; one, two and more pieces of
# the columns; a last tile, and a last warp's tiles, that are not whole
MANY = [([1] * 6, 0, 32, 14000), ([1, 0, 3] * 4, 2, 1024, 9999), ([8] * 5, 1, 479, 16001), ([2, 1, 0, 5], 0, 2056, 20488),
        ([1] * 30, 1, 2600, 2890), ([1] * 8, 3, 515, 11000), ([16, 9, 12], 1, 1096, 26000), ([9] * 9, 0, 4160, 9001),
        ([33, 0, 17, 20], 3, 1160, 15003), ([64, 40], 0, 264, 30000), ([1, 2] * 60, 1, 96, 9000), ([17] * 60, 0, 200, 8005),
        ([10, 16] * 40, 2, 352, 7010),
        # fewer: pairs of tiles of a CTA in fp32
        ([1], 0, 4104, 8000), ([5, 1], 1, 1024, 3999), ([1, 1, 3], 0, 2600, 2009), ([9, 0, 16], 2, 1160, 3600), ([3] * 8, 0, 200, 1000)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 96])
@pytest.mark.parametrize("shape", MANY, ids=[f"{len(s[0])}x{sum(s[0])}-{s[2]}-{s[3]}" for s in MANY])
def test_many_outputs(E, shape, group, dtype):
    test_product(E, shape, group, dtype, 3 if group == 96 else 0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_outputs_again(E, dtype):
    """Calls in a row, on two streams, and replayed give the same bits; a scale behind an infinite one is not read
    for columns that are not there."""
    e, d, o = 6, 2104, 14008
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((e, d), generator=g, device="cuda").to(dtype)
    q = torch.randint(0, 256, (e, o, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand((e, o, -(-d // 64)), generator=g, device="cuda")
    scale[1, 7, -1] = float("inf")
    off = torch.arange(e + 1, device="cuda").int()
    outs = [torch.full((e, o), 7.0, device="cuda", dtype=dtype) for _ in range(4)]
    E.expert_linear4(x, q, scale, outs[0], offsets=off)
    E.expert_linear4(x, q, scale, outs[1], offsets=off)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        E.expert_linear4(x, q, scale, outs[2], offsets=off)
    torch.cuda.current_stream().wait_stream(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        E.expert_linear4(x, q, scale, outs[3], offsets=off)
    outs[3].fill_(7)
    graph.replay()
    last = unpack(q[1, 7], torch.ones_like(scale[1, 7]), d, 64)[d // 64 * 64:] @ x[1, d // 64 * 64:].double()
    assert outs[0][1, 7].double() == math.copysign(math.inf, last)
    ok = torch.ones_like(outs[0], dtype=torch.bool)
    ok[1, 7] = False
    assert outs[0][ok].isfinite().all()
    for other in outs[1:]:
        assert torch.equal(outs[0], other)


def test_codes_anywhere(E):
    """Codes that start at any byte."""
    x = torch.randn((3, 64), device="cuda")
    store = torch.randint(0, 256, (20 * 32 + 5,), device="cuda", dtype=torch.uint8)
    scale = torch.rand((20, 2), device="cuda")
    for at in range(5):
        q = store[at:at + 640].view(20, 32)
        out = torch.empty((3, 20), device="cuda")
        E.expert_linear4(x, q, scale, out, group=32)
        want = x.double() @ unpack(q, scale, 64, 32).T
        assert torch.allclose(out.double(), want, rtol=1e-5, atol=1e-4)


@pytest.mark.parametrize("at", [0, 1, 4, 8, 16])
@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
def test_many_codes_anywhere(E, at, dtype):
    """Where codes start says which way they are brought, not what comes out; the last one's bytes end the buffer."""
    e, d, o = 8, 192, 12008
    g = torch.Generator(device="cuda")
    g.manual_seed(at)
    x = torch.randn((e, d), generator=g, device="cuda").to(dtype)
    store = torch.randint(0, 256, (at + e * o * d // 2,), generator=g, device="cuda", dtype=torch.uint8)
    q, scale = store[at:].view(e, o, d // 2), torch.rand((e, o, 3), generator=g, device="cuda")
    out, off = torch.empty((e, o), device="cuda", dtype=dtype), torch.arange(e + 1, device="cuda").int()
    E.expert_linear4(x, q, scale, out, offsets=off)
    w = unpack(q, scale, d, 64)
    want = torch.einsum("ed,eod->eo", x.double(), w)
    mag = torch.einsum("ed,eod->eo", x.double().abs(), w.abs())
    assert ((out.double() - want).abs() <= torch.finfo(dtype).eps / 2 * want.abs() + (d + 2) * 2.0 ** -23 * mag).all()


def test_rows_do_not_leak(E):
    """NaN and infinities in one row stay there."""
    x = torch.randn((6, 128), device="cuda").to(BF16)
    q = torch.randint(0, 256, (32, 64), device="cuda", dtype=torch.uint8)
    scale = torch.rand((32, 1), device="cuda")
    a, b = torch.empty((6, 32), device="cuda", dtype=BF16), torch.empty((6, 32), device="cuda", dtype=BF16)
    E.expert_linear4(x, q, scale, a, group=128)
    x[2], x[4] = float("nan"), float("inf")
    E.expert_linear4(x, q, scale, b, group=128)
    keep = [0, 1, 3, 5]
    assert torch.equal(a[keep], b[keep]) and not b[2].isfinite().any()
