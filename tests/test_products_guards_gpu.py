"""Offsets out of order or range with every kernel of the experts' products: some results, none of them outside
the outputs or the workspace."""
import pytest
import torch

from test_products_gpu import BF16, F32, NAMES, gen, rows, weights

pytestmark = pytest.mark.gpu
BAD = [[0, 500, 100, 9000, 200], [-5, 100, 50, 300, 3001], [2400, 1300, 1200, 100, 0], [0, 2 ** 31 - 1, -2 ** 31, 7, 9],
       [1200, 1200, 0, 1200, 0], [700, 650, 1190, 1100, 1199]]


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


class Room:
    """Outputs and workspaces inside larger buffers that hold one value."""
    def __init__(self):
        self.all = []

    def rows(self, n, d, dtype, pad=0):
        big = torch.full((n + 512, d + pad), 3.0, device="cuda", dtype=dtype)
        inner = big[256:256 + n, :d]
        self.all.append((big, inner, 3.0))
        return inner

    def matrices(self, e, o, i, dtype):
        big = torch.full((e + 2, o, i), 3.0, device="cuda", dtype=dtype)
        self.all.append((big, big[1:-1], 3.0))
        return big[1:-1]

    def bytes(self, n):
        big = torch.full((n + 8192,), 77, device="cuda", dtype=torch.uint8)
        inner = big[4096:4096 + n]
        self.all.append((big, inner, 77))
        return inner if n else None

    def check(self):
        for big, inner, value in self.all:
            inner.fill_(value)
            assert (big == value).all()


@pytest.mark.parametrize("off", BAD, ids=range(len(BAD)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("n,i,f", [(1200, 72, 136), (1200, 41, 67), (60, 41, 67)])
def test_bad_offsets(E, n, i, f, dtype, off):
    g = gen(51)
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    x, dout, gu = rows(n, i, dtype, g), rows(n, f, dtype, g), rows(n, 2 * f, dtype, g)
    w = weights(4, 2 * f, i, dtype, g)
    w1 = weights(4, f, i, dtype, g, "io")
    for pad in (0, 3):
        room = Room()
        out, h, gu2, dx = room.rows(n, f, dtype, pad), room.rows(n, f, dtype, pad), room.rows(n, 2 * f, dtype, pad), room.rows(n, i, dtype, pad)
        for dw_type in {F32, dtype}:
            dw, dw1 = room.matrices(4, 2 * f, i, dw_type), room.matrices(4, f, i, dw_type)
            E.expert_linear_backward(dout, x, w1, dx, dw1, offsets=o,
                                     workspace=room.bytes(E.expert_linear_backward_workspace(dout, x, w1, dx, dw1, offsets=o)))
            E.expert_gated_backward(dout, gu, x, w, dx, dw, offsets=o,
                                    workspace=room.bytes(E.expert_gated_backward_workspace(dout, gu, x, w, dx, dw, offsets=o)))
        E.expert_linear(x, w1, out, offsets=o, workspace=room.bytes(E.expert_linear_workspace(x, w1, out, offsets=o)))
        E.expert_gated(x, w, h, gu=gu2, offsets=o, workspace=room.bytes(E.expert_gated_workspace(x, w, h, gu=gu2, offsets=o)))
        torch.cuda.synchronize()
        room.check()


@pytest.mark.parametrize("off", BAD, ids=range(len(BAD)))
@pytest.mark.parametrize("dtype", [BF16, F32], ids=NAMES.get)
@pytest.mark.parametrize("n,d,f", [(4, 128, 600), (60, 128, 9000), (60, 66, 9001), (1200, 72, 9000), (30, 128, 3999)])
def test_bad_offsets_of_4_bit_products(E, n, d, f, dtype, off):
    g = gen(52)
    x = rows(n, d, dtype, g)
    q = torch.randint(0, 256, (4, f, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.rand((4, f, -(-d // 32)), generator=g, device="cuda")
    room = Room()
    out = room.rows(n, f, dtype)
    E.expert_linear4(x, q, scale, out, group=32, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    room.check()
