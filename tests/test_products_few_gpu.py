"""The products' kernel for few rows where tiles are so many that each warp has one of its own: some sixty
experts with up to 8, 16 and 32 rows each on average, weights either way round, outputs that end inside a warp's
tile and warps behind the last output; and many rows of one expert among experts of few."""
import pytest
import torch

import test_products_gpu as base

pytestmark = pytest.mark.gpu
F32, BF16 = base.F32, base.BF16


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


def counts(experts, most):
    return [(7 * i) % (most + 1) for i in range(experts)]


# as test_products_gpu.SHAPES
SHAPES = [
    (counts(60, 8), 3, 40, 443, "oi", 0, 0),
    (counts(60, 24), 0, 40, 443, "oi", 8, 0),
    (counts(63, 48), 1, 41, 443, "oi", 0, 1),
    (counts(60, 8), 0, 40, 883, "io", 0, 0),
    (counts(60, 24), 2, 41, 885, "io", 3, 1),
    (counts(63, 48), 0, 40, 888, "io", 0, 0),
    (counts(60, 8), 1, 264, 440, "oi", 0, 0),
    (counts(240, 8), 1, 24, 130, "io", 2, 0),
    ([3] * 40 + [0, 900, 1, 2] + [1] * 40, 2, 48, 600, "oi", 0, 0),  # (the one expert's rows go through several tiles)
]
IDS = [f"{len(s[0])}x{sum(s[0])}-{s[2]}-{s[3]}-{s[4]}" for s in SHAPES]


@pytest.mark.parametrize("dtype", [BF16, F32], ids=base.NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_linear(E, shape, dtype):
    base.test_linear(E, shape, dtype)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=base.NAMES.get)
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gated(E, shape, dtype, act):
    base.test_gated(E, shape, dtype, act)
