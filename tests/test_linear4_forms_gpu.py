"""Forms of the 4-bit product that test_linear4_gpu's shapes do not come to: codes that are not on the ring's boundaries
with 9 to 16 and 17 to 32 rows an expert and outputs so many that each warp has its own, and more tiles of rows than
a grid has."""
import pytest
import torch

import test_linear4_gpu as base

pytestmark = pytest.mark.gpu
F32, BF16 = base.F32, base.BF16


@pytest.fixture(scope="module")
def E():
    import recommender_model_embedding_gb300 as E
    return E


# rows of codes of 515, 33 and 7 bytes; last warps' tiles behind the last output
ANYWHERE = [([24] * 4, 1, 1030, 30000), ([12] * 4, 0, 1030, 30000), ([32, 0, 31, 17, 5], 2, 66, 24007), ([9, 16, 13, 0, 20], 0, 66, 24007),
            ([20] * 40, 1, 13, 5003), ([10] * 40, 1, 13, 5003), ([33, 64, 40], 0, 515, 24000)]


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("shape", ANYWHERE, ids=[f"{len(s[0])}x{sum(s[0])}-{s[2]}-{s[3]}" for s in ANYWHERE])
def test_many_outputs_of_more_rows(E, shape, group, dtype):
    base.test_product(E, shape, group, dtype, 3 if group == 32 else 0)


@pytest.mark.parametrize("dtype", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("d", [32, 30])
def test_more_tiles_than_a_grid(E, d, dtype):
    base.test_product(E, ([1500001, 0, 700000], 3, d, 3), 32, dtype, 0)
