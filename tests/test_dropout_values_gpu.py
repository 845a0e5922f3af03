"""Dropout's backward in fp32 against 64 bits: the scale is rounded once and the product once, 2^-24 of the value each."""
import pytest
import torch

from test_dropout_gpu import expected

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,d,pad", [(1, 1, 0), (33, 50, 0), (64, 1024, 0), (70, 479, 5)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.37, 0.999, 1.0])
def test_backward_in_fp32(n, d, pad, p):
    import recommender_model_embedding_gb300 as E
    g = torch.Generator(device="cuda")
    g.manual_seed(n + d)
    dout = torch.randn((n, d + pad), generator=g, device="cuda")[:, :d]
    seed, step, site = 0x7EDCBA9876543210, (3 << 32) + 5, 17
    dx = torch.empty((n, d), device="cuda")
    E.dropout_backward(dout, dx, p, torch.tensor([seed, step], device="cuda"), site=site)
    keep, want = expected(dout, None, p, seed, step, site, torch.float32)
    assert want.dtype == torch.float64
    assert ((dx.double() - want).abs() <= (2 * 2.0 ** -24 + 2.0 ** -47) * want.abs()).all()
    assert torch.equal(dx != 0, keep & (dout != 0))
