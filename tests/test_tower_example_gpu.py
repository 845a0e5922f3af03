"""The expert tower of the example against automatic differentiation of the same tower in 64
bits, written with dense masks, and its training loop together with the embedding layer."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def tower_module():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from helpers import build_lib
    build_lib()
    import expert_tower
    return expert_tower


def plain(p, feats, ids):
    """Logits of the tower with the given choice of experts, in the parameters' type."""
    rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + 1e-6)
    x = (rms(feats) * p["norm_in"]) @ p["w_in"]
    h = rms(x) * p["norm_block"]
    chosen = torch.zeros((x.shape[0], p["w1"].shape[0]), dtype=torch.bool, device=x.device).scatter_(1, ids, True)
    w = (h @ p["w_router"]).masked_fill(~chosen, float("-inf")).softmax(1)
    ys = torch.stack([(h @ p["w1"][e]).relu() @ p["w2"][e] for e in range(p["w1"].shape[0])], 1)
    y = (ys * w[..., None]).sum(1)
    x = x + p["res_scale"] * torch.sigmoid(h @ p["w_gate"]) * rms(y) * p["norm_post"]
    return ((rms(x) * p["norm_out"]) @ p["w_head"])[:, 0]


def test_tower_gradients_match_autograd(tower_module):
    """fp32 products of length up to 479 through about eight layers: relative errors of a few
    times 1e-6; 2e-4 of each gradient's size is the bound asserted."""
    tf32 = torch.backends.cuda.matmul.allow_tf32
    torch.backends.cuda.matmul.allow_tf32 = False
    try:
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        B, W = 333, 479
        feats = torch.randn((B, W), generator=g, device="cuda")
        dl = torch.randn(B, generator=g, device="cuda")
        t = tower_module.ExpertTower(W, hidden=64, experts=5, k=2, inner=48, seed=3)
        logit = t.forward(feats)
        dfeats = t.backward(dl)
        p64 = {k: v.double().requires_grad_() for k, v in t.p.items()}
        f64 = feats.double().requires_grad_()
        ref = plain(p64, f64, t.s["ids"])
        ref.backward(dl.double())
        close = lambda a, b: (a.double() - b).norm() <= 2e-4 * b.norm()
        assert close(logit, ref)
        assert close(dfeats, f64.grad)
        for k, v in t.g.items():
            assert close(v, p64[k].grad), k
        before = {k: v.clone() for k, v in t.g.items()}
        t.step(max_norm=0.01)
        norm = torch.sqrt(sum((v.double() ** 2).sum() for v in before.values()))
        assert abs(t.norm.item() - norm.item()) <= 1e-5 * norm.item()
        for k, v in t.g.items():
            assert close(v, before[k].double() * (0.01 / norm)), k
    finally:
        torch.backends.cuda.matmul.allow_tf32 = tf32


def test_training_loop_learns(tower_module):
    losses = tower_module.train(25, 1024)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) / 5 < 0.75 * losses[0]
