"""Values of the expert tower's operators where their arithmetic is most exposed, against plain
formulas in 64 bits.  u = 2^-24 is fp32's unit roundoff; every bound is the sum of the errors of
the operations that lead to the value."""
import pytest
import torch

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from helpers import build_lib
    build_lib()
    import recommender_model_embedding_gb300 as E
    return E


@pytest.mark.parametrize("cols", ["full", "row"])
def test_gate_is_as_exact_far_from_zero(E, cols):
    """The gate's relative error does not grow with the size of its argument.  With x = 0 and rows of
    ones, x_out = sigmoid(z) a, a = 1 / sqrt(1 + eps).  e = exp(-z) is within 5 u (a fast
    exponential's 2^-22 and a rounding), its sum with 1 rounds once and the reciprocal is within one
    unit (2 u): 8 u for the gate; a is within 2 units and a rounding (5 u), and two products round:
    15 u, 16 u asserted.  dgate = g a (1 - g), 1 - g = e g: at most 5 u for e in the product of both,
    twice 3 u for the sum and the reciprocal and 1 u, then a and three roundings: 20 u, 32 u
    asserted."""
    n, d, eps = 64, 256, 1e-6
    z = torch.linspace(-80.0, 80.0, n * d if cols == "full" else n, device="cuda").reshape(n, -1)
    x, y = torch.zeros((n, d), device="cuda"), torch.ones((n, d), device="cuda")
    out = torch.empty_like(x)
    E.gated_norm(x, y, out, None, gate=z, eps=eps)
    a = (1 + torch.tensor(eps, device="cuda").double()).rsqrt()  # eps as the call takes it
    g, rest = torch.sigmoid(z.double()), torch.sigmoid(-z.double())
    off = ((out.double() - g * a) / (g * a)).abs().max().item()
    assert off <= 16 * U32, off / U32
    dgate, one = torch.empty_like(z), torch.ones_like(x)
    E.gated_norm_backward(one, None, x, y, None, None, gate=z, dgate=dgate, eps=eps)
    ref = g * a * rest * (1 if cols == "full" else d)
    # one gate a row: d equal terms are added, of 8 a thread and then in pairs (at most 16 u more)
    off = ((dgate.double() - ref) / ref).abs().max().item()
    assert off <= (32 if cols == "full" else 48) * U32, off / U32


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("limit", [1.0, 1e-3, 1e-6, 1e-20, 1e-36])
def test_clip_factors_below_normal_numbers(E, limit, dtype):
    """A factor that fp32 alone would hold with few bits, or as zero.  The norm is within 20 u (16
    squares a sum in fp32, fp64 beyond, one rounding), the factor and its two products round
    three times, then the output rounds once; a result below the normal numbers keeps what its type
    has there."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    grads = [(torch.randn(m, generator=g, device="cuda").clamp(-3, 3) * 1e37).to(dtype) for m in (64, 7)]
    grads.append((torch.randn(900, generator=g, device="cuda") * 1e20).to(dtype))
    full = torch.cat([x.double() for x in grads]).norm().item()
    norm, out = torch.empty(1, device="cuda"), [torch.empty_like(x) for x in grads]
    E.clip_grads(grads, limit, norm, out=out)
    assert abs(norm.item() - full) <= 20 * U32 * full
    c = torch.tensor(limit, device="cuda").double() / full
    r, least = (U32, 2.0 ** -149) if dtype == torch.float32 else (2.0 ** -8, 2.0 ** -133)
    for x, o in zip(grads, out):
        ref = x.double() * c
        assert bool(((o.double() - ref).abs() <= (24 * U32 + r) * ref.abs() + least).all())
