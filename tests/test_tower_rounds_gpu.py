"""The tower's persistent kernels past their first rounds, and the gated norm's gradients against
differences of its formula in 64 bits.

CTAs of the gated norm take row after row, with the next rows on the way; a thread has 8 or 16
elements of a row and an SM at most 1024 threads, so 16 * 1024 / d rows an SM are more than one
round."""
import pytest
import torch

from test_tower_gpu import (E, TYPES, U32, clip_ref, gen, norm_case, norm_grad, norm_grad_ref,  # noqa: F401
                            norm_ref, rows, within)

pytestmark = pytest.mark.gpu


def five_rounds(d):
    """Rows that keep every CTA busy for five rounds at least, and a rest."""
    return torch.cuda.get_device_properties(0).multi_processor_count * -(-16 * 1024 // d) * 5 + 3


WIDTHS = [24, 64, 203, 479, 802, 1024, 2056, 3080, 4100, 8191, 8192]


@pytest.mark.parametrize("xt,bt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("d", WIDTHS)
def test_gated_norm_for_many_rounds(E, d, gate, xt, bt):
    n = five_rounds(d)
    s = norm_case(n, d, gate, TYPES[xt], TYPES[bt], 0, 0, d)
    xo, h = torch.empty_like(s["x"]), torch.empty_like(s["y"])
    vec = {k: s[k] for k in ("gate", "w_post", "res_scale", "w_pre")}
    E.gated_norm(s["x"], s["y"], xo, h, eps=1e-5, **vec)
    rx, ex, rh, eh = norm_ref(s, 1e-5)
    within(xo, rx, ex, "x_out")
    within(h, rh, eh, "h")
    again = s["x"].clone()
    E.gated_norm(again, s["y"], again, None, eps=1e-5, **vec)
    assert torch.equal(again, xo)


@pytest.mark.parametrize("xt,bt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16")])
@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("d", WIDTHS)
def test_gated_norm_backward_for_many_rounds(E, d, gate, xt, bt):
    n = five_rounds(d)
    s = norm_case(n, d, gate, TYPES[xt], TYPES[bt], 0, 0, d)
    ref, got = norm_grad_ref(s, 1e-5), norm_grad(E, s, 1e-5)
    for k, v in got.items():
        if v is not None:
            within(v, *ref[k], k)
    del ref
    # in place: dx over x_out or dx_out, dy over y
    for name in ("x", "dx_out"):
        m = {**s, "y": s["y"].clone(), name: s[name].clone()}
        E.gated_norm_backward(m["dx_out"], m["dh"], m["x"], m["y"], m[name], m["y"], gate=m["gate"],
                              w_post=m["w_post"], res_scale=m["res_scale"], w_pre=m["w_pre"], eps=1e-5)
        assert torch.equal(m[name], got["dx"]) and torch.equal(m["y"], got["dy"]), name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_clip_for_many_rounds(E, dtype):
    """More elements than every CTA takes in two rounds of its largest tiles (8 CTAs an SM, 16384
    elements)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    g, total = gen(3), sms * 8 * 16384 * 2
    grads = [torch.randn(m, generator=g, device="cuda").to(TYPES[dtype]) for m in (total + 100_003, 5, 777_777)]
    norm, out = torch.empty(1, device="cuda"), [torch.empty_like(x) for x in grads]
    ref, c = clip_ref(grads, 1.0)
    E.clip_grads(grads, 1.0, norm, out=out)
    # at most 16 squares a group in fp32, fp64 beyond: 18 u, half of it after the root, and a rounding
    assert abs(norm.item() - ref) <= 10 * U32 * ref
    for x, o in zip(grads, out):
        within(o, x.double() * c, 14 * U32 * c * x.double().abs(), "out")
    E.clip_grads(grads, 1.0, norm)
    assert all(torch.equal(x, o) for x, o in zip(grads, out))


@pytest.mark.parametrize("gate", ["none", "row", "full"])
def test_gated_norm_against_differences_in_64_bits(E, gate):
    """Slopes of L = sum(c1 x_out) + sum(c2 h), the formula in 64 bits, along random directions, by
    central differences of two steps extrapolated to the fourth order.  With steps e and 2 e what is
    left of the truncation is of the size of e^4 (1e-8 of L's terms is allowed), and the kernel's
    gradients are within the bounds carried through their formulas, taken twice for x_out's rounding:
    together a thousandth of the slope's own terms at most, so that no gradient can be missing."""
    n, d, e, eps = 11, 48, 2.0 ** -9, 1e-2
    s = norm_case(n, d, gate, torch.float32, torch.float32, 0, 0, 5)
    s["dx_out"], s["dh"] = rows(gen(6), n, d, torch.float32), rows(gen(7), n, d, torch.float32)
    eps32 = torch.tensor(eps).double().item()
    wide = {k: None if v is None else v.double() for k, v in s.items()}

    def forward(m):
        rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + eps32)
        g = 1.0 if m["gate"] is None else torch.sigmoid(m["gate"])
        xo = m["x"] + m["res_scale"] * g * rms(m["y"]) * m["w_post"]
        return xo, rms(xo) * m["w_pre"]

    def loss(m):
        xo, h = forward(m)
        return ((xo * wide["dx_out"]).sum() + (h * wide["dh"]).sum()).item()

    xo, h = forward(wide)
    mag = ((xo * wide["dx_out"]).abs().sum() + (h * wide["dh"]).abs().sum()).item()
    at = {**s, "x": xo.float()}
    got, ref = norm_grad(E, at, eps), norm_grad_ref(at, eps32)
    for name, grad in (("x", "dx"), ("y", "dy"), ("gate", "dgate"), ("w_post", "dw_post"),
                       ("res_scale", "dres_scale"), ("w_pre", "dw_pre")):
        if s[name] is None:
            continue
        v = torch.randn(s[name].shape, generator=gen(len(name)), device="cuda").double()
        slope = lambda t: (loss({**wide, name: wide[name] + t * v}) - loss({**wide, name: wide[name] - t * v})) / (2 * t)
        found = (4 * slope(e) - slope(2 * e)) / 3
        terms = got[grad].double() * v
        tol = 2 * (ref[grad][1] * v.abs()).sum().item() + 1e-8 * mag
        assert tol <= 1e-3 * terms.abs().sum().item(), (name, tol)
        assert abs(found - terms.sum().item()) <= tol, (name, found, terms.sum().item(), tol)
