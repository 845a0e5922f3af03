"""Refusals of the experts' products, the 4-bit products and dropout: the C entry points reject bad sizes, types, steps
and buffers on the host, and the binding rejects tensors that do not fit, before anything reaches a
device.  No GPU is needed."""
import ctypes

import pytest

from test_tower_binding import On, Stream
from test_tower_checks import E, FakeCuda, P  # noqa: F401  (E: fixture)


def _product(E, **kw):
    a = dict(rows=4, experts=2, in_=16, out=8, dtype=0, act=0, d_offsets=P, d_x=P, d_w=P, x_ld=16, w_ld=16, w_step=256,
             d_out=P, d_gu=P, out_ld=8, gu_ld=16, d_dout=P, d_dx=P, d_dw=P, dout_ld=8, dx_ld=16, dw_ld=16, dw_step=256)
    a.update(kw)
    return E.EmbProduct(**a)


def _all(E, p):
    L = E._lib
    return {n: (getattr(L, f"emb_expert_{n}_workspace")(ctypes.byref(p)),
                getattr(L, f"emb_expert_{n}")(ctypes.byref(p), P, 1 << 60, None))
            for n in ("linear", "linear_backward", "gated", "gated_backward")}


@pytest.mark.parametrize("bad", [
    dict(rows=-1), dict(rows=2 ** 31 - 1023), dict(experts=0), dict(experts=1025), dict(d_offsets=None), dict(in_=0), dict(out=0),
    dict(in_=65537, w_ld=65537, x_ld=65537), dict(out=65537, out_ld=65537, dout_ld=65537), dict(dtype=2), dict(dtype=-1),
    dict(x_ld=-1), dict(x_ld=1 << 30), dict(w_ld=-1), dict(w_step=-1), dict(w_step=1 << 41), dict(d_x=P + 2), dict(d_w=P + 1),
    dict(d_offsets=P + 2)])
def test_products_refuse(E, bad):
    for name, (need, status) in _all(E, _product(E, **bad)).items():
        assert need == -1 and status == E.EMB_EINVAL, name


@pytest.mark.parametrize("bad,names", [
    (dict(act=4), ("gated", "gated_backward")), (dict(act=-1), ("gated", "gated_backward")),
    (dict(out_ld=7), ("linear", "gated")), (dict(d_out=None), ("linear", "gated")), (dict(d_out=P + 2), ("linear", "gated")),
    (dict(d_x=None), ("linear", "gated", "linear_backward", "gated_backward")),
    (dict(d_w=None), ("linear", "gated", "linear_backward", "gated_backward")),
    (dict(gu_ld=15), ("gated",)), (dict(d_gu=P + 2), ("gated", "gated_backward")), (dict(d_gu=None), ("gated_backward",)),
    (dict(gu_ld=-1), ("gated", "gated_backward")), (dict(d_dout=None), ("linear_backward", "gated_backward")),
    (dict(dout_ld=-1), ("linear_backward", "gated_backward")), (dict(dx_ld=15), ("linear_backward", "gated_backward")),
    (dict(d_dx=None, d_dw=None), ("linear_backward", "gated_backward")), (dict(d_dx=P + 2), ("linear_backward", "gated_backward")),
    (dict(d_dw=P + 2), ("linear_backward", "gated_backward")), (dict(dw_dtype=1), ("linear_backward", "gated_backward")),
    (dict(dw_ld=15), ("linear_backward", "gated_backward")), (dict(dw_step=8), ("linear_backward", "gated_backward")),
    (dict(dw_step=0), ("linear_backward", "gated_backward"))])
def test_products_refuse_what_concerns_them(E, bad, names):
    for name, (need, status) in _all(E, _product(E, rows=4, **bad)).items():
        if name in names:
            assert need == -1 and status == E.EMB_EINVAL, name
        else:
            assert need >= 0, name


def test_products_refuse_workspaces(E):
    L = E._lib
    for name in ("linear", "linear_backward", "gated", "gated_backward"):
        p = _product(E, rows=4096)
        need = getattr(L, f"emb_expert_{name}_workspace")(ctypes.byref(p))
        assert need > 0  # fp32: at least the planes of both operands
        run = getattr(L, f"emb_expert_{name}")
        for ws, have in ((None, need), (P, need - 1), (P + 8, need)):
            assert run(ctypes.byref(p), ws, have, None) == E.EMB_EINVAL
    # bf16 on 16-byte boundaries: nothing to copy
    p = _product(E, rows=4096, dtype=1)
    assert L.emb_expert_linear_workspace(ctypes.byref(p)) == 0 and L.emb_expert_gated_workspace(ctypes.byref(p)) == 0
    assert getattr(L, "emb_expert_linear")(None, None, 0, None) == E.EMB_EINVAL


def test_workspace_sizes_from_tensors(E):
    """The package's sizes are the library's for the same call."""
    x, w, o, off = FakeCuda(F, 600, 16), FakeCuda(F, 2, 8, 16), FakeCuda(F, 600, 8), FakeCuda("int32", 3)
    p = _product(E, rows=600, w_step=128, dw_step=128)
    L = E._lib
    assert E.expert_linear_workspace(x, w, o, offsets=off) == L.emb_expert_linear_workspace(ctypes.byref(p)) > 0
    assert (E.expert_linear_backward_workspace(o, x, w, x, FakeCuda(F, 2, 8, 16), offsets=off)
            == L.emb_expert_linear_backward_workspace(ctypes.byref(p)) > 0)
    h, p.out, p.out_ld, p.dout_ld, p.gu_ld = FakeCuda(F, 600, 4), 4, 4, 4, 8
    assert E.expert_gated_workspace(x, w, h, gu=o, offsets=off) == L.emb_expert_gated_workspace(ctypes.byref(p)) > 0
    assert (E.expert_gated_backward_workspace(h, o, x, w, x, FakeCuda(F, 2, 8, 16), offsets=off)
            == L.emb_expert_gated_backward_workspace(ctypes.byref(p)) > 0)


def test_linear4_and_packing_refuse(E):
    L = E._lib
    ok = dict(rows=4, experts=2, in_=64, out=8, dtype=0, group=32, d_offsets=P, d_x=P, x_ld=64, d_q=P, d_scale=P, d_out=P, out_ld=8)
    for bad in (dict(rows=-1), dict(experts=0), dict(experts=1025), dict(d_offsets=None), dict(in_=0), dict(out=0), dict(in_=65537),
                dict(dtype=2), dict(group=0), dict(group=16), dict(group=48), dict(group=-32), dict(group=65568), dict(d_x=None),
                dict(d_q=None), dict(d_scale=None), dict(d_out=None), dict(x_ld=-1), dict(out_ld=7), dict(d_x=P + 2),
                dict(d_scale=P + 2), dict(d_out=P + 1), dict(rows=2 ** 31 - 1023)):
        assert L.emb_expert_linear4(ctypes.byref(E.EmbProduct4(**{**ok, **bad})), None) == E.EMB_EINVAL, bad
    assert L.emb_expert_linear4(None, None) == E.EMB_EINVAL
    quant = lambda w=P, ld=64, n=4, d=64, t=0, g=32, q=P, s=P: L.emb_quantize_rows4(w, ld, n, d, t, g, q, s, None)
    for bad in (dict(w=None), dict(ld=-1), dict(n=-1), dict(d=0), dict(d=65537), dict(t=2), dict(g=31), dict(g=0), dict(q=None),
                dict(s=None), dict(w=P + 2), dict(s=P + 2)):
        assert quant(**bad) == E.EMB_EINVAL, bad


def test_dropout_refuses(E):
    ok = dict(n=4, dim=8, dtype=0, out_dtype=0, site=0, p=0.5, d_rng=P, d_x=P, d_residual=P, d_out=P, x_ld=8, residual_ld=8, out_ld=8)
    nan = float("nan")
    for bad in (dict(n=-1), dict(n=2 ** 31), dict(dim=0), dict(dim=65537), dict(p=-0.1), dict(p=1.1), dict(p=nan), dict(dtype=2),
                dict(out_dtype=1), dict(dtype=1, out_dtype=0, d_residual=None), dict(d_rng=None), dict(d_rng=P + 4), dict(d_x=None),
                dict(d_out=None), dict(x_ld=-1), dict(residual_ld=-1), dict(out_ld=7), dict(d_x=P + 2), dict(d_residual=P + 2)):
        assert E._lib.emb_dropout(ctypes.byref(E.EmbDropoutRows(**{**ok, **bad})), None) == E.EMB_EINVAL, bad


F, H = "float32", "bfloat16"


def _calls(E):
    """Every call with its tensors' types and shapes, in the call's order."""
    x, w, o, off, ws = (H, 6, 16), (H, 2, 8, 16), (H, 6, 8), ("int32", 3), ("uint8", 1 << 20)
    return {
        "linear": (lambda t, **kw: E.expert_linear(*t[:3], offsets=t[3], workspace=t[4], **kw), [x, w, o, off, ws]),
        "linear_backward": (lambda t, **kw: E.expert_linear_backward(*t[:5], offsets=t[5], workspace=t[6], **kw),
                            [o, x, w, x, (F, 2, 8, 16), off, ws]),
        "gated": (lambda t, **kw: E.expert_gated(*t[:4], offsets=t[4], workspace=t[5], **kw), [x, w, (H, 6, 4), o, off, ws]),
        "gated_backward": (lambda t, **kw: E.expert_gated_backward(*t[:6], offsets=t[6], workspace=t[7], **kw),
                           [(H, 6, 4), o, x, w, x, (F, 2, 8, 16), off, ws]),
        "linear4": (lambda t, **kw: E.expert_linear4(*t[:4], group=32, offsets=t[4], **kw),
                    [x, ("uint8", 2, 8, 8), (F, 2, 8, 1), o, off]),
        "quantize4": (lambda t, **kw: E.quantize_rows4(*t, group=32, **kw), [(H, 8, 16), ("uint8", 8, 8), (F, 8, 1)]),
        "dropout": (lambda t, **kw: E.dropout(t[0], t[1], 0.5, t[2], residual=t[3], **kw), [x, x, ("int64", 2), x]),
    }


# tensors that a call looks at in every case (a workspace only where one is needed)
CALLS = [(n, i) for n, c in (("linear", 4), ("linear_backward", 6), ("gated", 5), ("gated_backward", 8), ("linear4", 5), ("quantize4", 3),
                             ("dropout", 4)) for i in range(c)]


@pytest.mark.parametrize("name,i", CALLS)
def test_binding_refuses_other_devices_types_and_shapes(E, name, i):
    run, specs = _calls(E)[name]
    make = lambda j, s: FakeCuda(*s) if j != i else None
    with pytest.raises(ValueError, match="cuda:[01], the call's first tensor is on cuda:[01]"):
        run([On("cuda:1" if j == i else "cuda:0", *s) for j, s in enumerate(specs)])
    if specs[i][0] != "uint8" or name in ("linear4", "quantize4"):  # (a workspace may be of any type)
        with pytest.raises(ValueError):
            run([make(j, s) or FakeCuda("float16", *s[1:]) for j, s in enumerate(specs)])
    with pytest.raises(ValueError):
        run([make(j, s) or FakeCuda(s[0], 1) for j, s in enumerate(specs)])


@pytest.mark.parametrize("name", ["linear", "linear_backward", "gated", "gated_backward", "linear4", "quantize4", "dropout"])
def test_binding_refuses_a_stream_of_another_device(E, name):
    run, specs = _calls(E)[name]
    with pytest.raises(ValueError, match="stream"):
        run([FakeCuda(*s) for s in specs], stream=Stream())


def test_binding_refuses_what_only_it_can_see(E):
    x, o, off = FakeCuda(H, 6, 16), FakeCuda(H, 6, 8), FakeCuda("int32", 3)
    w = FakeCuda(H, 2, 8, 16)
    bad = [
        lambda: E.expert_linear(x, w, o),  # no offsets for two experts
        lambda: E.expert_linear(x, FakeCuda(H, 2, 8, 15), o, offsets=off),
        lambda: E.expert_linear(x, FakeCuda(H, 2, 8, 16, stride=(512, 64, 2)), o, offsets=off),  # neither axis adjacent
        lambda: E.expert_linear(x, FakeCuda(F, 2, 8, 16), o, offsets=off),
        lambda: E.expert_linear(x, w, FakeCuda(H, 6, 9), offsets=off),
        lambda: E.expert_linear(x, w, FakeCuda(H, 6, 8, stride=(1, 6)), offsets=off),
        lambda: E.expert_linear(x, w, o, offsets=FakeCuda("int32", 2)),
        lambda: E.expert_linear(x, w, o, offsets=FakeCuda("int64", 3)),
        lambda: E.expert_gated(x, FakeCuda(H, 2, 9, 16), o, offsets=off),  # no two halves
        lambda: E.expert_gated(x, w, FakeCuda(H, 6, 4), offsets=off, act="tanh"),
        lambda: E.expert_gated(x, w, FakeCuda(H, 6, 4), gu=FakeCuda(H, 6, 4), offsets=off),
        lambda: E.expert_linear_backward(o, x, w, None, FakeCuda(H, 2, 16, 8), offsets=off),
        lambda: E.expert_linear_backward(o, x, w, None, FakeCuda("int32", 2, 8, 16), offsets=off),
        lambda: E.expert_linear4(x, FakeCuda("uint8", 2, 8, 8), FakeCuda(F, 2, 8, 1), o, group=33, offsets=off),
        lambda: E.expert_linear4(x, FakeCuda("uint8", 2, 8, 7), FakeCuda(F, 2, 8, 1), o, group=32, offsets=off),
        lambda: E.expert_linear4(x, FakeCuda("uint8", 2, 8, 8), FakeCuda(F, 2, 8, 2), o, group=32, offsets=off),
        lambda: E.dropout(x, x, 1.5, FakeCuda("int64", 2)),
        lambda: E.dropout(x, x, 0.5, FakeCuda("int64", 3)),
        lambda: E.dropout(x, FakeCuda(F, 6, 16), 0.5, FakeCuda("int64", 2)),  # another type without a residual
        lambda: E.dropout(FakeCuda(F, 6, 16), x, 0.5, FakeCuda("int64", 2), residual=x),
        lambda: E.dropout(x, x, 0.5, FakeCuda("int64", 2), site=-1),
        lambda: E.dropout(x, x, 0.5, FakeCuda("int64", 2), site=1 << 32),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} passed")
    class Here:
        cuda_stream, device_index = 0, 0

    with pytest.raises(E.EmbError):  # the library's own refusal: gradients of nothing
        E.expert_linear_backward(o, x, w, None, None, offsets=off, stream=Here())
