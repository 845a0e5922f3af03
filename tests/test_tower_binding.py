"""What the expert-tower calls refuse about buffers that fit in type and size.  No GPU is needed."""
import ctypes

import pytest

from test_tower_checks import E, FakeCuda, P, _norm  # noqa: F401  (E: fixture)


class On(FakeCuda):
    """A tensor of the given device."""

    def __init__(self, device, dtype, *shape, **kw):
        super().__init__(dtype, *shape, **kw)
        self.device = device


class Stream:
    cuda_stream, device_index = 0, 1


def _calls(E):
    """Every call with its tensors' types and shapes, in the call's order (None: left out)."""
    n, k, d, e = 4, 2, 8, 8
    f, i, x = "float32", "int32", ("float32", n, d)
    xs, pos, w, v = ("float32", n * k, d), (i, n * k), (f, n, k), (f, d)
    ws, m = ("uint8", 1 << 24), 40000  # (m rows: so many that the sort takes a workspace)
    return [
        (lambda t, **kw: E.expert_sort(t[0], e, *t[1:4], workspace=t[4], **kw),
         [("int64", m, k), (i, m * k), (i, m * k), (i, e + 1), ws]),
        (lambda t, **kw: E.expert_dispatch(*t, **kw), [x, pos, xs]),
        (lambda t, **kw: E.expert_dispatch_backward(*t, **kw), [xs, pos, x]),
        (lambda t, **kw: E.expert_combine(*t, **kw), [xs, pos, w, x]),
        (lambda t, **kw: E.expert_combine_backward(*t, **kw), [x, xs, pos, w, xs, w]),
        (lambda t, **kw: E.gated_norm(*t[:4], gate=t[4], w_post=t[5], res_scale=t[6], w_pre=t[7], **kw),
         [x, x, x, x, x, v, v, v]),
        (lambda t, **kw: E.gated_norm_backward(*t[:6], gate=t[6], w_post=t[7], res_scale=t[8], w_pre=t[9],
                                               dgate=t[10], dw_post=t[11], dres_scale=t[12], dw_pre=t[13],
                                               workspace=t[14], **kw),
         [x] * 7 + [v, v, v] + [x] + [v, v, v] + [ws]),
        (lambda t, **kw: E.clip_grads(t[:2], 1.0, t[4], out=t[2:4], workspace=t[5], **kw),
         [(f, 9), (f, 5), (f, 9), (f, 5), (f, 1), ws]),
    ]


@pytest.mark.parametrize("call", range(8))
def test_tensors_of_two_devices_are_refused(E, call):
    run, specs = _calls(E)[call]
    for i in range(len(specs)):
        t = [On("cuda:1" if j == i else "cuda:0", *s) for j, s in enumerate(specs)]
        with pytest.raises(ValueError, match="cuda:[01], the call's first tensor is on cuda:[01]"):
            run(t)


@pytest.mark.parametrize("call", range(8))
def test_stream_of_another_device_is_refused(E, call):
    run, specs = _calls(E)[call]
    with pytest.raises(ValueError, match="stream: on cuda:1"):
        run([On("cuda:0", *s) for s in specs], stream=Stream())


def test_slot_matrices_of_another_width_are_refused(E):
    """A pos, w or dw whose rows are not k long would be taken apart at the wrong places."""
    F = FakeCuda
    x, xs, pos, w = F("float32", 4, 8), F("float32", 8, 8), F("int32", 8), F("float32", 4, 2)
    wide, flipped = F("float32", 4, 3), F("float32", 2, 4)
    for bad in (wide, flipped):
        with pytest.raises(ValueError, match="w: .*expected .4, 2."):
            E.expert_combine(xs, pos, bad, x)
        with pytest.raises(ValueError, match="w: .*expected .4, 2."):
            E.expert_combine_backward(x, xs, pos, bad, xs, w)
        with pytest.raises(ValueError, match="dw: .*expected .4, 2."):
            E.expert_combine_backward(x, xs, pos, w, xs, bad)
    # the places of eight rows with the first four of them: not four rows of twice as many
    many, room = F("int32", 8, 2), F("float32", 16, 8)
    for call in (lambda: E.expert_dispatch(x, many, room), lambda: E.expert_dispatch_backward(room, many, x),
                 lambda: E.expert_combine(room, many, F("float32", 16), x)):
        with pytest.raises(ValueError, match="pos: .8, 2., expected .4, 4."):
            call()
    with pytest.raises(ValueError, match="pos: .4, 3., expected .4, 2."):
        E.expert_sort(F("int64", 4, 2), 8, pos, F("int32", 4, 3), F("int32", 9))


def test_c_calls_refuse_misaligned_buffers(E):
    """Every index, weight and vector buffer is on a boundary of its type: a kernel's access to one that
    is not would fault."""
    L, q, bad = E._lib, P + 2, E.EMB_EINVAL
    for i in range(4):
        b = [P] * 4
        b[i] = P + 4 if i == 0 else q
        assert L.emb_expert_sort(b[0], 4, 2, 8, b[1], b[2], b[3], P, 1 << 20, None) == bad
    assert L.emb_expert_dispatch(P, 8, q, 4, 2, 8, 1, P, 8, None) == bad
    assert L.emb_expert_dispatch_backward(P, 8, q, 4, 2, 8, 1, P, 8, None) == bad
    assert L.emb_expert_combine(P, 8, q, P, 4, 2, 8, 1, P, 8, None) == bad
    assert L.emb_expert_combine(P, 8, P, q, 4, 2, 8, 1, P, 8, None) == bad
    for i in range(3):
        b = [P] * 3
        b[i] = q
        assert L.emb_expert_combine_backward(P, 8, P, 8, b[0], b[1], 4, 2, 8, 1, P, 8, b[2], None) == bad
    for name in ("d_w_post", "d_res_scale", "d_w_pre"):
        assert L.emb_gated_norm(ctypes.byref(_norm(E, **{name: q})), None) == bad
    grad = dict(d_x=None, d_h=None, d_dx_out=P, d_dh=P, d_dx=P, d_dy=P, dx_out_ld=8, dh_ld=8, dx_ld=8, dy_ld=8)
    for name in ("d_w_post", "d_res_scale", "d_w_pre", "d_dw_post", "d_dres_scale", "d_dw_pre"):
        a = _norm(E, **grad, **{name: q})
        assert L.emb_gated_norm_backward(ctypes.byref(a), P, 1 << 40, None) == bad
    one = (E.EmbTensor * 1)(E.EmbTensor(d_src=P, d_out=P, numel=4, dtype=0))
    assert L.emb_clip_grads(one, 1, 1.0, q, P, 1 << 20, None) == bad
