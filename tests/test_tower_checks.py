"""Refusals of the expert-tower calls: the C entry points reject bad sizes, types, steps and
buffers on the host, and the binding rejects mistyped or short tensors, before anything
reaches a device.  No GPU is needed."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def E():
    from helpers import build_lib
    build_lib()
    import recommender_model_embedding_gb300 as E
    return E


P = 0x1000  # a non-NULL, 16-byte aligned address that is never followed


class FakeCuda:
    """Type, shape and steps of a CUDA tensor, without one."""

    def __init__(self, dtype, *shape, stride=None):
        import torch
        self.dtype, self.shape, self.is_cuda, self.device = getattr(torch, dtype), shape, True, "cuda:0"
        steps, s = [], 1
        for v in reversed(shape):
            steps.insert(0, s)
            s *= v
        self._n, self._dense, self._stride = s, tuple(steps), stride or tuple(steps)

    def stride(self):
        return self._stride

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self._n

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._stride == self._dense

    def data_ptr(self):
        return P


def test_sort_refuses_bad_sizes(E):
    L = E._lib
    sort = lambda n, k, e, ids=P, order=P, pos=P, off=P, ws=P, have=1 << 40: L.emb_expert_sort(
        ids, n, k, e, order, pos, off, ws, have, None)
    for n, k, e in [(-1, 2, 8), (4, 0, 8), (4, E.EXPERT_MAX_K + 1, 8), (4, 2, 0),
                    (4, 2, E.EXPERT_MAX + 1), (1 << 30, 2, 8), (1 << 62, 16, 8)]:
        assert sort(n, k, e) == E.EMB_EINVAL
        assert L.emb_expert_sort_workspace(n, k, e) == -1
    assert sort(4, 2, 8, ids=None) == E.EMB_EINVAL
    assert sort(4, 2, 8, order=None) == E.EMB_EINVAL
    assert sort(4, 2, 8, pos=None) == E.EMB_EINVAL
    assert sort(0, 2, 8, off=None) == E.EMB_EINVAL
    need = L.emb_expert_sort_workspace(1 << 20, 2, 8)
    if need:  # nothing to be short of where one chunk covers the batch
        assert sort(1 << 20, 2, 8, have=need - 1) == E.EMB_EINVAL
        assert sort(1 << 20, 2, 8, ws=P + 4) == E.EMB_EINVAL
        assert sort(1 << 20, 2, 8, ws=None) == E.EMB_EINVAL


@pytest.mark.parametrize("n,k,dim,dtype,ld_in,ld_out", [
    (-1, 2, 8, 0, 8, 8), (4, 0, 8, 0, 8, 8), (4, 17, 8, 0, 8, 8), (4, 2, 0, 0, 8, 8),
    (4, 2, 65537, 0, 1 << 17, 1 << 17), (4, 2, 8, 2, 8, 8), (4, 2, 8, 0, -8, 8), (4, 2, 8, 0, 8, 7),
    (1 << 30, 2, 8, 0, 8, 8)])
def test_row_calls_refuse_bad_sizes(E, n, k, dim, dtype, ld_in, ld_out):
    L = E._lib
    assert L.emb_expert_dispatch(P, ld_in, P, n, k, dim, dtype, P, ld_out, None) == E.EMB_EINVAL
    assert L.emb_expert_dispatch_backward(P, ld_in, P, n, k, dim, dtype, P, ld_out, None) == E.EMB_EINVAL
    assert L.emb_expert_combine(P, ld_in, P, P, n, k, dim, dtype, P, ld_out, None) == E.EMB_EINVAL
    assert L.emb_expert_combine_backward(P, ld_in, P, 8, P, P, n, k, dim, dtype, P, ld_out, P,
                                         None) == E.EMB_EINVAL


def test_row_calls_refuse_missing_and_misaligned_buffers(E):
    L = E._lib
    for i in range(3):
        a = [P, P, P]
        a[i] = None
        assert L.emb_expert_dispatch(a[0], 8, a[1], 4, 2, 8, 0, a[2], 8, None) == E.EMB_EINVAL
        assert L.emb_expert_dispatch_backward(a[0], 8, a[1], 4, 2, 8, 0, a[2], 8, None) == E.EMB_EINVAL
    for i in range(4):
        a = [P, P, P, P]
        a[i] = None
        assert L.emb_expert_combine(a[0], 8, a[1], a[2], 4, 2, 8, 0, a[3], 8, None) == E.EMB_EINVAL
    for i in range(6):
        a = [P] * 6
        a[i] = None
        assert L.emb_expert_combine_backward(a[0], 8, a[1], 8, a[2], a[3], 4, 2, 8, 0, a[4], 8, a[5],
                                             None) == E.EMB_EINVAL
    assert L.emb_expert_dispatch(P + 2, 8, P, 4, 2, 8, 0, P, 8, None) == E.EMB_EINVAL
    assert L.emb_expert_combine(P + 1, 8, P, P, 4, 2, 8, 1, P, 8, None) == E.EMB_EINVAL


def _norm(E, **kw):
    a = dict(n=4, dim=8, x_dtype=0, dtype=0, gate_cols=0, eps=1e-6, d_x=P, d_y=P, d_x_out=P, d_h=P,
             x_ld=8, y_ld=8, x_out_ld=8, h_ld=8)
    a.update(kw)
    return E.EmbNorm(**a)


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(dim=0), dict(dim=8193), dict(x_dtype=2), dict(dtype=3), dict(x_dtype=1, dtype=0),
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(d_gate=P, gate_cols=0), dict(d_gate=P, gate_cols=3), dict(d_y=None, d_gate=P, gate_cols=1),
    dict(d_x=None), dict(d_x_out=None), dict(d_y=None, d_h=None), dict(x_out_ld=7), dict(h_ld=7),
    dict(x_ld=-1), dict(d_x=P + 2), dict(d_h=P + 1)])
def test_norm_refuses(E, bad):
    a = _norm(E, **bad)
    assert E._lib.emb_gated_norm(ctypes.byref(a), None) == E.EMB_EINVAL


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(dim=8193), dict(eps=0.0), dict(d_dh=None, d_dx_out=None), dict(d_x_out=None),
    dict(d_dh=None, d_dw_pre=P), dict(d_y=None), dict(d_y=None, d_dy=None, d_dw_post=P),
    dict(d_dgate=P), dict(dx_ld=7), dict(dy_ld=7), dict(d_gate=P, gate_cols=8, d_dgate=P, dgate_ld=7),
    dict(d_dx=None, d_dy=None)])
def test_norm_backward_refuses(E, bad):
    base = dict(d_x=None, d_h=None, d_dx_out=P, d_dh=P, d_dx=P, d_dy=P, dx_out_ld=8, dh_ld=8, dx_ld=8,
                dy_ld=8)
    base.update(bad)
    a = _norm(E, **base)
    assert E._lib.emb_gated_norm_backward(ctypes.byref(a), P, 1 << 40, None) == E.EMB_EINVAL


def test_norm_backward_refuses_short_workspace(E):
    a = _norm(E, d_x=None, d_h=None, d_dx_out=P, d_dh=P, d_dx=P, d_dy=P, dx_out_ld=8, dh_ld=8, dx_ld=8,
              dy_ld=8)
    need = E.gated_norm_backward_workspace(4, 8)
    for ws, have in ((None, need), (P, need - 1), (P + 4, need)):
        assert E._lib.emb_gated_norm_backward(ctypes.byref(a), ws, have, None) == E.EMB_EINVAL
    assert E._lib.emb_gated_norm_backward(None, P, need, None) == E.EMB_EINVAL
    assert E._lib.emb_gated_norm(None, None) == E.EMB_EINVAL


def test_clip_refuses(E):
    L = E._lib
    one = lambda **kw: (E.EmbTensor * 1)(E.EmbTensor(**{**dict(d_src=P, d_out=P, numel=4, dtype=0), **kw}))
    need = E.clip_grads_workspace(1)
    call = lambda lst, count=1, m=1.0, norm=P, ws=P, have=need: L.emb_clip_grads(
        lst, count, m, norm, ws, have, None)
    assert call(one(numel=-1)) == E.EMB_EINVAL
    assert call(one(dtype=2)) == E.EMB_EINVAL
    assert call(one(d_src=None)) == E.EMB_EINVAL
    assert call(one(d_out=None)) == E.EMB_EINVAL
    assert call(one(d_src=P + 2)) == E.EMB_EINVAL
    assert call(one(d_out=P + 1, dtype=1)) == E.EMB_EINVAL
    assert call(one(), m=-1.0) == E.EMB_EINVAL
    assert call(one(), m=float("nan")) == E.EMB_EINVAL
    assert call(one(), norm=None) == E.EMB_EINVAL
    assert call(one(), ws=None) == E.EMB_EINVAL
    assert call(one(), have=need - 1) == E.EMB_EINVAL
    assert call(one(), count=-1) == E.EMB_EINVAL
    assert call(None, count=1) == E.EMB_EINVAL
    assert call(None, count=65537, have=1 << 40) == E.EMB_EINVAL
    assert E.clip_grads_workspace(65537) == -1


def test_binding_checks_tensors(E):
    F = FakeCuda
    with pytest.raises(ValueError, match="ids"):
        E.expert_sort(F("int32", 4, 2), 8, F("int32", 8), F("int32", 8), F("int32", 9))
    with pytest.raises(ValueError, match="offsets"):
        E.expert_sort(F("int64", 4, 2), 8, F("int32", 8), F("int32", 8), F("int32", 8))
    with pytest.raises(ValueError, match="pos"):  # 7 places for 4 rows
        E.expert_dispatch(F("float32", 4, 8), F("int32", 7), F("float32", 8, 8))
    with pytest.raises(ValueError, match="xs"):
        E.expert_dispatch(F("float32", 4, 8), F("int32", 8), F("float32", 7, 8))
    with pytest.raises(ValueError, match="xs"):
        E.expert_dispatch(F("float32", 4, 8), F("int32", 8), F("bfloat16", 8, 8))
    with pytest.raises(ValueError, match="float16"):
        E.expert_dispatch(F("float16", 4, 8), F("int32", 8), F("float16", 8, 8))
    with pytest.raises(ValueError, match="adjacent"):
        E.expert_dispatch(F("float32", 4, 8, stride=(1, 4)), F("int32", 8), F("float32", 8, 8))
    with pytest.raises(ValueError, match="w"):
        E.expert_combine(F("float32", 8, 8), F("int32", 8), F("float32", 7), F("float32", 4, 8))
    with pytest.raises(ValueError, match="gate"):
        E.gated_norm(F("float32", 4, 8), F("float32", 4, 8), F("float32", 4, 8), None,
                     gate=F("float32", 4, 2))
    with pytest.raises(ValueError, match="w_pre"):
        E.gated_norm(F("float32", 4, 8), None, None, F("float32", 4, 8), w_pre=F("float32", 9))
    with pytest.raises(ValueError, match="workspace"):
        E.gated_norm_backward(F("float32", 4, 8), F("float32", 4, 8), F("float32", 4, 8), None,
                              F("float32", 4, 8), None, workspace=F("uint8", 8))
    with pytest.raises(ValueError, match="out"):
        E.clip_grads([F("float32", 8)], 1.0, F("float32", 1), out=[F("float32", 7)])
    with pytest.raises(ValueError, match="out"):
        E.clip_grads([F("float32", 8)], 1.0, F("float32", 1), out=[])
    with pytest.raises(ValueError, match="contiguous"):
        E.clip_grads([F("float32", 4, 8, stride=(1, 4))], 1.0, F("float32", 1))
    with pytest.raises(ValueError, match="norm"):
        E.clip_grads([F("float32", 8)], 1.0, F("float64", 1))
