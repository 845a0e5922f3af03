"""GB300-native sparse embedding layer for DLRM-style recommenders.

A thin binding over libemb.so, the CUDA library declared in include/emb.h: ctypes, and a small
compiled module for the expert tower's calls (csrc/py_tower.cpp).  Every method marshals its
arguments (torch tensors -> device pointers, the current CUDA stream) and calls the C entry
point of the same name; all arithmetic runs in the library's kernels.  There is no CPU path:
if libemb.so is missing this package fails to import, and if the compiled module is missing the
tower's calls fail.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libemb.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the CUDA library first "
        "(python -c 'import __graft_entry__ as g; g.build()' or "
        "python recommender_model_embedding_gb300/build.py)")

_lib = ctypes.CDLL(LIB_PATH)

TOWER_PATH = os.path.join(_HERE, "_tower.so")


class _LoadTower:
    """Stands in for the compiled module of the tower's calls until the first of them: the module
    needs torch, and the rest of the package imports and runs without either."""

    def __getattr__(self, name):
        import importlib

        if not os.path.exists(TOWER_PATH):
            raise ImportError(f"{TOWER_PATH} is missing: the tower's calls need it, built with torch "
                              "installed (python recommender_model_embedding_gb300/build.py)")

        import torch  # (its libraries have to be there first)

        global _tower
        tower = importlib.import_module(__name__ + "._tower")
        if tower.torch_version != torch.__version__:
            _tower = self  # (importing a submodule puts it in this stand-in's place)
            raise ImportError(f"{TOWER_PATH} was built for torch {tower.torch_version}, this is "
                              f"{torch.__version__}: build it again")
        return getattr(tower, name)


_tower = _LoadTower()

EMB_OK, EMB_EINVAL, EMB_ENOMEM, EMB_ESTATE, EMB_ECUDA = 0, 1, 2, 3, 4
FLAG_ID_RANGE, FLAG_BAD_KEY, FLAG_TABLE_FULL, FLAG_BAD_OFFSETS = 0x1, 0x2, 0x4, 0x8
FLAG_WAIT_LIMIT = 0x10
F32, BF16 = 0, 1
POOL_SUM, POOL_MEAN = 0, 1
ADAGRAD, ADAGRAD_ROWWISE = 0, 1


class EmbConfig(ctypes.Structure):
    _fields_ = [("num_tables", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("rows", ctypes.POINTER(ctypes.c_int64)), ("hashed", ctypes.c_int32),
                ("capacity", ctypes.c_int64), ("dtype", ctypes.c_int32),
                ("pooling", ctypes.c_int32), ("optimizer", ctypes.c_int32),
                ("lr", ctypes.c_float), ("eps", ctypes.c_float), ("init_acc", ctypes.c_float),
                ("init_lo", ctypes.c_float), ("init_hi", ctypes.c_float),
                ("hash_init", ctypes.c_float), ("seed", ctypes.c_uint64),
                ("max_batch", ctypes.c_int64), ("max_lookups", ctypes.c_int64)]


# The tower's structures and signatures, for calls of the C entry points themselves (the package's own
# go through the compiled module).
class EmbNorm(ctypes.Structure):
    _P, _I64 = ctypes.c_void_p, ctypes.c_int64
    _fields_ = [("n", _I64), ("dim", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("gate_cols", ctypes.c_int32), ("eps", ctypes.c_float),
                ("d_y", _P), ("d_gate", _P), ("d_w_post", _P), ("d_res_scale", _P),
                ("d_w_pre", _P), ("d_x_out", _P), ("y_ld", _I64), ("gate_ld", _I64),
                ("x_out_ld", _I64), ("d_x", _P), ("d_h", _P), ("x_ld", _I64), ("h_ld", _I64),
                ("d_dx_out", _P), ("d_dh", _P), ("d_dx", _P), ("d_dy", _P), ("d_dgate", _P),
                ("d_dw_post", _P), ("d_dres_scale", _P), ("d_dw_pre", _P), ("dx_out_ld", _I64),
                ("dh_ld", _I64), ("dx_ld", _I64), ("dy_ld", _I64), ("dgate_ld", _I64)]


class EmbTensor(ctypes.Structure):
    _fields_ = [("d_src", ctypes.c_void_p), ("d_out", ctypes.c_void_p), ("numel", ctypes.c_int64),
                ("dtype", ctypes.c_int32)]


_P, _I64, _I32, _U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
_SIGS = {
    "emb_status_str": ([ctypes.c_int], ctypes.c_char_p),
    "emb_create": ([ctypes.POINTER(EmbConfig), ctypes.POINTER(_P)], ctypes.c_int),
    "emb_create_tiered": ([ctypes.POINTER(EmbConfig), _I64, ctypes.POINTER(_P)], ctypes.c_int),
    "emb_destroy": ([_P], None),
    "emb_forward": ([_P, _P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "emb_interact": ([_P, _P, _P, _I64, _P, _P], ctypes.c_int),
    "emb_interact_backward": ([_P, _P, _P, _P, _I64, _P, _P, _P], ctypes.c_int),
    "emb_backward_adagrad": ([_P, _P, _P], ctypes.c_int),
    "emb_forward_interact": ([_P, _P, _P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "emb_backward_interact_adagrad": ([_P, _P, _P, _P, _P], ctypes.c_int),
    "emb_train_step_host": ([_P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P], ctypes.c_int),
    "emb_get_status": ([_P, _P, ctypes.POINTER(_U32)], ctypes.c_int),
    "emb_read_rows": ([_P, _I32, _P, _I64, _P, _P, _P], ctypes.c_int),
    "emb_read_unique": ([_P, _P, _P, _I64, ctypes.POINTER(_I64)], ctypes.c_int),
    "emb_export_hash": ([_P, _P, _P, _P, _I64, ctypes.POINTER(_I64)], ctypes.c_int),
    "emb_profile": ([_P, _I32], ctypes.c_int),
    "emb_profile_read": ([_P, _I32, ctypes.POINTER(ctypes.c_char_p), ctypes.POINTER(ctypes.c_double),
                          ctypes.POINTER(_I64)], ctypes.c_int),
    "emb_profile_reset": ([_P], ctypes.c_int),
    "emb_launch_count": ([_P], _I64),
    "emb_step_tracks_once": ([_P], _I32),
    "emb_set_admission": ([_P, _U32], ctypes.c_int),
    "emb_set_adagrad_decay": ([_P, ctypes.c_float, _U32], ctypes.c_int),
    "emb_quantize_rows": ([_P, _I64, _I32, _P, _P, _P], ctypes.c_int),
    "emb_cross_forward": ([_P, _P, _P, _P, _I64, _I32, _P, _P], ctypes.c_int),
    "emb_cross_backward": ([_P, _P, _P, _P, _I64, _I32, _P, _P, _P, _P, _P], ctypes.c_int),
    "emb_dequantize_rows": ([_P, _P, _I64, _I32, _P, _P], ctypes.c_int),
    "emb_evict": ([_P, _U32, _U32, _P, ctypes.POINTER(_I64)], ctypes.c_int),
    "emb_read_key_stats": ([_P, _P, _I64, _P, _P], ctypes.c_int),
    "emb_prefetch": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "emb_set_tier_watermark": ([_P, _I64, _I64], ctypes.c_int),
    "emb_tier_occupancy": ([_P, ctypes.POINTER(_I64)], ctypes.c_int),
    "emb_expert_sort_workspace": ([_I64, _I32, _I32], _I64),
    "emb_expert_sort": ([_P, _I64, _I32, _I32, _P, _P, _P, _P, _I64, _P], ctypes.c_int),
    "emb_expert_dispatch": ([_P, _I64, _P, _I64, _I32, _I32, _I32, _P, _I64, _P], ctypes.c_int),
    "emb_expert_dispatch_backward": ([_P, _I64, _P, _I64, _I32, _I32, _I32, _P, _I64, _P], ctypes.c_int),
    "emb_expert_combine": ([_P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P, _I64, _P], ctypes.c_int),
    "emb_expert_combine_backward": ([_P, _I64, _P, _I64, _P, _P, _I64, _I32, _I32, _I32, _P, _I64,
                                     _P, _P], ctypes.c_int),
    "emb_gated_norm": ([ctypes.POINTER(EmbNorm), _P], ctypes.c_int),
    "emb_gated_norm_backward_workspace": ([_I64, _I32], _I64),
    "emb_gated_norm_backward": ([ctypes.POINTER(EmbNorm), _P, _I64, _P], ctypes.c_int),
    "emb_clip_grads_workspace": ([_I64], _I64),
    "emb_clip_grads": ([ctypes.POINTER(EmbTensor), _I64, ctypes.c_float, _P, _P, _I64, _P], ctypes.c_int),
    "emb_unique_keys_noalloc": ([_P, _I64, _P, _P, _P, _P], ctypes.c_int),
}
NOALLOC_MAX_KEYS = 524288


CROSS_MAX_K = 9216


def cross_forward(x0, xl, w, b, out, stream=None):
    """One cross layer: out = x0 * (xl . w) + b + xl per sample (CUDA tensors [B, K], [K])."""
    B, K = x0.shape
    _check("emb_cross_forward",
           _lib.emb_cross_forward(_dptr(x0, "f32", B * K, "x0"), _dptr(xl, "f32", B * K, "xl"),
                                  _dptr(w, "f32", K, "w"), _dptr(b, "f32", K, "b"), B, K,
                                  _dptr(out, "f32", B * K, "out"), _stream(stream)))


def cross_backward(x0, xl, w, dout, dx0, dxl, dw, db, stream=None):
    """Gradients of one cross layer (dw, db overwritten); CUDA tensors, asynchronous."""
    B, K = x0.shape
    _check("emb_cross_backward",
           _lib.emb_cross_backward(_dptr(x0, "f32", B * K, "x0"), _dptr(xl, "f32", B * K, "xl"),
                                   _dptr(w, "f32", K, "w"), _dptr(dout, "f32", B * K, "dout"), B, K,
                                   _dptr(dx0, "f32", B * K, "dx0"), _dptr(dxl, "f32", B * K, "dxl"),
                                   _dptr(dw, "f32", K, "dw"), _dptr(db, "f32", K, "db"),
                                   _stream(stream)))


def quantize_rows(x, q, scale, stream=None):
    """int8 codes `q` (int8 [n, d]) and per-row scales `scale` (float32 [n]) of the rows of
    `x` (float32 [n, d]); CUDA tensors, asynchronous."""
    n, d = x.shape
    _check("emb_quantize_rows",
           _lib.emb_quantize_rows(_dptr(x, "f32", n * d, "x"), n, d, _dptr(q, "i8", n * d, "q"),
                                  _dptr(scale, "f32", n, "scale"), _stream(stream)))


def dequantize_rows(q, scale, x, stream=None):
    """x = code * scale row by row (CUDA tensors, asynchronous)."""
    n, d = q.shape
    _check("emb_dequantize_rows",
           _lib.emb_dequantize_rows(_dptr(q, "i8", n * d, "q"), _dptr(scale, "f32", n, "scale"),
                                    n, d, _dptr(x, "f32", n * d, "x"), _stream(stream)))


def unique_keys_noalloc(keys, unique, inverse, num_unique, stream=None):
    """Unique keys of `keys` (int64 CUDA tensor) into `unique` (int64, same length),
    `inverse` (int32, same length) and `num_unique` (int32, one element), with no device
    allocation (scratch lives in the library's fixed device array).  Asynchronous."""
    n = keys.numel()
    _check("emb_unique_keys_noalloc",
           _lib.emb_unique_keys_noalloc(_dptr(keys, "i64", n, "keys"), n,
                                        _dptr(unique, "i64", n, "unique"),
                                        _dptr(inverse, "i32", n, "inverse"),
                                        _dptr(num_unique, "i32", 1, "num_unique"), _stream(stream)))
for _name, (_args, _res) in _SIGS.items():
    _f = getattr(_lib, _name)
    _f.argtypes = _args
    _f.restype = _res


class EmbError(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} failed: {status_str(status)} ({status})")
        self.status = status


def status_str(s: int) -> str:
    return _lib.emb_status_str(int(s)).decode()


def _check(call: str, st: int):
    if st != EMB_OK:
        raise EmbError(call, st)


_DTYPES = {"i64": "int64", "i32": "int32", "f32": "float32", "i8": "int8"}


def _dptr(t, dtype: Optional[str] = None, numel: int = 0, name: str = "tensor") -> Optional[int]:
    """Device pointer of a contiguous CUDA tensor (None passes NULL).  With dtype ("i64",
    "i32", "f32", "i8") and numel, the tensor must have that element type and at least that
    many elements; a mismatch raises ValueError before anything reaches the device (a short
    or mistyped buffer would otherwise be read or written past its end)."""
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CUDA tensor")
    if dtype is not None and str(t.dtype) != "torch." + _DTYPES[dtype]:
        raise ValueError(f"{name}: expected dtype {_DTYPES[dtype]}, got {t.dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, at least {numel} needed")
    return t.data_ptr()


def _hptr(a, dtype: Optional[str] = None, numel: int = 0, name: str = "array") -> Optional[int]:
    """Host pointer of a contiguous numpy array or CPU tensor (None passes NULL), with the
    same dtype and size checks as _dptr."""
    if a is None:
        return None
    if hasattr(a, "ctypes"):
        if not a.flags["C_CONTIGUOUS"]:
            raise ValueError(f"{name}: expected a C-contiguous array")
        if dtype is not None and str(a.dtype) != _DTYPES[dtype]:
            raise ValueError(f"{name}: expected dtype {_DTYPES[dtype]}, got {a.dtype}")
        if a.size < numel:
            raise ValueError(f"{name}: {a.size} elements, at least {numel} needed")
        return a.ctypes.data
    if a.is_cuda or not a.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous CPU tensor")
    if dtype is not None and str(a.dtype) != "torch." + _DTYPES[dtype]:
        raise ValueError(f"{name}: expected dtype {_DTYPES[dtype]}, got {a.dtype}")
    if a.numel() < numel:
        raise ValueError(f"{name}: {a.numel()} elements, at least {numel} needed")
    return a.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


# ---- expert tower (context-free; arguments are checked and passed on by the _tower module) ----
# A call's tensors, workspace and stream are on one device (else ValueError), and the call runs there
# whichever device is current; the *_workspace sizes are the current device's.  The calls are no
# autograd functions; what one writes counts as changed in place, so a backward that saved it says so.
EXPERT_MAX, EXPERT_MAX_K, EXPERT_MAX_DIM, NORM_MAX_DIM = 1024, 16, 65536, 8192


def expert_sort_workspace(n: int, k: int, num_experts: int) -> int:
    """Bytes of workspace of expert_sort."""
    return int(_lib.emb_expert_sort_workspace(n, k, num_experts))


def expert_sort(ids, num_experts: int, order, pos, offsets, workspace=None, stream=None):
    """Sort the slots of `ids` (int64 [n, k]: the experts each row chose; outside
    [0, num_experts): dropped) stably by expert into `order` (int32 [n*k], slot at each place),
    `pos` (int32 [n*k], place of each slot, -1 - place when dropped) and `offsets` (int32
    [num_experts + 1], first place of each expert; the last: kept slots).  Asynchronous."""
    _tower.sort(ids, num_experts, order, pos, offsets, workspace, stream)


def expert_dispatch(x, pos, xs, stream=None):
    """xs[pos[i, j]] = x[i] for the kept slots, zero rows at the dropped ones' places.  x [n, d]
    and xs [n*k, d] float32 or bfloat16, rows any step apart; pos of expert_sort."""
    _tower.dispatch(x, pos, xs, stream)


def expert_dispatch_backward(dxs, pos, dx, stream=None):
    """dx[i] = sum of dxs over row i's kept places (dxs [n*k, d], dx [n, d])."""
    _tower.dispatch_backward(dxs, pos, dx, stream)


def expert_combine(ys, pos, w, out, stream=None):
    """out[i] = sum over row i's kept slots of w[i, j] * ys[place] (ys [n*k, d], w float32
    [n, k], out [n, d])."""
    _tower.combine(ys, pos, w, out, stream)


def expert_combine_backward(dout, ys, pos, w, dys, dw, stream=None):
    """Gradients of expert_combine: dys [n*k, d] (zero rows at dropped places) and dw float32
    [n, k] (0 when dropped)."""
    _tower.combine_backward(dout, ys, pos, w, dys, dw, stream)


def gated_norm(x, y, x_out, h, gate=None, w_post=None, res_scale=None, w_pre=None,
               eps: float = 1e-6, stream=None):
    """The end of a residual block and the start of the next in one pass:
    x_out = x + res_scale * sigmoid(gate) * (y / rms(y) * w_post), h = x_out / rms(x_out) * w_pre.
    x, x_out [n, d] float32 or bfloat16; y, h, gate ([n, d], or [n, 1]: one gate a row) of one
    type, bfloat16 or as x; vectors float32 [d], None counts as ones.  y None: h from x alone
    (x_out is then not written); h None: only x_out.  x_out may be x.  Asynchronous."""
    _tower.norm(x, y, x_out, h, gate, w_post, res_scale, w_pre, eps, stream)


def gated_norm_backward_workspace(n: int, d: int) -> int:
    """Bytes of workspace of gated_norm_backward."""
    return int(_lib.emb_gated_norm_backward_workspace(n, d))


def gated_norm_backward(dx_out, dh, x_out, y, dx, dy, gate=None, w_post=None, res_scale=None,
                        w_pre=None, dgate=None, dw_post=None, dres_scale=None, dw_pre=None,
                        eps: float = 1e-6, workspace=None, stream=None):
    """Gradients of gated_norm from dx_out (None: zero) and dh (None: no h), with x_out, y, gate
    and the vectors of the forward: dx, dy, dgate and the vectors' (float32 [d], overwritten).
    Outputs may be None; dx may be dx_out or x_out, and dy y.  Asynchronous."""
    _tower.norm_backward(dx_out, dh, x_out, y, dx, dy, gate, w_post, res_scale, w_pre, dgate, dw_post,
                         dres_scale, dw_pre, eps, workspace, stream)


def clip_grads_workspace(count: int) -> int:
    """Bytes of workspace of clip_grads."""
    return int(_lib.emb_clip_grads_workspace(count))


def clip_grads(grads, max_norm: float, norm, out=None, workspace=None, stream=None):
    """norm (float32 [1]) = sqrt(sum of squares over all of `grads`), and every gradient times
    min(1, max_norm / norm), in place or into `out` (contiguous CUDA tensors, float32 or
    bfloat16, of the gradients' types and sizes; none may overlap another, so a shared gradient
    is listed once).  An infinite or NaN norm clips nothing.  The embedding layer's own gradients,
    applied by its backward, are not part of the norm.  Asynchronous."""
    _tower.clip(grads, max_norm, norm, out, workspace, stream)


class EmbCtx:
    """One embedding layer (tables, accumulators, workspace) owned by libemb.so."""

    def __init__(self, num_tables: int, dim: int, rows: Optional[Sequence[int]] = None,
                 hashed: bool = False, capacity: int = 0, dtype: int = F32,
                 pooling: int = POOL_SUM, optimizer: int = ADAGRAD, lr: float = 0.01,
                 eps: float = 1e-8, init_acc: float = 0.1, init_lo: float = -0.05,
                 init_hi: float = 0.05, hash_init: float = 0.0, seed: int = 0,
                 max_batch: int = 1, max_lookups: int = 1, cache_rows: int = 0):
        self._h = None
        self.T, self.D = num_tables, dim
        self.hashed = bool(hashed)
        self.rowwise = optimizer == ADAGRAD_ROWWISE
        rows_arr = None
        if rows is not None:
            rows_arr = (ctypes.c_int64 * len(rows))(*[int(r) for r in rows])
        cfg = EmbConfig(num_tables, dim,
                        ctypes.cast(rows_arr, ctypes.POINTER(ctypes.c_int64)) if rows_arr else None,
                        int(hashed), int(capacity), int(dtype), int(pooling), int(optimizer),
                        lr, eps, init_acc, init_lo, init_hi, hash_init,
                        int(seed) & (2**64 - 1), int(max_batch), int(max_lookups))
        h = _P()
        if cache_rows > 0:  # tiered static tables: host tier plus an HBM cache of cache_rows
            _check("emb_create_tiered", _lib.emb_create_tiered(ctypes.byref(cfg), int(cache_rows),
                                                               ctypes.byref(h)))
        else:
            _check("emb_create", _lib.emb_create(ctypes.byref(cfg), ctypes.byref(h)))
        self._h = h
        self.F = num_tables + 1
        self.out_width = dim + self.F * (self.F - 1) // 2
        self._last = ("", 0)  # kind and batch of the last forward (sizes of its backward)

    @classmethod
    def from_workload(cls, w, max_batch: Optional[int] = None, max_lookups: Optional[int] = None,
                      cache_rows: int = 0):
        """Context for a workload description (any object with the fields of synth.Workload);
        cache_rows > 0: static tables in the host tier with an HBM cache of that many rows."""
        return cls(w.num_tables, w.dim, rows=w.rows, hashed=w.hashed, capacity=w.capacity,
                   dtype=BF16 if w.dtype == "bf16" else F32,
                   pooling=POOL_MEAN if w.pooling == "mean" else POOL_SUM,
                   optimizer=ADAGRAD_ROWWISE if w.optimizer == "adagrad_row" else ADAGRAD,
                   lr=w.lr, eps=w.eps, init_acc=w.init_acc, init_lo=w.init_lo,
                   init_hi=w.init_hi, hash_init=w.hash_init, seed=w.seed,
                   max_batch=max_batch or w.batch, max_lookups=max_lookups or w.max_lookups(),
                   cache_rows=cache_rows)

    def close(self):
        if self._h:
            _lib.emb_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    # ---- compute calls (stream-ordered, asynchronous) ----
    # Every tensor is checked for dtype and size against the call's layout before the
    # library sees its pointer (the library trusts the caller's buffers).
    def _lookups(self, ids, offsets, batch: int):
        nnz = ids.numel()
        if offsets is not None:
            _dptr(offsets, "i32", batch * self.T + 1, "offsets")
        elif nnz != batch * self.T:
            raise ValueError(f"ids: {nnz} elements for a one-hot batch of {batch} x {self.T}")
        _dptr(ids, "i64", nnz, "ids")
        return nnz

    def forward(self, ids, offsets, batch: int, pooled, stream=None):
        nnz = self._lookups(ids, offsets, batch)
        _check("emb_forward", _lib.emb_forward(self._h, _dptr(ids), _dptr(offsets), nnz, batch,
                                               _dptr(pooled, "f32", batch * self.T * self.D, "pooled"),
                                               _stream(stream)))
        self._last = ("forward", batch)

    def interact(self, dense, pooled, batch: int, out, stream=None):
        _check("emb_interact",
               _lib.emb_interact(self._h, _dptr(dense, "f32", batch * self.D, "dense"),
                                 _dptr(pooled, "f32", batch * self.T * self.D, "pooled"), batch,
                                 _dptr(out, "f32", batch * self.out_width, "out"), _stream(stream)))

    def interact_backward(self, dout, dense, pooled, batch: int, ddense, dpooled, stream=None):
        BD, BTD = batch * self.D, batch * self.T * self.D
        _check("emb_interact_backward",
               _lib.emb_interact_backward(self._h, _dptr(dout, "f32", batch * self.out_width, "dout"),
                                          _dptr(dense, "f32", BD, "dense"),
                                          _dptr(pooled, "f32", BTD, "pooled"), batch,
                                          _dptr(ddense, "f32", BD, "ddense"),
                                          _dptr(dpooled, "f32", BTD, "dpooled"), _stream(stream)))

    def backward_adagrad(self, dpooled, stream=None):
        kind, batch = self._last
        need = batch * self.T * self.D if kind == "forward" else 0
        _check("emb_backward_adagrad",
               _lib.emb_backward_adagrad(self._h, _dptr(dpooled, "f32", need, "dpooled"),
                                         _stream(stream)))

    def forward_interact(self, ids, offsets, batch: int, dense, out, stream=None):
        nnz = self._lookups(ids, offsets, batch)
        _check("emb_forward_interact",
               _lib.emb_forward_interact(self._h, _dptr(ids), _dptr(offsets), nnz, batch,
                                         _dptr(dense, "f32", batch * self.D, "dense"),
                                         _dptr(out, "f32", batch * self.out_width, "out"),
                                         _stream(stream)))
        self._last = ("forward_interact", batch)

    def backward_interact_adagrad(self, dout, dense, ddense, stream=None):
        kind, batch = self._last
        b = batch if kind == "forward_interact" else 0
        _check("emb_backward_interact_adagrad",
               _lib.emb_backward_interact_adagrad(self._h, _dptr(dout, "f32", b * self.out_width, "dout"),
                                                  _dptr(dense, "f32", b * self.D, "dense"),
                                                  _dptr(ddense, "f32", b * self.D, "ddense"),
                                                  _stream(stream)))

    def train_step_host(self, ids, offsets, batch: int, dense, dout, out, ddense, stream=None):
        """Host buffers (pinned CPU tensors or numpy arrays); asynchronous on `stream`."""
        nnz = int(ids.shape[0])
        if offsets is None and nnz != batch * self.T:
            raise ValueError(f"ids: {nnz} elements for a one-hot batch of {batch} x {self.T}")
        W = self.out_width
        _check("emb_train_step_host",
               _lib.emb_train_step_host(self._h, _hptr(ids, "i64", nnz, "ids"),
                                        _hptr(offsets, "i32", batch * self.T + 1, "offsets"), nnz,
                                        batch, _hptr(dense, "f32", batch * self.D, "dense"),
                                        _hptr(dout, "f32", batch * W, "dout"),
                                        _hptr(out, "f32", batch * W, "out"),
                                        _hptr(ddense, "f32", batch * self.D, "ddense"),
                                        _stream(stream)))

    # ---- synchronous queries ----
    def get_status(self, stream=None) -> int:
        f = _U32(0)
        _check("emb_get_status", _lib.emb_get_status(self._h, _stream(stream), ctypes.byref(f)))
        return int(f.value)

    def read_rows(self, table: int, ids):
        """(w [n, D] float32, acc [n, D or 1] float32, found [n] bool) as numpy arrays."""
        import numpy as np
        ids = np.ascontiguousarray(ids, dtype=np.int64)
        n = ids.shape[0]
        w = np.empty((n, self.D), np.float32)
        acc = np.empty((n, 1 if self.rowwise else self.D), np.float32)
        found = np.empty(n, np.int8)
        _check("emb_read_rows", _lib.emb_read_rows(self._h, table, _hptr(ids), n, _hptr(w),
                                                   _hptr(acc), _hptr(found)))
        return w, acc, found.astype(bool)

    def read_unique(self):
        """(keys int64 [U], counts int32 [U]) of the last forward, in no fixed order."""
        import numpy as np
        U = _I64(0)
        _check("emb_read_unique", _lib.emb_read_unique(self._h, None, None, 0, ctypes.byref(U)))
        keys = np.empty(U.value, np.int64)
        counts = np.empty(U.value, np.int32)
        _check("emb_read_unique", _lib.emb_read_unique(self._h, _hptr(keys), _hptr(counts),
                                                       U.value, ctypes.byref(U)))
        return keys, counts

    def export_hash(self):
        """(keys int64 [n], w [n, D], acc [n, D or 1]) of every occupied slot."""
        import numpy as np
        n = _I64(0)
        _check("emb_export_hash", _lib.emb_export_hash(self._h, None, None, None, 0, ctypes.byref(n)))
        cap = n.value
        keys = np.empty(cap, np.int64)
        w = np.empty((cap, self.D), np.float32)
        acc = np.empty((cap, 1 if self.rowwise else self.D), np.float32)
        _check("emb_export_hash", _lib.emb_export_hash(self._h, _hptr(keys), _hptr(w), _hptr(acc),
                                                       cap, ctypes.byref(n)))
        return keys[:min(cap, n.value)], w[:min(cap, n.value)], acc[:min(cap, n.value)]

    def profile(self, enable: bool):
        _check("emb_profile", _lib.emb_profile(self._h, 1 if enable else 0))

    def profile_read(self) -> dict:
        """{kernel name: (total ms, launches)} for kernels launched since the last reset."""
        out = {}
        idx = 0
        name, ms, n = ctypes.c_char_p(), ctypes.c_double(), _I64()
        while _lib.emb_profile_read(self._h, idx, ctypes.byref(name), ctypes.byref(ms),
                                    ctypes.byref(n)) == EMB_OK:
            if n.value:
                out[name.value.decode()] = (ms.value, n.value)
            idx += 1
        return out

    def profile_reset(self):
        _check("emb_profile_reset", _lib.emb_profile_reset(self._h))

    def launch_count(self) -> int:
        return int(_lib.emb_launch_count(self._h))

    def set_adagrad_decay(self, rate: float, period_steps: int):
        """Adagrad Decay: accumulators discounted by `rate` per period of `period_steps`
        backward steps, applied when a row is next updated (0 steps: off)."""
        _check("emb_set_adagrad_decay", _lib.emb_set_adagrad_decay(self._h, float(rate),
                                                                   int(period_steps)))

    def set_admission(self, min_count: int):
        """Hashed tables: hold a key's updates until it has been looked up min_count times
        over all steps (0 or 1: no hold).  The first call starts the per-key counts and last
        steps that admission and eviction read."""
        _check("emb_set_admission", _lib.emb_set_admission(self._h, int(min_count)))

    def evict(self, max_idle_steps: int, min_count: int, stream=None, wait: bool = True):
        """Hashed tables: remove keys idle for more than max_idle_steps backward steps
        (max_idle_steps > 0) or looked up fewer than min_count times.  wait=True: waits and
        returns how many were removed; wait=False: only enqueues (returns None)."""
        n = _I64(0)
        _check("emb_evict", _lib.emb_evict(self._h, int(max_idle_steps), int(min_count),
                                           _stream(stream), ctypes.byref(n) if wait else None))
        return int(n.value) if wait else None

    def prefetch(self, ids, offsets, batch: int, stream=None):
        """Tiered tables: copy a later batch's uncached rows into the HBM cache, enqueued on
        `stream` (a second stream overlaps it with the current step); the next forward,
        eviction or watermark check waits for it.  ids/offsets as for forward, ready in the
        order of `stream` (e.g. stream.wait_stream after copying them on another stream)
        and kept alive until the stream has run it."""
        nnz = self._lookups(ids, offsets, batch)
        _check("emb_prefetch", _lib.emb_prefetch(self._h, _dptr(ids), _dptr(offsets), nnz, batch,
                                                 _stream(stream)))

    def set_tier_watermark(self, high: int, low: int = 0):
        """Tiered tables: after every backward step, when more than `high` cache rows are in
        use, write the longest-idle rows back until at most `low` remain (high = 0: off)."""
        _check("emb_set_tier_watermark", _lib.emb_set_tier_watermark(self._h, int(high), int(low)))

    def tier_occupancy(self) -> int:
        """Tiered tables: cache rows in use (waits for the device)."""
        n = _I64(0)
        _check("emb_tier_occupancy", _lib.emb_tier_occupancy(self._h, ctypes.byref(n)))
        return int(n.value)

    def key_stats(self, keys):
        """(lookup counts uint32, last step uint32) of hashed keys (0, 0: absent)."""
        import numpy as np
        keys = np.ascontiguousarray(keys, dtype=np.int64)
        cnt = np.empty(keys.size, np.uint32)
        last = np.empty(keys.size, np.uint32)
        _check("emb_read_key_stats", _lib.emb_read_key_stats(self._h, _hptr(keys), keys.size,
                                                             _hptr(cnt), _hptr(last)))
        return cnt, last

    def step_tracks_once(self) -> bool:
        """Whether the last forward's step updates rows looked up once in the backward."""
        return int(_lib.emb_step_tracks_once(self._h)) == 1
