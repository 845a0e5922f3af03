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


def _each_call(E, make):
    """(call, inputs, outputs) of every tower call, on tensors from make(shape, dtype)."""
    n, k, d, e = 6, 2, 16, 4
    f, i = torch.float32, torch.int32
    x, w, xs = lambda: make((n, d), f), lambda: make((n, k), f), lambda: make((n * k, d), f)
    ids, pos = make((n, k), torch.int64), make((n * k,), i)
    o3 = make((n * k,), i), make((n * k,), i), make((e + 1,), i)
    yield lambda: E.expert_sort(ids, e, *o3), [ids], o3
    E.expert_sort(ids, e, make((n * k,), i), pos, make((e + 1,), i))
    a, b = x(), xs()
    yield lambda: E.expert_dispatch(a, pos, b), [a, pos], [b]
    c, dd = xs(), x()
    yield lambda: E.expert_dispatch_backward(c, pos, dd), [c, pos], [dd]
    y, ww, o = xs(), w(), x()
    yield lambda: E.expert_combine(y, pos, ww, o), [y, pos, ww], [o]
    do, dy, dw = x(), xs(), w()
    yield lambda: E.expert_combine_backward(do, y, pos, ww, dy, dw), [do, y, pos, ww], [dy, dw]
    g, h, v = x(), x(), [make((d,), f) for _ in range(6)]
    yield lambda: E.gated_norm(a, do, o, h, gate=g, w_post=v[0]), [a, do, g, v[0]], [o, h]
    dx, dy2, dg = x(), x(), x()
    yield (lambda: E.gated_norm_backward(a, h, o, do, dx, dy2, gate=g, w_post=v[0], dgate=dg, dw_post=v[3],
                                         dres_scale=v[4], dw_pre=v[5]), [a, h, o, do, g, v[0]], [dx, dy2, dg] + v[3:])
    norm, into = make((1,), f), [x(), xs()]
    yield lambda: E.clip_grads([dx, dy], 1.0, norm, out=into), [dx, dy], into + [norm]
    yield lambda: E.clip_grads(into, 1.0, norm), [], into + [norm]


def _make(shape, dtype):
    if dtype.is_floating_point:
        return torch.randn(shape, device="cuda").to(dtype)
    return torch.randint(0, 4, shape, dtype=dtype, device="cuda")


def test_written_tensors_are_new_to_autograd(E):
    for call, ins, outs in _each_call(E, _make):
        before = [t._version for t in ins], [t._version for t in outs]
        call()
        assert [t._version for t in ins] == before[0]
        assert all(t._version > b for t, b in zip(outs, before[1]))
    x = torch.randn((5, 16), device="cuda", requires_grad=True)
    kept = x.exp()  # its backward needs the values it has now
    E.gated_norm(x.detach(), None, None, kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        kept.sum().backward()
    # an x_out beside no block is not written
    unwritten = torch.zeros((5, 16), device="cuda")
    E.gated_norm(x.detach(), None, unwritten, kept)
    assert unwritten._version == 0 and not bool(unwritten.any())


def test_inference_tensors_and_subclasses(E):
    """Tensors without versions, and tensors of a subclass of torch's, are taken like any other."""
    class Named(torch.Tensor):
        pass

    with torch.inference_mode():
        for call, _, _ in _each_call(E, _make):
            call()
    for call, _, _ in _each_call(E, lambda s, t: _make(s, t).as_subclass(Named)):
        call()
    x, y = _make((9, 33), torch.float32), _make((9, 33), torch.float32)
    a, b = torch.empty_like(x), torch.empty_like(x)
    E.gated_norm(x, y, a, None)
    E.gated_norm(x.as_subclass(Named), y.as_subclass(Named), b.as_subclass(Named), None)
    assert torch.equal(a, b)


@pytest.mark.parametrize("eps", [1e-6, 1e-30, 1e-42])
def test_rows_of_zeros(E, eps):
    """A row that no expert took is zero.  Its norm's gradient is w / sqrt(eps) times what comes in, also
    for an eps whose reciprocal is past fp32 (1e-42).  The root is within 2 units (4 u); three to five
    products round once each."""
    n, d = 5, 192
    x = _make((n, d), torch.float32)
    x[1:4] = 0
    dh, w = _make((n, d), torch.float32), _make((d,), torch.float32)
    r = torch.tensor(eps, device="cuda").double().rsqrt()  # eps as the call takes it
    h, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty_like(w)
    E.gated_norm(x, None, None, h, w_pre=w, eps=eps)
    assert not bool(h[1:4].any()) and bool(h.isfinite().all())
    E.gated_norm_backward(None, dh, x, None, dx, None, w_pre=w, dw_pre=dw, eps=eps)
    ref = dh.double() * w.double() * r
    assert bool(((dx.double() - ref).abs() <= 10 * U32 * ref.abs())[1:4].all())
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())
    gate, dy, dg = _make((n, 1), torch.float32), torch.empty_like(x), torch.empty((n, 1), device="cuda")
    out = torch.ones_like(x)
    E.gated_norm_backward(dh, None, out, x, None, dy, gate=gate, w_post=w, dgate=dg, dw_post=dw, eps=eps)
    ref = dh.double() * w.double() * torch.sigmoid(gate.double()) * r
    assert bool(((dy.double() - ref).abs() <= 20 * U32 * ref.abs())[1:4].all())
    assert bool(dy.isfinite().all()) and not bool(dg[1:4].any()) and bool(dw.isfinite().all())


def test_workspace_out_of_memory(E):
    """A workspace that torch's allocator has no room for is torch's out-of-memory error, and the next
    call works."""
    n, d = 3000, 8192
    x, dh, dx = _make((n, d), torch.float32), _make((n, d), torch.float32), torch.empty((n, d), device="cuda")
    dw = torch.empty(d, device="cuda")
    assert E.gated_norm_backward_workspace(n, d) > 1 << 24
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (1 << 20)) / total)
    filler = []
    try:
        while True:  # what the allocator still holds free, in pieces of less than a workspace
            try:
                filler.append(torch.empty(1 << 22, dtype=torch.uint8, device="cuda"))
            except torch.cuda.OutOfMemoryError:
                break
        with pytest.raises(torch.cuda.OutOfMemoryError):
            E.gated_norm_backward(None, dh, x, None, dx, None, dw_pre=dw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
        filler.clear()
    E.gated_norm_backward(None, dh, x, None, dx, None, dw_pre=dw)
    torch.cuda.synchronize()
    assert bool(dx.isfinite().all()) and bool(dw.isfinite().all())


@pytest.mark.parametrize("d", [96, 479, 1024, 4100])
def test_vectors_written_by_the_call_before(E, d):
    """A vector that the call just ahead writes in place, off any wide boundary, over and over: each call
    sees what the one before it left, as with a wait after every call."""
    n, rounds = 700, 20
    x, y, base = _make((n, d), torch.float32), _make((n, d), torch.float32), _make((3 * d + 7,), torch.float32)

    def run(wait):
        pause = torch.cuda.synchronize if wait else (lambda: None)
        flat = base.clone()
        v = [flat[1 + i * d:1 + (i + 1) * d] for i in range(3)]
        xo, dw, norm = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(1, device="cuda")
        hs, ds = ([torch.empty_like(x) for _ in range(rounds)] for _ in range(2))
        for r in range(rounds):
            E.gated_norm(x, y, xo, hs[r], w_post=v[0], res_scale=v[1], w_pre=v[2])
            pause()
            E.clip_grads(v, 20.0 / (r + 1), norm)
            pause()
            E.gated_norm_backward(x, hs[r], xo, y, ds[r], None, w_post=v[0], res_scale=v[1], w_pre=v[2], dw_pre=dw)
            pause()
            E.clip_grads([v[2], v[0]], 10.0 / (r + 1), norm)
            pause()
        torch.cuda.synchronize()
        return hs + ds + [flat, dw]

    ref = run(True)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(ref, run(False)))


def test_empty_batch_beside_infinite_vectors(E):
    """A sum over no rows is zero whatever factors it would have had."""
    z, v = torch.empty((0, 40), device="cuda"), torch.full((40,), float("inf"), device="cuda")
    dw = [torch.full((40,), 3.0, device="cuda") for _ in range(3)]
    E.gated_norm_backward(z, z, z, z, z, z, w_post=v, res_scale=v * 0, w_pre=v, dw_post=dw[0], dres_scale=dw[1],
                          dw_pre=dw[2])
    assert all(bool((x == 0).all()) for x in dw)
