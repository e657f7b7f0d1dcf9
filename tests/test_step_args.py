"""Argument checks of the norm, the calls on rows by expert and the clipping:
every call here is refused on the host, before any HIP call, so no GPU is
needed and nothing is written.  The plan of a clipping is made on the host and
checked whole."""
import ctypes
import random

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_routed_expert_router_amd as coli
from int4_routed_expert_router_amd import binding

FAKE = 0x100000  # 256-byte aligned, never dereferenced
BIG = 1 << 40
INVALID, UNSUPPORTED, WORKSPACE, ALIGN = -1, -2, -3, -4
INF, NAN = float("inf"), float("nan")


def _lib():
    return binding.raw_library()


def norm_c(hidden=2048, eps=1e-6, weight=FAKE, dtype=0):
    return binding._NormC(hidden, eps, weight, dtype)


def norm(n=None, x=FAKE, residual=FAKE, rd=0, T=8, total=FAKE, y=FAKE, fmt=0, q=None, scales=None):
    n = norm_c() if n is None else n
    return _lib().coli_moe_norm((ctypes.byref(n) if n else None), x, residual, rd, T, total, y, fmt, q,
                                scales, None)


def norm_backward(n=None, total=FAKE, td=0, dy=FAKE, d_total=FAKE, T=8, dx=FAKE, dr=FAKE, dw=FAKE,
                  ws=FAKE, nb=BIG):
    n = norm_c() if n is None else n
    return _lib().coli_moe_norm_backward((ctypes.byref(n) if n else None), total, td, dy, d_total, T, dx, dr,
                                         dw, ws, nb, None)


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_sizes(call):
    assert call(n=False) == INVALID
    for h in (0, -8, 4, 12, 16392, 32768):
        assert call(n=norm_c(hidden=h)) == INVALID
    for eps in (0.0, -1e-6, INF, NAN):
        assert call(n=norm_c(eps=eps)) == INVALID
    assert call(n=norm_c(dtype=2)) == INVALID
    assert call(n=norm_c(weight=FAKE + 8)) == ALIGN
    for T in (0, -1, (1 << 24) + 1):
        assert call(T=T) == INVALID


def test_norm_refusals():
    assert norm(x=None) == INVALID
    assert norm(residual=None) == INVALID
    assert norm(total=None) == INVALID
    assert norm(rd=2) == INVALID
    assert norm(fmt=3, q=FAKE, scales=FAKE) == INVALID
    assert norm(fmt=-1, q=FAKE, scales=FAKE) == INVALID
    assert norm(y=None) == INVALID
    assert norm(q=FAKE, scales=FAKE) == INVALID  # codes without a format
    for fmt in (1, 2):
        assert norm(fmt=fmt) == INVALID
        assert norm(fmt=fmt, q=FAKE) == INVALID
        assert norm(fmt=fmt, scales=FAKE) == INVALID
        assert norm(n=norm_c(hidden=2056), fmt=fmt, q=FAKE, scales=FAKE) == UNSUPPORTED
        assert norm(fmt=fmt, q=FAKE + 8, scales=FAKE) == ALIGN
        assert norm(fmt=fmt, q=FAKE, scales=FAKE + 2) == ALIGN
    for name in ("x", "residual", "total", "y"):
        assert norm(**{name: FAKE + 8}) == ALIGN


def test_norm_backward_refusals():
    assert norm_backward(total=None) == INVALID
    assert norm_backward(dy=None) == INVALID
    assert norm_backward(td=2) == INVALID
    assert norm_backward(dx=None, dr=None, dw=None) == INVALID
    assert norm_backward(ws=None) == INVALID
    assert norm_backward(ws=FAKE + 128) == ALIGN
    n = norm_c()
    need = _lib().coli_moe_norm_workspace_bytes(ctypes.byref(n), 8)
    assert need >= 2048 * 4
    assert norm_backward(nb=need - 1) == WORKSPACE
    for name in ("total", "dy", "d_total", "dx", "dr", "dw"):
        assert norm_backward(**{name: FAKE + 8}) == ALIGN
    # outputs over inputs of another type
    far = [FAKE + (i << 20) for i in range(1, 5)]
    assert norm_backward(td=1, dy=far[0], d_total=far[1], dx=far[1], dr=far[2]) == INVALID
    assert norm_backward(td=1, dy=far[0], d_total=far[1], dx=far[2], dr=far[2]) == INVALID
    assert norm_backward(td=1, dy=far[0], d_total=far[1], dx=far[2], dr=far[0]) == INVALID


def test_norm_workspace():
    w = _lib().coli_moe_norm_workspace_bytes
    sizes = [w(ctypes.byref(norm_c()), T) for T in (1, 2, 100, 5000, 1 << 24)]
    assert all(s > 0 and s % 256 == 0 for s in sizes) and sizes == sorted(sizes)
    assert w(None, 8) == 0 and w(ctypes.byref(norm_c()), 0) == 0
    assert w(ctypes.byref(norm_c(hidden=7)), 8) == 0


def layer(**kw):
    a = dict(hidden=2048, inter=512, n_experts=4, n_shared=1, top_k=2, flags=0)
    a.update(kw)
    return coli.Layer(a["hidden"], a["inter"], a["n_experts"], a["n_shared"], a["top_k"],
                      a["flags"], None, None)


def route(**kw):
    a = {n: FAKE for n, _ in binding._RouteC._fields_}
    a.update(kw)
    return binding._RouteC(*[a[n] for n, _ in binding._RouteC._fields_])


def dispatch(L=None, r=None, one=FAKE, dtype=0, T=8, other=FAKE, n_rows=16, **kw):
    L, r = layer() if L is None else L, route() if r is None else r
    return _lib().coli_moe_dispatch((ctypes.byref(L.c) if L else None),
        (ctypes.byref(r) if r else None), one, dtype, T,
                                    other, n_rows, None)


def _from_rows(name):
    def call(L=None, r=None, one=FAKE, dtype=0, T=8, other=FAKE, n_rows=16, other_dtype=0,
             beside=FAKE):
        L, r = layer() if L is None else L, route() if r is None else r
        return getattr(_lib(), name)((ctypes.byref(L.c) if L else None),
        (ctypes.byref(r) if r else None), one, dtype,
                                     n_rows, beside, T, other, other_dtype, None)
    call.__name__ = name
    return call


dispatch_backward = _from_rows("coli_moe_dispatch_backward")
combine = _from_rows("coli_moe_combine")


def combine_backward(L=None, r=None, one=FAKE, dtype=0, T=8, other=FAKE, n_rows=16, other_dtype=0,
                     d_rows=FAKE, d_w=FAKE):
    L, r = layer() if L is None else L, route() if r is None else r
    return _lib().coli_moe_combine_backward((ctypes.byref(L.c) if L else None),
        (ctypes.byref(r) if r else None), one,
                                            dtype, n_rows, other, other_dtype, T, d_rows, d_w,
                                            None)


@pytest.mark.parametrize("call", [dispatch, dispatch_backward, combine, combine_backward])
def test_rows_refusals(call):
    assert call(L=False) == INVALID
    assert call(L=layer(hidden=100)) == INVALID
    assert call(r=False) == INVALID
    assert call(r=route(pair_pos=None)) == INVALID
    assert call(r=route(pair_pos=FAKE + 2)) == ALIGN
    assert call(one=None) == INVALID
    assert call(other=None) == INVALID
    assert call(one=FAKE + 8) == ALIGN
    assert call(other=FAKE + 8) == ALIGN
    assert call(dtype=2) == INVALID
    for T in (0, -1, 65537):
        assert call(T=T) == INVALID
    assert call(L=layer(n_experts=64, top_k=32), T=32769) == INVALID  # T*k over 2^20
    for n in (0, -1, (1 << 21) + 1):
        assert call(n_rows=n) == INVALID
    if call is not dispatch:
        assert call(other_dtype=-1) == INVALID
    if call in (combine, combine_backward):
        assert call(r=route(topk_w=None)) == INVALID
        assert call(r=route(topk_w=FAKE + 1)) == ALIGN
    if call in (combine, dispatch_backward):
        assert call(beside=FAKE + 4) == ALIGN
        # onto beside, of another type
        assert call(dtype=1, other_dtype=0, beside=FAKE, other=FAKE) == INVALID
        assert call(dtype=0, other_dtype=1, beside=FAKE, other=FAKE) == INVALID


def test_combine_backward_outputs():
    assert combine_backward(d_rows=None, d_w=None) == INVALID
    assert combine_backward(one=None, d_w=FAKE) == INVALID
    assert combine_backward(d_rows=FAKE + 8) == ALIGN
    assert combine_backward(d_w=FAKE + 2) == ALIGN


def test_prefill_quantized_refusals():
    f = _lib().coli_moe_forward_prefill_quantized
    L = coli.Layer(2048, 512, 4, 1, 2, 0, FAKE, FAKE)
    r = route()
    a = [ctypes.byref(L.c), ctypes.byref(r), FAKE, FAKE, 8, FAKE, 0, FAKE, BIG, None]
    for at, bad, rc in ((0, None, INVALID), (1, None, INVALID), (2, None, INVALID),
                        (3, None, INVALID), (2, FAKE + 8, ALIGN), (3, FAKE + 8, ALIGN),
                        (4, 0, INVALID), (4, 65537, INVALID), (5, None, INVALID),
                        (5, FAKE + 8, ALIGN), (6, 2, INVALID), (7, None, INVALID),
                        (8, 1, WORKSPACE)):
        b = list(a)
        b[at] = bad
        assert f(*b) == rc, (at, bad)
    mx = coli.Layer(2048, 64, 4, 1, 2, coli.COLI_ACT_MXFP8, FAKE, FAKE, mxfp4=True)
    assert f(ctypes.byref(mx.c), *a[1:]) == UNSUPPORTED


# ---------------------------------------------------------------- clipping

def grads(*g):
    return (binding._GradientC * max(1, len(g)))(*[binding._GradientC(*x) for x in g])


def plan(*g):
    """The plan's items, or its error."""
    c = grads(*g)
    n = _lib().coli_moe_clip_items(c, len(g))
    if n < 0:
        return n
    items = (binding._ClipItemC * max(1, n))()
    rc = _lib().coli_moe_clip_plan(c, len(g), items, n)
    return rc if rc else list(items)[:n]


def test_plan_refusals():
    f = _lib().coli_moe_clip_items
    assert f(None, 1) == INVALID and f(grads(), -1) == INVALID
    assert f(grads((FAKE, FAKE, 4, 1, 1)), (1 << 20) + 1) == INVALID
    assert plan((FAKE, FAKE, 1 << 35, 0, 0), (BIG, BIG, (1 << 35) + 1, 0, 0)) == INVALID
    for g, rc in (((FAKE, FAKE, -1, 1, 1), INVALID), ((FAKE, FAKE, (1 << 36) + 1, 1, 1), INVALID),
                  ((None, FAKE, 4, 1, 1), INVALID), ((FAKE, None, 4, 1, 1), INVALID),
                  ((FAKE, FAKE, 4, 2, 2), INVALID), ((FAKE, FAKE, 4, 1, 0), INVALID),
                  ((FAKE + 2, FAKE, 4, 1, 1), ALIGN), ((FAKE, FAKE + 1, 4, 1, 0), ALIGN)):
        assert plan(g) == rc, g
    # wrong number of items, or nowhere to put them
    c = grads((FAKE, FAKE, 4, 1, 1))
    items = (binding._ClipItemC * 2)()
    assert _lib().coli_moe_clip_plan(c, 1, items, 2) == INVALID
    assert _lib().coli_moe_clip_plan(c, 1, None, 1) == INVALID


def test_plan_overlaps():
    far = FAKE + (1 << 30)
    assert len(plan((FAKE, FAKE, 4, 1, 1), (FAKE + 16, FAKE + 16, 4, 1, 1))) == 2
    # the same tensor twice in place; two outputs over each other
    assert plan((FAKE, FAKE, 4, 1, 1), (FAKE, FAKE, 4, 1, 1)) == INVALID
    assert plan((FAKE, far, 100, 1, 1), (FAKE + 4096, far + 396, 100, 1, 1)) == INVALID
    # an output over its own gradient, shifted, and over another's
    assert plan((FAKE, FAKE + 16, 100, 1, 1)) == INVALID
    assert plan((FAKE, far, 100, 1, 1), (FAKE + 4096, FAKE + 396, 100, 1, 1)) == INVALID
    assert plan((FAKE, far, 1 << 20, 1, 1), (FAKE + (1 << 22), FAKE + 40000, 8, 1, 1)) == INVALID
    # the same gradient read twice is in order, and so are neighbours
    assert len(plan((FAKE, far, 100, 1, 1), (FAKE, far + 400, 100, 1, 0))) == 2


@pytest.mark.parametrize("seed", range(6))
def test_plan_covers_everything_once(seed):
    rng = random.Random(seed)
    g, at = [], FAKE
    for _ in range(rng.choice((1, 3, 40))):
        n = rng.choice((0, 1, 7, 2047, 2048, 2049, 70001, rng.randrange(1, 1 << 21)))
        gd, od = rng.randrange(2), rng.randrange(2)
        here = at + (4 if gd else 2) * rng.randrange(9)
        at = (here + 4 * n + 255) // 256 * 256
        there = here
        if gd != od or rng.random() < 0.5:
            there = at + (4 if od else 2) * rng.randrange(9)
            at = (there + 4 * n + 255) // 256 * 256
        g.append((here, there, n, gd, od))
    items = plan(*g)
    assert [i.order for i in items] == list(range(len(items)))
    k = 0
    for here, there, n, gd, od in g:
        done = 0
        while done < n:
            it = items[k]
            assert it.grad == here + done * (4 if gd else 2)
            assert it.out == there + done * (4 if od else 2)
            assert it.dtypes == gd + 2 * od and 1 <= it.n <= 32768 + 7
            assert done == 0 or it.grad % 16 == 0  # only a gradient's first item has a ragged start
            done += it.n
            k += 1
        assert done == n
    assert k == len(items)


def test_clip_refusals():
    f = _lib().coli_moe_clip_gradients
    need = _lib().coli_moe_clip_workspace_bytes()
    assert f(None, 1, 1.0, FAKE, FAKE, BIG, None) == INVALID
    assert f(FAKE, -1, 1.0, FAKE, FAKE, BIG, None) == INVALID
    assert f(FAKE, 1 << 24, 1.0, FAKE, FAKE, BIG, None) == INVALID
    for m in (-1.0, NAN, -INF):
        assert f(FAKE, 1, m, FAKE, FAKE, BIG, None) == INVALID
    assert f(FAKE, 1, 1.0, None, FAKE, BIG, None) == INVALID
    assert f(FAKE, 1, 1.0, FAKE, None, BIG, None) == INVALID
    assert f(FAKE + 4, 1, 1.0, FAKE, FAKE, BIG, None) == ALIGN
    assert f(FAKE, 1, 1.0, FAKE + 2, FAKE, BIG, None) == ALIGN
    assert f(FAKE, 1, 1.0, FAKE, FAKE + 8, BIG, None) == ALIGN
    assert f(FAKE, 1, 1.0, FAKE, FAKE, need - 1, None) == WORKSPACE


# ---------------------------------------------------------------- binding

def test_binding_refuses_wrong_tensors():
    """Types, sizes, strides and devices, before the library is called.  The
    inputs are shapes without memory that say they are on a GPU."""
    bf, f32, T, H = torch.bfloat16, torch.float32, 8, 128
    with FakeTensorMode():
        new = lambda *s, dt=bf: torch.empty(*s, dtype=dt, device="cuda")  # noqa: E731
        x, res, short, wide, ints = new(T, H), new(T, H, dt=f32), new(T, 64), new(T, 2 * H), new(
            T, H, dt=torch.int32)
        rows, dw = new(2 * T, H), new(2 * T, dt=f32)
        q, sc, w = new(T, H, dt=torch.int8), new(T, 4, dt=torch.float16), new(H)
        ws = new(1 << 20, dt=torch.uint8)
    cpu = torch.empty(T, H, dtype=bf)
    n = coli.Norm(H)
    bad = (short, wide[:, ::2], ints, cpu)
    for t in bad:
        with pytest.raises(ValueError):
            coli.coli_moe_norm(n, x, None, None, T, t)
        with pytest.raises(ValueError):
            coli.coli_moe_norm(n, x, res, t, T, x)
        with pytest.raises(ValueError):
            coli.coli_moe_norm_backward(n, x, T, t, None, x, None, None)
    with pytest.raises(ValueError):
        coli.coli_moe_norm(n, cpu, None, None, T, cpu)  # not on a GPU
    with pytest.raises(ValueError):
        coli.coli_moe_norm(n, x, None, None, T, x, coli.COLI_NORM_Q8_0, x, sc)
    with pytest.raises(ValueError):
        coli.coli_moe_norm(n, x, None, None, T, x, coli.COLI_NORM_MXFP8, q, sc)
    with pytest.raises(ValueError):
        coli.Norm(H, torch.empty(H, dtype=torch.float16))
    with pytest.raises(ValueError):
        coli.Norm(H, torch.empty(H - 8, dtype=bf))
    n.weight = torch.empty(H, dtype=bf)  # on the host
    with pytest.raises(ValueError, match="weight on"):
        coli.coli_moe_norm(n, x, None, None, T, x)
    L = layer(hidden=H)
    r = coli.Route(L, T, device="cpu")
    with pytest.raises(ValueError, match="route"):
        coli.coli_moe_dispatch(L, r, x, T, rows)
    with pytest.raises(ValueError, match="route"):
        coli.coli_moe_forward_prefill_quantized(L, r, q, sc, T, x, coli.COLI_OUT_BF16, ws)
    with FakeTensorMode():
        r.pair_pos = torch.empty(2 * T, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="x: expected"):
        coli.coli_moe_dispatch(L, r, res, T, rows)
    for t in bad:
        with pytest.raises(ValueError):
            coli.coli_moe_dispatch(L, r, t, T, rows)
        with pytest.raises(ValueError):
            coli.coli_moe_combine(L, r, rows, t, T, x)
        with pytest.raises(ValueError):
            coli.coli_moe_dispatch_backward(L, r, rows, None, T, t)
        with pytest.raises(ValueError):
            coli.coli_moe_combine_backward(L, r, rows, t, T, rows, dw)
    with pytest.raises(ValueError):
        coli.coli_moe_combine_backward(L, r, rows, x, T, x, dw)  # d_rows of fewer rows
    with pytest.raises(ValueError):
        coli.coli_moe_combine_backward(L, r, rows, x, T, rows, dw[:-1])
    del w


def test_gradients_refuse_wrong_tensors():
    f = torch.float32
    with pytest.raises(ValueError):
        coli.Gradients([])
    with pytest.raises(ValueError):
        coli.Gradients([torch.empty(4), torch.empty(4)], [torch.empty(4)])
    with pytest.raises(ValueError):
        coli.Gradients([torch.empty(4, dtype=torch.float16)])
    with pytest.raises(ValueError):
        coli.Gradients([torch.empty(8, 8)[:, ::2]])
    with pytest.raises(ValueError):
        coli.Gradients([torch.empty(4)], [torch.empty(5)])
    t = torch.empty(64, dtype=f)
    with pytest.raises(coli.ColiError):
        coli.Gradients([t, t])
    with pytest.raises(coli.ColiError):
        coli.Gradients([t[:32], t[16:48]])
    g = coli.Gradients([t[:32], t[32:], torch.empty(0)])
    assert g.n == 2
    with pytest.raises(ValueError):  # on the host
        coli.coli_moe_clip_gradients(g, 1.0, torch.empty(2), coli.clip_workspace("cpu"))
