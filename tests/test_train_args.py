"""Argument checks of the projection with adapters, the balance loss and the
route's gradient: every call here is refused on the host, before any HIP call,
so no GPU is needed and nothing is written."""
import ctypes

import pytest
import torch

import int4_routed_expert_router_amd as coli
from int4_routed_expert_router_amd import binding

FAKE = 0x100000  # 256-byte aligned, never dereferenced
BIG = 1 << 40
OK, INVALID, WORKSPACE, ALIGN = 0, -1, -3, -4


def layer(**kw):
    a = dict(hidden=2048, inter=512, n_experts=4, n_shared=1, top_k=2, flags=0, q4=FAKE, scales=FAKE)
    a.update(kw)
    return coli.Layer(a["hidden"], a["inter"], a["n_experts"], a["n_shared"], a["top_k"],
                      a["flags"], a["q4"], a["scales"])


def adapters(n=2, r=16, a=FAKE, b=FAKE, rank=FAKE, scale=FAKE):
    return binding._AdaptersC(n, r, a, b, rank, scale)


def requests(n=3, off=FAKE, who=FAKE):
    return binding._RequestsC(n, off, who)


def project(L=None, expert=4, matrix=0, ad=0, rq=0, x=FAKE, T=8, y=FAKE, dt=0, ws=FAKE, nb=BIG):
    L = layer() if L is None else L
    ad = adapters() if ad == 0 else ad
    rq = requests() if rq == 0 else rq
    return binding.raw_library().coli_moe_project(
        ctypes.byref(L.c), expert, matrix, ad and ctypes.byref(ad), rq and ctypes.byref(rq), x, T,
        y, dt, ws, nb, None)


def backward(L=None, expert=4, matrix=0, ad=0, rq=0, x=FAKE, dy=FAKE, T=8, dx=FAKE, da=FAKE,
             db=FAKE, ws=FAKE, nb=BIG):
    L = layer() if L is None else L
    ad = adapters() if ad == 0 else ad
    rq = requests() if rq == 0 else rq
    return binding.raw_library().coli_moe_project_backward(
        ctypes.byref(L.c), expert, matrix, ad and ctypes.byref(ad), rq and ctypes.byref(rq), x,
        dy, T, dx, da, db, ws, nb, None)


@pytest.mark.parametrize("call", [project, backward])
def test_project_refusals(call):
    assert call(L=layer(hidden=100)) == INVALID
    assert call(L=layer(q4=0)) == INVALID
    assert call(L=layer(q4=FAKE + 8)) == ALIGN
    for kw in (dict(expert=-1), dict(expert=5), dict(matrix=-1), dict(matrix=3), dict(x=0),
               dict(T=0), dict(T=-1), dict(T=65537), dict(ad=None), dict(rq=None)):
        assert call(**kw) == INVALID, kw
    assert call(L=layer(n_shared=0), expert=4) == INVALID  # no shared expert in this layer
    for kw in (dict(n=0), dict(n=4097), dict(r=0), dict(r=4), dict(r=20), dict(r=136), dict(a=0),
               dict(b=0)):
        assert call(ad=adapters(**kw)) == INVALID, kw
    for kw in (dict(a=FAKE + 8), dict(b=FAKE + 2), dict(rank=FAKE + 2), dict(scale=FAKE + 1)):
        assert call(ad=adapters(**kw)) == ALIGN, kw
    for kw in (dict(n=0), dict(n=-3), dict(n=65537), dict(off=0), dict(who=0)):
        assert call(rq=requests(**kw)) == INVALID, kw
    for kw in (dict(off=FAKE + 2), dict(who=FAKE + 1)):
        assert call(rq=requests(**kw)) == ALIGN, kw
    assert call(x=FAKE + 8) == ALIGN
    need = binding.raw_library().coli_moe_project_workspace_bytes(
        ctypes.byref(layer().c), 0, ctypes.byref(adapters()), 8, int(call is backward))
    assert need > 0
    assert call(nb=need - 1) == WORKSPACE
    assert call(ws=0, nb=need) == INVALID
    assert call(ws=FAKE + 16, nb=need) == ALIGN


def test_project_outputs_refused():
    assert project(y=0) == INVALID
    assert project(dt=2) == INVALID
    assert project(y=FAKE + 8) == ALIGN
    assert backward(dy=0) == INVALID
    assert backward(da=0) == INVALID  # one gradient without the other
    assert backward(db=0) == INVALID
    assert backward(dx=0, da=0, db=0) == INVALID  # nothing wanted
    assert backward(ad=None, rq=None) == INVALID  # gradients of no adapters
    for n in ("dy", "dx", "da", "db"):
        assert backward(**{n: FAKE + 8}) == ALIGN, n


def test_project_workspace_sizes():
    ws = binding.raw_library().coli_moe_project_workspace_bytes
    L, a = ctypes.byref(layer().c), ctypes.byref(adapters())
    assert ws(L, 0, a, 8, 0) > ws(L, 0, None, 8, 0) > 0
    assert ws(L, 0, a, 8, 1) > ws(L, 0, a, 8, 0)
    assert ws(L, 3, a, 8, 0) == 0 and ws(L, 0, a, 0, 0) == 0 and ws(L, 0, a, 65537, 0) == 0
    assert ws(L, 0, ctypes.byref(adapters(r=12)), 8, 0) == 0
    assert ws(ctypes.byref(layer(hidden=100).c), 0, a, 8, 0) == 0
    # sizes past 32 bits are counted in 64
    huge = layer(hidden=16384, inter=16384)
    assert ws(ctypes.byref(huge.c), 0, ctypes.byref(adapters(n=4096, r=128)), 65536, 1) > 1 << 35


def balance(n=1, off=FAKE, valid=0, counts=FAKE, mean=FAKE, tokens=FAKE, totals=FAKE, loss=FAKE):
    return binding._BalanceC(n, off, valid, counts, mean, tokens, totals, loss)


def loss(L=None, logits=FAKE, idx=FAKE, T=8, b=0, ws=FAKE, nb=BIG):
    L = layer() if L is None else L
    b = balance() if b == 0 else b
    return binding.raw_library().coli_moe_balance_loss(
        ctypes.byref(L.c), logits, idx, T, b and ctypes.byref(b), ws, nb, None)


def gradient(L=None, logits=FAKE, idx=FAKE, T=8, dw=FAKE, b=0, dl=FAKE, out=FAKE):
    L = layer() if L is None else L
    b = balance() if b == 0 else b
    return binding.raw_library().coli_moe_route_backward(
        ctypes.byref(L.c), logits, idx, T, dw, b and ctypes.byref(b), dl, out, None)


@pytest.mark.parametrize("call", [loss, gradient])
def test_balance_refusals(call):
    assert call(L=layer(top_k=0)) == INVALID
    for kw in (dict(logits=0), dict(idx=0), dict(T=0), dict(T=65537)):
        assert call(**kw) == INVALID, kw
    assert call(L=layer(n_experts=64, top_k=32), T=40000) == INVALID  # T*k > 2^20
    for kw in (dict(n=0), dict(n=65537), dict(n=2, off=0), dict(counts=0), dict(tokens=0),
               dict(totals=0)):
        assert call(b=balance(**kw)) == INVALID, kw
    for n in ("off", "counts", "tokens", "totals", "mean", "loss"):
        assert call(b=balance(**{n: FAKE + 2})) == ALIGN, n
    assert call(logits=FAKE + 1) == ALIGN
    assert call(idx=FAKE + 2) == ALIGN


def test_balance_own_refusals():
    assert loss(b=None) == INVALID
    assert loss(b=balance(mean=0)) == INVALID
    assert loss(b=balance(loss=0)) == INVALID
    need = coli.coli_moe_balance_workspace_bytes(layer(), 8, 1)
    assert need > 0 and coli.coli_moe_balance_workspace_bytes(layer(), 8, 0) == 0
    assert coli.coli_moe_balance_workspace_bytes(layer(), 0, 1) == 0
    assert loss(nb=need - 1) == WORKSPACE
    assert loss(ws=FAKE + 8, nb=need) == ALIGN
    assert gradient(out=0) == INVALID
    assert gradient(b=None) == INVALID       # d_loss without a balance
    assert gradient(dl=0) == INVALID         # a balance without d_loss
    assert gradient(dw=0, b=None, dl=0) == INVALID  # nothing to differentiate
    assert gradient(out=FAKE + 2) == ALIGN
    assert gradient(dw=FAKE + 1) == ALIGN
    assert gradient(dl=FAKE + 3) == ALIGN


def test_binding_refuses_tensors_that_do_not_fit():
    """Types, sizes, strides and devices are checked before the library is called."""
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    a, b = torch.zeros(2, 8, 2048, dtype=bf), torch.zeros(2, 512, 8, dtype=bf)
    with pytest.raises(ValueError):
        coli.Adapters(a.float(), b)
    with pytest.raises(ValueError):
        coli.Adapters(a, b[:1])
    with pytest.raises(ValueError):
        coli.Adapters(a[:, :, ::2], b)
    with pytest.raises(ValueError):
        coli.Adapters(a, b, rank=torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError):
        coli.Adapters(a, b, scale=torch.zeros(2, dtype=torch.float64))
    with pytest.raises(ValueError):
        coli.Requests(torch.zeros(2, dtype=i32), torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError):
        coli.Requests(torch.zeros(3, dtype=torch.int64), torch.zeros(2, dtype=i32))
    L, ad = layer(), coli.Adapters(a, b)
    rq = coli.Requests(torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32))
    x, y, ws = torch.zeros(8, 2048, dtype=bf), torch.zeros(8, 512, dtype=bf), torch.zeros(64)
    go = lambda x=x, y=y, m=0, T=8: coli.coli_moe_project(L, 4, m, ad, rq, x, T, y, 0, ws)  # noqa: E731
    for kw in (dict(), dict(x=x.float()), dict(x=x[:4]), dict(x=x.t()), dict(y=y.float()),
               dict(y=y[:, ::2]), dict(m=2), dict(T=9)):
        with pytest.raises(ValueError):  # the first: everything fits, but on the CPU
            go(**kw)
    with pytest.raises(ValueError):
        coli.Balance(L, 3, torch.zeros(3, dtype=i32), device="cpu")
    lg, idx = torch.zeros(8, 4), torch.zeros(8, 2, dtype=i32)
    bal = coli.Balance(L, 1, None, torch.ones(4, dtype=torch.uint8), device="cpu")
    with pytest.raises(ValueError):  # a mask of four rows for eight
        coli.coli_moe_balance_loss(L, lg, idx, 8, bal, ws)
    with pytest.raises(ValueError):
        coli.coli_moe_balance_loss(L, lg, idx.long(), 8, coli.Balance(L, device="cpu"), ws)
    with pytest.raises(ValueError):
        coli.coli_moe_route_backward(L, lg, idx, 8, torch.zeros(8, 1), None, None, lg)


def test_workspace_of_a_batch_does_for_smaller_ones():
    """The paths of short, middle and long batches need different buffers."""
    lib = binding.raw_library()
    ws = lib.coli_moe_project_workspace_bytes
    for hidden, inter in ((6144, 2048), (256, 128), (64, 16384)):
        L, a = layer(hidden=hidden, inter=inter), adapters()
        for matrix in (0, 2):
            for back in (0, 1):
                last = 0
                for T in (1, 16, 17, 32, 33, 100, 128, 129, 512, 513, 1000, 1536, 4000, 24576, 24577,
                          65536):
                    n = ws(ctypes.byref(L.c), matrix, ctypes.byref(a), T, back)
                    assert n >= last > -1, (hidden, matrix, back, T)
                    last = n
