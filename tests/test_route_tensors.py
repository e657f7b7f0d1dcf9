"""A Route whose positions or weights a caller replaced: the addresses that the
C description holds stay those of living tensors, and a route call puts back
what it writes.  On the CPU nothing is launched: a stand-in takes the library's
place."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_routed_expert_router_amd as coli
from int4_routed_expert_router_amd import binding

NAMES = [n for n, _ in binding._RouteC._fields_]


def _layer(**kw):
    a = dict(hidden=256, inter=128, n_experts=8, n_shared=0, top_k=2, flags=0)
    a.update(kw)
    return coli.Layer(*a.values(), None, None)


class _Library:
    """Route calls that do nothing and return `status`."""

    def __init__(self, status=0):
        self.status, self.seen = status, []

    def coli_moe_route(self, *args):
        self.seen.append([getattr(args[4]._obj, n) for n in NAMES])
        return self.status

    def coli_moe_route_hidden(self, *args):
        self.seen.append([getattr(args[6]._obj, n) for n in NAMES])
        return self.status

    def coli_moe_strerror(self, status):
        return b"refused"


@pytest.mark.parametrize("how", ["attribute", "data"])
@pytest.mark.parametrize("name", NAMES)
def test_replaced_tensors_stay_alive(name, how):
    r = coli.Route(_layer(), 5, device="cpu")
    t = getattr(r, name)
    address = t.data_ptr()
    n, dtype = t.numel(), t.dtype
    if how == "attribute":
        setattr(r, name, torch.empty(n, dtype=dtype))
    else:
        t.data = torch.empty(n, dtype=dtype)
    del t
    assert getattr(r.c, name) == address
    # memory that is still somebody's is not handed out again
    new = [torch.empty(n, dtype=dtype) for _ in range(64)]
    assert all(x.data_ptr() != address for x in new)
    held = [x for v in vars(r).values() for x in (v if isinstance(v, (list, tuple)) else [v])]
    assert any(isinstance(x, torch.Tensor) and x.data_ptr() == address and x.numel() == n
               for x in held)


@pytest.mark.parametrize("hidden", [False, True])
def test_a_route_call_puts_its_own_tensors_back(hidden, monkeypatch):
    L, lib = _layer(), _Library()
    r = coli.Route(L, 5, device="cpu")
    own = {n: getattr(r, n) for n in NAMES}
    addresses = [own[n].data_ptr() for n in NAMES]
    monkeypatch.setattr(binding, "_load", lambda: lib)
    logits = torch.empty(5, 8)

    def call():
        if hidden:
            coli.coli_moe_route_hidden(L, None, None, None, 5, logits, r, stream=0)
        else:
            coli.coli_moe_route(L, logits, None, 5, r, stream=0)

    for _ in range(2):
        for n in ("pair_pos", "topk_w"):
            setattr(r, n, torch.empty_like(own[n]))
        call()
        assert all(getattr(r, n) is own[n] for n in NAMES)
    assert lib.seen == [addresses, addresses]
    # a call that is refused writes nothing, and leaves what the caller put there
    mine = r.pair_pos = torch.empty_like(own["pair_pos"])
    lib.status = -1
    with pytest.raises(coli.ColiError):
        call()
    assert r.pair_pos is mine


def test_quantised_prefill_checks_what_it_passes():
    """The forward calls read the route's own weights, wherever a replacement is."""
    L = _layer()
    r = coli.Route(L, 8, device="cpu")
    with FakeTensorMode():
        q = torch.empty(8, 256, dtype=torch.int8, device="cuda")
        scales = torch.empty(8, 8, dtype=torch.float16, device="cuda")
        y = torch.empty(8, 256, dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        r.topk_w = torch.empty(16, dtype=torch.float32, device="cuda")
    with pytest.raises(ValueError, match="route"):
        coli.coli_moe_forward_prefill_quantized(L, r, q, scales, 8, y, coli.COLI_OUT_BF16, ws)


@pytest.mark.gpu
def test_routing_again_after_a_replacement():
    L = _layer(flags=coli.COLI_ROUTE_RENORM)
    T, g = 40, torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, 8, generator=g, device="cuda")
    fresh, r = coli.Route(L, T), coli.Route(L, T)
    coli.coli_moe_route(L, logits, None, T, fresh)
    r.pair_pos = torch.arange(2 * T, dtype=torch.int32, device="cuda")
    r.topk_w = torch.full((2 * T,), 2.0, device="cuda")
    # tensors of the sizes that the route's own had
    others = [torch.full((2 * T,), 7, dtype=torch.int32, device="cuda") for _ in range(8)]
    others += [torch.full((2 * T,), 7.0, device="cuda") for _ in range(8)]
    x = torch.randn(T, 256, generator=g, device="cuda")
    rows, y = torch.zeros(2 * T, 256, device="cuda"), torch.empty(T, 256, device="cuda")
    coli.coli_moe_dispatch(L, r, x, T, rows)  # the caller's positions
    torch.cuda.synchronize()
    assert torch.equal(rows, x.repeat_interleave(2, dim=0))
    coli.coli_moe_route(L, logits, None, T, r)
    want = torch.zeros_like(rows)
    coli.coli_moe_dispatch(L, fresh, x, T, want)
    coli.coli_moe_dispatch(L, r, x, T, rows)  # the route's again
    torch.cuda.synchronize()
    assert torch.equal(rows, want)
    for n in ("topk_idx", "topk_w", "pairs", "pair_pos", "counts", "offsets"):
        assert torch.equal(getattr(r, n), getattr(fresh, n)), n
    assert all((t == 7).all() for t in others)
    coli.coli_moe_combine(L, r, rows, None, T, y)
    want_y = torch.empty_like(y)
    coli.coli_moe_combine(L, fresh, rows, None, T, want_y)
    torch.cuda.synchronize()
    assert torch.equal(y, want_y)
