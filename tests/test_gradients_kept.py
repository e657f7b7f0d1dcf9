"""The memory that a clipping plan writes stays the plan's, whatever becomes of
the tensors it was made from.  Plans are made on the host: no GPU is needed."""
import ctypes

import torch

import int4_routed_expert_router_amd as coli
from int4_routed_expert_router_amd import binding


def _items(g):
    n = g.items.numel() // ctypes.sizeof(binding._ClipItemC)
    return list((binding._ClipItemC * n).from_address(g.items.data_ptr()))[:g.n]


def _new(n):
    return torch.zeros(n)


def test_moved_and_dropped_gradients():
    grads, out = [_new(100), _new(300)], [_new(100), _new(300)]
    g = coli.Gradients(grads, out)
    items = _items(g)
    addresses = [t.data_ptr() for t in grads + out]
    assert [i.grad for i in items] + [i.out for i in items] == addresses
    for t in grads + out:
        t.data = _new(t.numel())  # the memory itself
    for holder in (grads, out, g.grads, g.out):  # the tensors
        try:
            holder.clear()
        except AttributeError:  # a tuple
            pass
    g.grads = g.out = None
    del grads, out, t
    new = [_new(n) for _ in range(64) for n in (100, 300)]
    assert not set(addresses) & {x.data_ptr() for x in new}
    assert [i.grad for i in items] + [i.out for i in items] == addresses


def test_in_place():
    t = _new(500)
    g = coli.Gradients([t])
    at = t.data_ptr()
    t.data = _new(500)
    g.grads = g.out = None
    del t
    assert at not in {x.data_ptr() for x in [_new(500) for _ in range(64)]}
    assert [(i.grad, i.out) for i in _items(g)] == [(at, at)]
