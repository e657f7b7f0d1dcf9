"""A Norm whose weight a caller replaced: the calls take the weight as it is
now, of its own type, and check its size.  Without a GPU: a stand-in takes the
library's place, and the inputs are shapes without memory."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_routed_expert_router_amd as coli
from int4_routed_expert_router_amd import binding

H, T = 64, 4
BF, F32 = torch.bfloat16, torch.float32


def _calls(monkeypatch):
    """Both calls of the norm `n`, each returning (weight's address, its type)."""
    seen = []
    monkeypatch.setattr(binding, "_run", lambda name, on, stream, c, *args: seen.append(
        (c._obj.weight, c._obj.weight_dtype)))

    class X:  # a tensor on no device, as the weights of this test are
        dtype, device = BF, "cpu"
        get_device = staticmethod(lambda: -1)
        numel = staticmethod(lambda: T * H)
        is_contiguous = staticmethod(lambda: True)
        data_ptr = staticmethod(lambda: 0x100000)

    def run(n):
        seen.clear()
        coli.coli_moe_norm(n, X, None, None, T, X)
        coli.coli_moe_norm_backward(n, X, T, X, None, X, None, None)
        assert len(seen) == 2 and seen[0] == seen[1]
        return seen[0]

    return run


def test_the_weight_as_it_is_now(monkeypatch):
    run = _calls(monkeypatch)
    n = coli.Norm(H, torch.ones(H, dtype=BF))
    assert run(n) == (n.weight.data_ptr(), coli.COLI_SRC_BF16)
    n.weight = torch.ones(H)
    assert run(n) == (n.weight.data_ptr(), coli.COLI_SRC_F32)
    n.weight.data = torch.ones(H)
    assert run(n) == (n.weight.data_ptr(), coli.COLI_SRC_F32)
    n.weight = None
    assert run(n)[0] is None
    n.weight = torch.ones(H, dtype=BF)
    assert run(n) == (n.weight.data_ptr(), coli.COLI_SRC_BF16)


def test_a_replacement_is_checked(monkeypatch):
    run = _calls(monkeypatch)
    n = coli.Norm(H, torch.ones(H, dtype=BF))
    with FakeTensorMode():
        elsewhere = torch.ones(H, dtype=BF, device="cuda")
    for w in (torch.ones(H - 1), torch.ones(2 * H)[::2], torch.ones(H, dtype=torch.float16), elsewhere):
        n.weight = w
        with pytest.raises(ValueError):
            run(n)


def test_the_width_is_that_of_the_description():
    n = coli.Norm(H)
    with pytest.raises(AttributeError):  # the kernels would go on with the first one
        n.hidden = H // 2
    assert n.hidden == n.c.hidden == H


@pytest.mark.gpu
def test_replaced_weights_on_the_gpu():
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(9, 2048, generator=g, device="cuda").to(BF)
    w = [torch.rand(2048, generator=g, device="cuda").to(dt) for dt in (BF, F32)]
    n = coli.Norm(2048, w[0].clone())
    y, want = torch.empty_like(x), torch.empty_like(x)
    for weight in (w[0], w[1], None, w[0]):
        n.weight = None if weight is None else weight.clone()
        other = torch.full((2048,), 9.0, dtype=BF, device="cuda")  # where the last one may have been
        coli.coli_moe_norm(n, x, None, None, 9, y)
        coli.coli_moe_norm(coli.Norm(2048, weight), x, None, None, 9, want)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and (other == 9).all()
