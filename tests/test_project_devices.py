"""A projection refuses a layer whose weights are not where its inputs are,
before the library is called.  The inputs are shapes without memory that say
they are on a GPU, so the test needs none."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import int4_routed_expert_router_amd as coli

H, I, T = 128, 64, 8


@pytest.mark.parametrize("where", ["both", "codes", "scales"])
def test_weights_on_another_device(where):
    def weights(device="cpu"):
        return (torch.empty(3 * 3 * H * I // 2, dtype=torch.uint8, device=device),
                torch.empty(3 * 3 * H * I // 64, dtype=torch.float16, device=device))

    bf = torch.bfloat16
    with FakeTensorMode():
        x, dx = (torch.empty(T, H, dtype=bf, device="cuda") for _ in range(2))
        y = torch.empty(T, I, dtype=bf, device="cuda")
        ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
        there = weights("cuda")
    here = weights()
    q4, scales = {"both": here, "codes": (here[0], there[1]), "scales": (there[0], here[1])}[where]
    L = coli.Layer(H, I, 2, 1, 1, 0, 0x100000, 0x100000)
    L.q4, L.scales = q4, scales
    with pytest.raises(ValueError, match="weights on"):
        coli.coli_moe_project(L, 2, 0, None, None, x, T, y, coli.COLI_OUT_BF16, ws)
    with pytest.raises(ValueError, match="weights on"):
        coli.coli_moe_project_backward(L, 2, 0, None, None, x, y, T, dx, None, None, ws)
