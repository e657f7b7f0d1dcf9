"""Precision of the projection with adapters where a linear bound on all
products cannot see it: large inputs that meet zero codes, and inputs whose
sums are exact in fp32, so that every bit of u, v and the weights counts."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import train_util as tu
from test_gpu_project import E24, Case, _spec

pytestmark = pytest.mark.gpu

# rows, hidden, inter of matrix 0: the codes streamed (three tiles), x
# staged in LDS, and the tiled product
PATHS = [(5, 64, 128), (20, 64, 128), (40, 4160, 128), (90, 64, 128), (300, 256, 128), (1100, 64, 4096)]


def _zero_codes(c, cols):
    """Clears the codes of these columns of the case's matrix, int4 or int8 or
    MXFP4, on the device and in its dense form."""
    N, K = c.N, c.K
    per = c.q4.numel() // ((c.spec.n_experts + 1) * 3)
    q = c.q4.view(-1, per)[3 * c.expert + c.matrix].view(N, -1)
    if q.shape[1] == K:
        q[:, cols] = 0
    else:
        for k in cols:
            q[:, k // 2] &= 0x0f if k % 2 else 0xf0
    c.w[:, cols] = 0


@pytest.mark.parametrize("fmt", ["int4", "int8", "mxfp4"])
@pytest.mark.parametrize("T,H,I", PATHS)
def test_large_inputs_at_zero_codes(fmt, T, H, I):
    """A column of W that is zero adds nothing, whatever x holds there: the
    error stays within the bound of the other columns' products."""
    print("zero codes", fmt, T, H, I, flush=True)
    c = Case(_spec(fmt, H, I), 0, T, None, None, None, seed=T)
    cols = [1, 6, 19, 40, 63] + list(range(70, H, 97))
    _zero_codes(c, cols)
    g = torch.Generator().manual_seed(T)
    big = torch.randn(T, len(cols), generator=g) * 2.0 ** 14
    c.x[:, cols] = big.to(torch.bfloat16)
    y, S = tu.project(c.w, None, c.own, tu.host(c.x))
    tol = (2 * c.K + 8) * E24 * S
    got = tu.host(c.forward(True))
    bad = ~(np.abs(got - y) <= tol)
    assert not bad.any(), (bad.mean(), np.max(np.abs(got - y) / tol))
    got = tu.host(c.forward(False))
    bad = ~(np.abs(got - y) <= tol + tu.HALF[torch.bfloat16] * (np.abs(y) + tol))
    assert not bad.any(), bad.mean()
