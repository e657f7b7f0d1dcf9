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


def _in_parts(v, p):
    """v (float64) as p bf16 parts, each the rounding of what the earlier ones leave."""
    out, rest = 0.0, torch.tensor(v, dtype=torch.float64)
    for _ in range(p):
        part = rest.to(torch.bfloat16).double()
        out, rest = out + part.item(), rest - part
    return out


# 24 bits apart: the sum needs every bit of fp32, any order of adding it is exact
TERMS = np.array([1.0, 2.0 ** -8, 2.0 ** -16, 2.0 ** -23])


def test_the_terms_tell_parts_apart():
    v = TERMS.sum()
    assert np.float32(v) == v
    assert _in_parts(v, 3) == v and _in_parts(v, 2) != v and _in_parts(v, 1) != v


@pytest.mark.parametrize("fmt,code", [("int4", 0x07), ("int8", 0x7f), ("mxfp4", 0x07)])
@pytest.mark.parametrize("T,H,I", PATHS)
def test_weights_keep_all_their_bits(fmt, code, T, H, I):
    """One code a row with a scale of 11 bits, times powers of two: y is exact,
    which W rounded to bf16, or a scale of fewer bits, would not give."""
    print("weights", fmt, T, H, I, flush=True)
    c = Case(_spec(fmt, H, I), 0, T, None, None, None, seed=T)
    _zero_codes(c, list(range(H)))
    per = c.q4.numel() // ((c.spec.n_experts + 1) * 3)
    q = c.q4.view(-1, per)[3 * c.expert].view(I, -1)
    at = np.arange(I) * 37 % H
    for n, k in enumerate(at):
        if fmt == "int8":
            q[n, k] = code
        else:
            q[n, k // 2] = code << 4 if k % 2 else code
    if fmt == "mxfp4":
        w = 6.0
        c.sc.fill_(127)
    else:
        w = code * (1 + 2.0 ** -10)
        c.sc.fill_(1 + 2.0 ** -10)
    x = 2.0 ** ((np.arange(T)[:, None] + np.arange(H)) % 7 - 3)
    c.x = torch.from_numpy(x).to(torch.bfloat16)
    y = w * x[:, at]
    assert np.array_equal(y, y.astype(np.float32))
    assert np.array_equal(tu.host(c.forward(True)), y)
    assert np.array_equal(tu.host(c.forward(False)), tu.bf16_round(y))


@pytest.mark.parametrize("R", [8, 40])
@pytest.mark.parametrize("each", [True, False])
@pytest.mark.parametrize("T,H,I", PATHS)
def test_adapters_keep_all_bits_of_their_sums(T, H, I, each, R):
    """W of zeros, one rank with TERMS across K, and across N: u and v need 24
    bits, and y and both gradients are single products with them."""
    print("adapters", T, H, I, each, R, flush=True)
    off = list(range(T + 1)) if each else [0, T // 2, T]
    who = [i % 2 for i in range(len(off) - 1)]
    low = tu.Low(2, R, I, H)
    low.scales = torch.tensor([0.5, -2.0])
    low.a.zero_()
    low.b.zero_()
    r = R - 3
    ka, nb = np.arange(4) * (H // 4) + 5, np.arange(4) * (I // 4) + 3
    low.a[:, r, ka] = torch.from_numpy(TERMS).to(torch.bfloat16)
    b = 2.0 ** (np.arange(I) % 5 - 2)
    low.b[:, :, r] = torch.from_numpy(b).to(torch.bfloat16)
    c = Case(_spec("int4", H, I), 0, T, off, who, low, seed=T)
    c.q4.zero_()
    c.w[:] = 0
    t = np.arange(T)
    xs, ds = 2.0 ** (t % 5 - 2), -2.0 ** (t % 3)
    c.x = torch.from_numpy(np.repeat(xs[:, None], H, axis=1)).to(torch.bfloat16)
    u = low.scales.double().numpy()[c.own] * xs * TERMS.sum()
    y = u[:, None] * b
    assert np.array_equal(tu.host(c.forward(True)), y)
    assert np.array_equal(tu.host(c.forward(False)), tu.bf16_round(y))
    # gradients: one row of each adapter is not zero
    low.b.zero_()
    low.b[:, nb, r] = torch.from_numpy(TERMS).to(torch.bfloat16)
    c.ad = low.device()
    rows = [int(np.nonzero(c.own == i)[0][-1]) for i in range(2)]
    still = np.setdiff1d(t, rows)
    c.x[still] = 0
    c.dy = torch.from_numpy(np.repeat(ds[:, None], I, axis=1)).to(torch.bfloat16)
    c.dy[still] = 0
    v = low.scales.double().numpy()[c.own] * ds * TERMS.sum()
    dx, da, db = (tu.host(g) for g in c.backward())
    ref_a, ref_b, ref_x = np.zeros(low.a.shape), np.zeros(low.b.shape), np.zeros((T, H))
    for i, row in enumerate(rows):
        ref_a[i, r], ref_b[i, :, r] = v[row] * xs[row], u[row] * ds[row]
        ref_x[row, ka] = v[row] * TERMS
    assert np.array_equal(da, ref_a) and np.array_equal(db, ref_b)
    assert np.array_equal(dx, tu.bf16_round(ref_x))
