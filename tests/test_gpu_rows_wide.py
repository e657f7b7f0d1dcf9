"""Rows by expert of wide rows with the most choices a token can have: the
routing weights' gradient of every layout that sums over several wavefronts,
with all of a token's pairs in one workgroup and spread over many.  Tolerances
as in test_gpu_rows.py."""
import pytest
import torch

import int4_routed_expert_router_amd as coli
from test_gpu_rows import BF, F32, Case, _check_backward, _check_sum

pytestmark = pytest.mark.gpu

# 256 lanes of one, two and three chunks; 512 and 1,024 lanes
WIDTHS = [1088, 2048, 4096, 6144, 6208, 8192, 8256, 16384]


@pytest.mark.parametrize("dtype,dy_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,k", [(3, 32), (40, 31), (520, 32)])
@pytest.mark.parametrize("H", WIDTHS)
def test_most_choices(H, T, k, dtype, dy_dtype):
    c = Case(T, H, 64, k, seed=H + T, drop=0.2, spare=7)
    rows, dy = c.new(c.n, dtype), c.new(T, dy_dtype, 1e-2)
    rows[~c.owned()] = float("nan")  # not read
    before = torch.full_like(rows, 7.0)
    d_rows, d_w = before.clone(), torch.full((T * k,), 7.0, device="cuda")
    coli.coli_moe_combine_backward(c.L, c.r, rows, dy, T, d_rows, d_w)
    torch.cuda.synchronize()
    for at in torch.arange(T).split(130):  # some tokens at a time: 64 bits of every pair
        part = Case.__new__(Case)
        part.T, part.k, part.H, part.n = len(at), k, H, c.n
        part.pos, part.has, part.w = (t[at[0]:at[-1] + 1] for t in (c.pos, c.has, c.w))
        _check_backward(part, rows, dy[at[0]:at[-1] + 1], None, d_w.view(T, k)[at[0]:at[-1] + 1], None)
        v = (part.w[:, :, None] * dy[at[0]:at[-1] + 1].float()[:, None, :]).to(dtype)
        assert torch.equal(d_rows[part.pos[part.has]], v[part.has])
    assert (d_rows[~c.owned()] == 7.0).all()
    again = torch.full_like(d_w, 7.0)
    coli.coli_moe_combine_backward(c.L, c.r, rows, dy, T, None, again)
    torch.cuda.synchronize()
    assert torch.equal(again, d_w)


@pytest.mark.parametrize("H", [6208, 16384])
def test_most_choices_summed(H):
    c = Case(70, H, 64, 32, seed=H, drop=0.1)
    rows, y = c.new(c.n, BF), torch.empty(70, H, device="cuda")
    rows[~c.owned()] = float("nan")
    coli.coli_moe_combine(c.L, c.r, rows, None, 70, y)
    torch.cuda.synchronize()
    _check_sum(c, rows, c.w, None, y)
