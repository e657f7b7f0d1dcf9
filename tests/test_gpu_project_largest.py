"""The projection and its backward pass at the largest sizes the calls take:
65,536 rows of a 16,384 x 16,384 matrix, whose buffers pass 2 GiB.  Rows at
both ends and at the boundaries of requests against float64 (tolerances as in
test_gpu_project.py)."""
import pytest
import torch

import int4_routed_expert_router_amd as coli

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24
T, D, R = 65536, 16384, 8
OFF, WHO = [0, 1, 40000, 65535, 65536], [1, 0, 1, 0]
ROWS = [0, 1, 32767, 39999, 40000, 65534, 65535]


def _dense(codes, scales):
    """Matrix 1 of the first expert in float64, a block of rows at a time."""
    q = codes[D * D // 2:D * D].view(D, D // 2)
    w = torch.empty(D, D, dtype=torch.float64, device="cuda")
    for r in range(0, D, 1024):
        b = q[r:r + 1024]
        nib = torch.stack((b & 15, b >> 4), dim=-1).view(-1, D).to(torch.int16)
        w[r:r + 1024] = (nib - 16 * (nib > 7)).double()
    s = scales[D * D // 64:2 * D * D // 64].view(D, D // 64).double()
    w.view(D, D // 64, 64).mul_(s[:, :, None])
    return w


def test_largest_batch():
    print("largest", flush=True)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (3 * D * D // 2,), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(3 * D * D // 64, generator=g, device="cuda") * 0.02 + 0.001).half()
    L = coli.Layer(D, D, 1, 0, 1, 0, codes, scales)
    x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    a = (torch.randn(2, R, D, generator=g, device="cuda") * D ** -0.5).to(torch.bfloat16)
    b = torch.randn(2, D, R, generator=g, device="cuda").to(torch.bfloat16)
    ad = coli.Adapters(a, b)
    rq = coli.Requests(torch.tensor(OFF, dtype=torch.int32).cuda(),
                       torch.tensor(WHO, dtype=torch.int32).cuda())
    y = torch.full((T, D), float("nan"), device="cuda")
    ws = coli.project_workspace(L, 1, ad, T)
    ws.fill_(0xff)
    coli.coli_moe_project(L, 0, 1, ad, rq, x, T, y, coli.COLI_OUT_F32, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(y.view(-1, D)).all()
    w = _dense(codes, scales)
    owner = [next(WHO[i] for i in range(4) if OFF[i] <= t < OFF[i + 1]) for t in ROWS]

    def check(got, ref, S, n, half, what):
        tol = (2 * n + R + 8) * E24 * S
        tol = tol + (half * (ref.abs() + tol + 2.0 ** -16 * S) + 2.0 ** -16 * S if half else 0)
        bad = ~((got.double() - ref).abs() <= tol)
        assert not bad.any(), (what, bad.nonzero()[:4].tolist())

    def sums(z, m, outer, inner):
        """z m^T, the owners' adapters added, and the same of absolute values."""
        out = torch.empty(2, len(ROWS), D, dtype=torch.float64, device="cuda")
        for i, t in enumerate(ROWS):
            for j, f in enumerate((lambda v: v, torch.abs)):
                p, q = f(outer[owner[i]].double()), f(inner[owner[i]].double())
                zi = f(z[t].double())
                out[j, i] = p.mv(q.mv(zi))
        zr = z[ROWS].double()
        for r in range(0, D, 2048):
            out[0, :, r:r + 2048] += zr @ m[r:r + 2048].t()
            out[1, :, r:r + 2048] += zr.abs() @ m[r:r + 2048].abs().t()
        return out[0], out[1]

    ref, S = sums(x, w, b, a)
    check(y[ROWS], ref, S, D, 0, "y")
    del y, ws
    dy = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    dx = torch.full((T, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    da, db = torch.empty(a.shape, device="cuda"), torch.empty(b.shape, device="cuda")
    ws = coli.project_workspace(L, 1, ad, T, True)
    ws.fill_(0xff)
    coli.coli_moe_project_backward(L, 0, 1, ad, rq, x, dy, T, dx, da, db, ws)
    torch.cuda.synchronize()
    assert torch.isfinite(dx).all()
    wt = w.float().to(torch.bfloat16).double().t().contiguous()
    del w
    ref, S = sums(dy, wt, a.transpose(1, 2), b.transpose(1, 2))
    check(dx[ROWS], ref, S, D, 2.0 ** -8, "dx")
    # the gradients' first ranks, columns at both ends: sums over all rows
    cols = [0, 1, 8191, D - 1]
    part = torch.zeros(2, 2, len(cols), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(part)
    for i in range(4):
        for lo in range(OFF[i], OFF[i + 1], 8192):
            at = slice(lo, min(lo + 8192, OFF[i + 1]))
            xs, ds, q = x[at].double(), dy[at].double(), WHO[i]
            a0, b0 = a[q, 0].double(), b[q, :, 0].double()
            part[0, q] += xs[:, cols].t() @ ds.mv(b0)
            part[1, q] += ds[:, cols].t() @ xs.mv(a0)
            size[0, q] += xs[:, cols].abs().t() @ ds.abs().mv(b0.abs())
            size[1, q] += ds[:, cols].abs().t() @ xs.abs().mv(a0.abs())
    tol = (D + T + 8) * E24 * size
    assert ((da[:, 0, cols].double() - part[0]).abs() <= tol[0]).all()
    assert ((db[:, cols, 0].double() - part[1]).abs() <= tol[1]).all()
