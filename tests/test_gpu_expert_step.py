"""A training step of a layer with frozen experts through its parts, as they
are used together: norm, route, rows by expert, each expert's projections, rows
back to their tokens, the gradients of all of it back to the residual stream,
the router and the norm, and clipping -- against float64 autograd of the same
step.

Tolerance.  Values pass from call to call in bf16.  A rounding moves a vector
by at most half a step, 2^-8 of its 2-norm, and the products in between (random
matrices of many rows) pass relative errors on as they are; the longest chain,
from x to d_weight, has 16 roundings, counting both factors of SwiGLU's
gradient: results are within 16 * 2^-8 of their 2-norm.  A wrong weight, row or
sign is off by about 1."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import synth
import train_util as tu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def _near(got, ref, what, tol=16 * 2.0 ** -8):
    got, ref = got.detach().double().cpu(), ref.detach().double().cpu()
    err = float((got - ref).norm() / ref.norm())
    assert err <= tol, (what, err)


def _experts(L, r, rows, back=None):
    """The experts' outputs of sorted rows; with `back` (their gradient) the
    gradient of the rows."""
    n, H = rows.shape
    I, out = L.inter, torch.empty_like(rows)
    off = r.offsets.tolist()
    for e in range(L.n_experts):
        t = off[e + 1] - off[e]
        if t == 0:
            continue
        x = rows[off[e]:off[e + 1]]
        ws = [coli.project_workspace(L, m, None, t, back is not None) for m in range(3)]
        fw = [coli.project_workspace(L, m, None, t) for m in range(3)]
        g, u = (torch.empty(t, I, dtype=BF, device="cuda") for _ in range(2))
        coli.coli_moe_project(L, e, 0, None, None, x, t, g, coli.COLI_OUT_BF16, fw[0])
        coli.coli_moe_project(L, e, 1, None, None, x, t, u, coli.COLI_OUT_BF16, fw[1])
        gf, uf = g.float().requires_grad_(True), u.float().requires_grad_(True)
        h = torch.nn.functional.silu(gf) * uf
        if back is None:
            coli.coli_moe_project(L, e, 2, None, None, h.detach().to(BF), t, out[off[e]:off[e + 1]],
                                  coli.COLI_OUT_BF16, fw[2])
            continue
        dh = torch.empty(t, I, dtype=BF, device="cuda")
        dy = back[off[e]:off[e + 1]]
        coli.coli_moe_project_backward(L, e, 2, None, None, h.detach().to(BF), dy, t, dh, None,
                                       None, ws[2])
        h.backward(dh.float())
        dx = [torch.empty(t, H, dtype=BF, device="cuda") for _ in range(2)]
        for m, d in ((0, gf.grad), (1, uf.grad)):
            coli.coli_moe_project_backward(L, e, m, None, None, x, d.to(BF), t, dx[m], None, None,
                                           ws[m])
        out[off[e]:off[e + 1]] = (dx[0].float() + dx[1].float()).to(BF)
    return out


@pytest.mark.parametrize("residual", [BF, torch.float32])
def test_step(residual):
    spec = synth.LayerSpec(256, 128, 8, 0, 2, sigmoid=True, renorm=True, routed_scale=2.0)
    T, H, E, k = 61, 256, 8, 2
    q4, sc = synth.make_weights(spec, device="cuda")
    L = coli.Layer.from_spec(spec, q4, sc)
    g = torch.Generator().manual_seed(0)
    x, res = torch.randn(T, H, generator=g).to(BF).cuda(), torch.randn(T, H, generator=g).to(residual).cuda()
    w_r = synth.make_router_weights(spec).cuda()
    w_n = (torch.randn(H, generator=g) * 0.2 + 1).cuda()
    dy, d_stream = torch.randn(T, H, generator=g).to(BF).cuda(), torch.randn(T, H, generator=g).to(residual).cuda()

    # ---- forward
    n, r = coli.Norm(H, w_n), coli.Route(L, T)
    total, xn = torch.empty_like(res), torch.empty_like(x)
    coli.coli_moe_norm(n, x, res, total, T, xn)
    logits = torch.empty(T, E, device="cuda")
    coli.coli_moe_route_hidden(L, w_r, xn, None, T, logits, r)
    rows = torch.empty(T * k, H, dtype=BF, device="cuda")
    coli.coli_moe_dispatch(L, r, xn, T, rows)
    outs = _experts(L, r, rows)
    y = torch.empty(T, H, device="cuda")
    coli.coli_moe_combine(L, r, outs, None, T, y)
    # the layer's own forward call of the same input
    whole = torch.empty(T, H, device="cuda")
    coli.coli_moe_forward_decode(L, r, xn, T, whole, coli.COLI_OUT_F32,
                                 coli.workspace(L, T, coli.COLI_ENTRY_DECODE))
    _near(y, whole, "forward call", 4 * 2.0 ** -8)  # gate, up, h and the output in bf16

    # ---- backward
    d_outs, d_w = torch.empty_like(outs), torch.empty(T * k, device="cuda")
    coli.coli_moe_combine_backward(L, r, outs, dy, T, d_outs, d_w)
    d_rows = _experts(L, r, rows, d_outs)
    d_logits = torch.empty(T, E, device="cuda")
    coli.coli_moe_route_backward(L, logits, r.topk_idx, T, d_w, None, None, d_logits)
    d_router = d_logits.t() @ xn.float()
    through = (d_logits @ w_r.float()).to(BF)
    d_xn = torch.empty_like(x)
    coli.coli_moe_dispatch_backward(L, r, d_rows, through, T, d_xn)
    dx, d_res, d_wn = torch.empty_like(x), torch.empty_like(res), torch.empty(H, device="cuda")
    coli.coli_moe_norm_backward(n, total, T, d_xn, d_stream, dx, d_res, d_wn,
                                coli.norm_workspace(n, T))
    grads = [d_router.contiguous(), d_wn]
    before = [t.clone() for t in grads]
    norm = torch.empty(2, device="cuda")
    coli.coli_moe_clip_gradients(coli.Gradients(grads), 0.5, norm, coli.clip_workspace())
    torch.cuda.synchronize()

    # ---- float64, on the host
    leaf = lambda t: t.detach().cpu().double().requires_grad_(True)  # noqa: E731
    xh, rh, wr, wn = leaf(x), leaf(res), leaf(w_r), leaf(w_n)
    s = xh + rh
    v = s / torch.sqrt(s.square().mean(dim=1, keepdim=True) + 1e-6) * wn
    lg = v @ wr.t()
    idx = r.topk_idx.cpu().long().view(T, k)
    w = torch.sigmoid(lg).gather(1, idx)
    w = 2.0 * w / w.sum(dim=1, keepdim=True)
    ref = torch.zeros(T, H, dtype=torch.float64)
    for e in range(E):
        gate, up, down = (torch.from_numpy(tu.dense(spec, q4, sc, e, m)) for m in range(3))
        f = (torch.nn.functional.silu(v @ gate.t()) * (v @ up.t())) @ down.t()
        ref = ref + f * (w * (idx == e)).sum(dim=1, keepdim=True)
    ((ref * dy.cpu().double()).sum() + (s * d_stream.cpu().double()).sum()).backward()
    _near(y, ref, "y")
    _near(dx, xh.grad, "dx")
    _near(d_res, rh.grad, "d_residual")
    _near(before[0], wr.grad, "d_router")
    _near(before[1], wn.grad, "d_weight")
    size = np.sqrt(sum(float(t.double().square().sum()) for t in before))
    assert abs(float(norm[0]) - size) <= size * 2.0 ** -23 and size > 0.5
    for a, b in zip(before, grads):
        assert torch.equal(a * norm[1], b)
    after = np.sqrt(sum(float(t.double().square().sum()) for t in grads))
    assert abs(after - 0.5) <= 0.5 * 2.0 ** -21  # the factor's, the products' and the norm's half steps


def test_serving_step_on_codes():
    """Norm with codes in front of the MX path: the layer's output of the codes
    is that of the norm's y, which the router sees."""
    spec = synth.LayerSpec(512, 256, 16, 1, 4, sigmoid=True, renorm=True, mxfp4=True)
    T = 200
    q4, sc = synth.make_weights(spec, device="cuda")
    L = coli.Layer(512, 256, 16, 1, 4, spec.flags | coli.COLI_ACT_MXFP8, q4, sc, mxfp4=True)
    x, res = synth.make_x(spec, T, seed=1).cuda(), synth.make_x(spec, T, seed=2).cuda()
    w_r = synth.make_router_weights(spec).cuda()
    n, r = coli.Norm(512, torch.ones(512, device="cuda")), coli.Route(L, T)
    y, total = torch.empty_like(x), torch.empty_like(res)
    q, e = (torch.empty(T, m, dtype=torch.uint8, device="cuda") for m in (512, 16))
    logits = torch.empty(T, 16, device="cuda")
    out = [torch.empty(T, 512, dtype=BF, device="cuda") for _ in range(2)]
    ws = coli.workspace(L, T, coli.COLI_ENTRY_PREFILL)
    coli.coli_moe_norm(n, x, res, total, T, y, coli.COLI_NORM_MXFP8, q, e)
    coli.coli_moe_route_hidden(L, w_r, y, None, T, logits, r)
    coli.coli_moe_forward_prefill_quantized(L, r, q, e, T, out[0], coli.COLI_OUT_BF16, ws)
    coli.coli_moe_forward_prefill(L, r, y, T, out[1], coli.COLI_OUT_BF16, ws)
    torch.cuda.synchronize()
    assert torch.equal(out[0], out[1]) and out[0].float().abs().max() > 0
