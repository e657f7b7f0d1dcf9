"""One training step of a layer with frozen experts, as its parts are used
together: route, balance loss, routed experts, the shared expert through three
projections with adapters, and all gradients -- against float64 autograd of
the same step on the host.

Every bf16 value that passes between the calls (gate, up, h, and their
gradients) is rounded on both sides at the same places, so what is left are
fp32 sums; values next to a rounding border may go either way, which moves a
sum of n terms by at most one bf16 step of one term.  The tolerance is
2^-7 of the root mean square for outputs that pass through such roundings."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import synth
import train_util as tu

pytestmark = pytest.mark.gpu


def _close(got, ref, what, tol=2.0 ** -7):
    got, ref = np.asarray(got), np.asarray(ref)
    rms = np.sqrt(np.mean(ref ** 2))
    err = np.max(np.abs(got - ref) / np.maximum(np.abs(ref), rms))
    assert err <= tol, (what, err)


def test_shared_expert_through_projections_equals_the_layer():
    """A layer's shared expert computed by three projections adds up with the
    routed experts to what the layer computes in one call."""
    spec = synth.LayerSpec(256, 128, 8, 1, 2, sigmoid=True, renorm=True)
    T = 9
    q4, sc = synth.make_weights(spec, device="cuda")
    whole = coli.Layer.from_spec(spec, q4, sc)
    routed = coli.Layer(256, 128, 8, 0, 2, spec.flags, q4, sc)
    lg, x = synth.make_logits(spec, T).cuda(), synth.make_x(spec, T).cuda()
    r = coli.Route(whole, T)
    coli.coli_moe_route(whole, lg, None, T, r)
    y = [torch.empty(T, 256, device="cuda") for _ in range(2)]
    for L, out in ((whole, y[0]), (routed, y[1])):
        coli.coli_moe_forward_decode(L, r, x, T, out, coli.COLI_OUT_F32,
                                     coli.workspace(L, T, coli.COLI_ENTRY_DECODE))
    ws = coli.project_workspace(whole, 0, None, T)
    wd = coli.project_workspace(whole, 2, None, T)
    g, u = (torch.empty(T, 128, device="cuda") for _ in range(2))
    coli.coli_moe_project(whole, 8, 0, None, None, x, T, g, coli.COLI_OUT_F32, ws)
    coli.coli_moe_project(whole, 8, 1, None, None, x, T, u, coli.COLI_OUT_F32, ws)
    h = (torch.nn.functional.silu(g) * u).to(torch.bfloat16)  # the layer keeps 16 bits of h
    s = torch.empty(T, 256, device="cuda")
    coli.coli_moe_project(whole, 8, 2, None, None, h, T, s, coli.COLI_OUT_F32, wd)
    _close((y[1] + s).cpu().numpy(), y[0].cpu().numpy(), "y")


def test_training_step_matches_autograd():
    spec = synth.LayerSpec(256, 128, 8, 1, 2, sigmoid=True, renorm=True, routed_scale=2.0)
    T, H, I, E, k = 50, 256, 128, 8, 2
    q4, sc = synth.make_weights(spec)
    L = coli.Layer.from_spec(spec, q4.cuda(), sc.cuda())
    routed = coli.Layer(H, I, E, 0, k, spec.flags, q4.cuda(), sc.cuda(), routed_scale=2.0)
    w_r, x = synth.make_router_weights(spec), synth.make_x(spec, T)
    off, who, valid = [0, 20, 45], [1, 0], np.ones(T, np.uint8)
    valid[[3, 30]] = 0
    low = {m: tu.Low(2, 8, *((H, I) if m == 2 else (I, H)), ranks=(8, 5), seed=m) for m in range(3)}
    ad = {m: low[m].device() for m in low}
    rq = coli.Requests(torch.tensor(off, dtype=torch.int32).cuda(),
                       torch.tensor(who, dtype=torch.int32).cuda())
    xd = x.cuda()

    # ---- device: forward
    r = coli.Route(L, T)
    logits = torch.empty(T, E, device="cuda")
    coli.coli_moe_route_hidden(L, w_r.cuda(), xd, None, T, logits, r)
    bal = coli.Balance(L, 2, torch.tensor(off, dtype=torch.int32).cuda(), torch.tensor(valid).cuda())
    coli.coli_moe_balance_loss(L, logits, r.topk_idx, T, bal, coli.balance_workspace(L, T, 2))
    y = torch.empty(T, H, device="cuda")
    coli.coli_moe_forward_decode(routed, r, xd, T, y, coli.COLI_OUT_F32,
                                 coli.workspace(routed, T, coli.COLI_ENTRY_DECODE))
    bf = torch.bfloat16
    g, u, s = (torch.empty(T, n, dtype=bf, device="cuda") for n in (I, I, H))
    ws = {m: coli.project_workspace(L, m, ad[m], T, True) for m in ad}
    wf = {m: coli.project_workspace(L, m, ad[m], T) for m in ad}
    for m, src, out in ((0, xd, g), (1, xd, u)):
        coli.coli_moe_project(L, E, m, ad[m], rq, src, T, out, coli.COLI_OUT_BF16, wf[m])
    h = (torch.nn.functional.silu(g.float()) * u.float()).to(bf)
    coli.coli_moe_project(L, E, 2, ad[2], rq, h, T, s, coli.COLI_OUT_BF16, wf[2])
    # ---- device: backward of sum(dy * (routed + shared)) + losses
    gen = torch.Generator().manual_seed(1)
    dy = torch.randn(T, H, generator=gen).to(bf)
    dyd = dy.cuda()
    new = lambda m: (torch.empty(low[m].a.shape, device="cuda"), torch.empty(low[m].b.shape, device="cuda"))  # noqa: E731
    grads = {m: new(m) for m in ad}
    dh = torch.empty(T, I, dtype=bf, device="cuda")
    coli.coli_moe_project_backward(L, E, 2, ad[2], rq, h, dyd, T, dh, *grads[2], ws[2])
    gf, uf = g.float().requires_grad_(True), u.float().requires_grad_(True)
    (torch.nn.functional.silu(gf) * uf).backward(dh.float())
    dx = [torch.empty(T, H, dtype=bf, device="cuda") for _ in range(2)]
    dgu = [gf.grad.to(bf), uf.grad.to(bf)]
    for m in (0, 1):
        coli.coli_moe_project_backward(L, E, m, ad[m], rq, xd, dgu[m], T, dx[m], *grads[m], ws[m])
    # gradient of the routing weights: each choice's expert output times dy, on the host
    dw = torch.randn(T * k, generator=gen)
    d_loss = torch.tensor([0.3, 0.05])
    dl = torch.empty(T, E, device="cuda")
    coli.coli_moe_route_backward(L, logits, r.topk_idx, T, dw.cuda(), bal, d_loss.cuda(), dl)
    torch.cuda.synchronize()

    # ---- host, float64
    own = tu.owners(off, who, 2, T)
    w = [tu.dense(spec, q4, sc, E, m) for m in range(3)]
    q = lambda a: torch.from_numpy(np.asarray(a)).to(bf).double().numpy()  # noqa: E731
    xh = tu.host(x)
    gh, uh = (q(tu.project(w[m], low[m], own, xh)[0]) for m in (0, 1))
    _close(tu.host(g), gh, "gate")
    _close(tu.host(u), uh, "up")
    hh = tu.host(h)
    _close(hh, gh * tu.sigmoid(gh) * uh, "h", 2.0 ** -6)
    _close(tu.host(s), tu.project(w[2], low[2], own, hh)[0], "shared")
    wr = [tu.bf16_round(m) for m in w]  # the backward pass is defined with W in bf16
    (dhh, _), (da2, _), (db2, _) = tu.project_backward(wr[2], low[2], own, hh, tu.host(dy))
    _close(tu.host(dh), dhh, "dh")
    _close(tu.host(grads[2][0]), da2, "da down")
    _close(tu.host(grads[2][1]), db2, "db down")
    for m in (0, 1):
        (dxh, _), (da, _), (db, _) = tu.project_backward(wr[m], low[m], own, xh, tu.host(dgu[m]))
        _close(tu.host(dx[m]), dxh, "dx")
        _close(tu.host(grads[m][0]), da, "da")
        _close(tu.host(grads[m][1]), db, "db")
    lh, idx = tu.host(logits), r.topk_idx.cpu().numpy().reshape(T, k).astype(np.int64)
    loss, counts, mean, tokens, totals = tu.balance(lh, idx, off, valid, True)
    assert np.array_equal(bal.counts.cpu().numpy(), counts)
    assert np.array_equal(bal.tokens.cpu().numpy(), tokens)
    _close(tu.host(bal.loss), loss, "loss", 1e-5)
    ref = tu.route_backward(lh, idx, True, True, 2.0, tu.host(dw).reshape(T, k),
                            (off, valid, counts, tokens), d_loss.double().numpy())
    _close(tu.host(dl), ref, "d_logits", 1e-5)
    # counts of the whole batch agree with the route's own where nothing is masked
    one = coli.Balance(L)
    coli.coli_moe_balance_loss(L, logits, r.topk_idx, T, one, coli.balance_workspace(L, T))
    assert torch.equal(one.counts[0], r.counts)
