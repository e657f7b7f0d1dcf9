"""Balance loss, per-expert counts and the gradient of the route against
float64 references (tests/train_util.py).

Tolerances.  The exponential's argument l - max is rounded to half a step and
multiplied by log2 e, so a spread D of the logits costs up to 2 D half steps
(2^-24) of each probability; the hardware exponential, the logarithm and the
divisions a few steps more.  A row's sum of E terms adds E half steps and a
mean over n rows n: REL = (2 D + E + 32) * 2^-24 for a probability, + n for
means.  Gradients are differences of products of these: REL of the sum of the
absolute values of what is subtracted."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import train_util as tu

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def _layer(E, k, sig, renorm=False, scale=1.0):
    flags = (coli.COLI_ROUTE_SIGMOID if sig else coli.COLI_ROUTE_SOFTMAX) | (
        coli.COLI_ROUTE_RENORM if renorm else 0)
    return coli.Layer(64, 64, E, 0, k, flags, None, None, routed_scale=scale)


def _inputs(T, E, k, seed=0, spread=1.5, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * spread + shift
    return l, l.topk(k, dim=1).indices.to(torch.int32)


def _run(L, l, idx, T, off=None, valid=None):
    n = 1 if off is None else len(off) - 1
    o = None if off is None else torch.tensor(off, dtype=torch.int32).cuda()
    v = None if valid is None else torch.tensor(valid, dtype=torch.uint8).cuda()
    b = coli.Balance(L, n, o, v)
    for t in (b.counts, b.tokens, b.totals):
        t.fill_(-7)
    b.mean_prob.fill_(float("nan"))
    b.loss.fill_(float("nan"))
    ws = coli.balance_workspace(L, T, n)
    ws.fill_(0xff)
    coli.coli_moe_balance_loss(L, l.cuda(), idx.cuda(), T, b, ws)
    torch.cuda.synchronize()
    return b


def _check(L, l, idx, off, valid, sig, b):
    T, E = l.shape
    live = np.zeros(T, bool)
    for s, e in tu.spans([0, T] if off is None else off, T):
        live[s:e] = True
    if valid is not None:
        live &= np.asarray(valid) != 0
    lh = tu.host(l)
    lh[~live] = 0.0
    loss, counts, mean, tokens, totals = tu.balance(
        lh, idx.numpy().astype(np.int64), [0, T] if off is None else off, valid, sig)
    assert np.array_equal(b.counts.cpu().numpy(), counts)
    assert np.array_equal(b.tokens.cpu().numpy(), tokens)
    assert np.array_equal(b.totals.cpu().numpy(), totals)
    fin = np.where(np.isfinite(lh), lh, 0.0)
    D = np.max(np.max(fin, axis=1) - np.min(fin, axis=1))
    rel = (2 * D + E + 32) * E24
    n = tokens.max() if len(tokens) else 0
    assert (np.abs(tu.host(b.mean_prob) - mean) <= (rel + n * E24) * mean + 1e-30).all()
    got = tu.host(b.loss)
    assert abs(got[0] - loss[0]) <= (rel + (n + 4) * E24) * loss[0]
    # the logarithm's argument is off by rel, so lse by rel, absolutely; max |lse| bounds the square
    m = np.max(np.abs(tu.lse(np.where(np.isfinite(lh), lh, -1e30)))) if T else 0.0
    assert abs(got[1] - loss[1]) <= 2 * m * (rel + 4 * E24 * m) + 4 * E24 * loss[1]
    return counts, tokens


# T, sequence offsets: one row, one tile, cut tiles, empty sequences, rows outside, many tiles
BATCHES = [
    (1, None), (4, None), (5, [0, 2, 2, 5]), (64, [0, 64]), (65, None), (70, [3, 3, 9, 60]),
    (513, [0, 8, 16, 17, 400, 513]), (2051, [0, 1000, 1000, 2048]),
    (5000, [10, 11, 4096, 4990]), (300, list(range(0, 301, 3))),
]


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (256, 8), (160, 6), (7, 3), (1, 1), (1024, 32),
                                 (30, 30)])
@pytest.mark.parametrize("sig", [False, True])
def test_balance_matches_reference(E, k, sig):
    L = _layer(E, k, sig)
    for i, (T, off) in enumerate(BATCHES):
        if E == 1024 and T > 600:
            continue
        print("balance", E, k, sig, T, flush=True)
        l, idx = _inputs(T, E, k, seed=i)
        valid = None if i % 2 == 0 else (np.arange(T) * 7 % 5 != 1).astype(np.uint8)
        _check(L, l, idx, off, valid, sig, _run(L, l, idx, T, off, valid))


def test_many_sequences():
    """More sequences than workgroups; most of them empty."""
    T, E = 700, 64
    rng = np.random.default_rng(3)
    off = np.sort(rng.integers(0, T + 1, 6001)).tolist()
    l, idx = _inputs(T, E, 4)
    L = _layer(E, 4, True)
    _check(L, l, idx, off, None, True, _run(L, l, idx, T, off))


def test_rows_that_do_not_count_may_hold_anything():
    T, E, k = 200, 64, 4
    L = _layer(E, k, False)
    l, idx = _inputs(T, E, k)
    off, valid = [20, 90, 150], np.ones(T, np.uint8)
    valid[30:60] = 0
    l[30:60], l[:20], l[150:] = float("nan"), float("inf"), float("-inf")
    idx[30:60] = 1 << 30
    b = _run(L, l, idx, T, off, valid)
    idx2 = idx.clone()
    idx2[30:60] = 0
    counts, tokens = _check(L, l, idx2, off, valid, False, b)
    dl = torch.full((T, E), float("nan"), device="cuda")
    dw = torch.ones(T, k)
    dw[30:60] = float("nan")
    coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, dw.cuda(), b,
                                 torch.ones(2).cuda(), dl)
    got = tu.host(dl)
    dead = np.r_[0:20, 30:60, 150:T]
    assert np.array_equal(got[dead], np.zeros_like(got[dead]))
    assert np.isfinite(got).all()


def test_nothing_counts():
    T, E = 40, 64
    L = _layer(E, 4, True)
    l, idx = _inputs(T, E, 4)
    for off, valid in ((None, np.zeros(T, np.uint8)), ([5, 5], None), ([40, 40, 40], None)):
        b = _run(L, l, idx, T, off, valid)
        for t in (b.counts, b.mean_prob, b.tokens, b.totals, b.loss):
            assert (t == 0).all()
        dl = torch.full((T, E), float("nan"), device="cuda")
        coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, None, b, torch.ones(2).cuda(), dl)
        assert (dl == 0).all()


@pytest.mark.parametrize("sig", [False, True])
def test_extreme_logits(sig):
    """Spreads and offsets at which exponentials leave the range of fp32, and
    experts switched off by -inf."""
    T, E, k = 48, 64, 4
    L = _layer(E, k, sig)
    for shift, spread in ((-200.0, 3.0), (200.0, 3.0), (0.0, 60.0), (1e4, 1.0), (-1e4, 1.0)):
        l, idx = _inputs(T, E, k, spread=spread, shift=shift)
        l[::2, 10:30] = float("-inf")
        idx = l.topk(k, dim=1).indices.to(torch.int32)
        b = _run(L, l, idx, T)
        lh = tu.host(l)
        with np.errstate(all="ignore"):
            loss, counts, mean, _, _ = tu.balance(lh, idx.numpy().astype(np.int64), [0, T], None, sig)
        D = np.max(lh) - np.min(lh[np.isfinite(lh)])
        # a logit's own half step, |l| 2^-24, moves its probability by as much
        rel = (2 * D + 2 * np.abs(lh[np.isfinite(lh)]).max() + E + T + 32) * E24
        assert (np.abs(tu.host(b.mean_prob) - mean) <= rel * mean + 1e-30).all(), (shift, spread)
        assert abs(tu.host(b.loss)[0] - loss[0]) <= rel * loss[0]
        assert abs(tu.host(b.loss)[1] - loss[1]) <= 2 * rel * (loss[1] + np.sqrt(loss[1]))
    l[3] = float("-inf")  # a row without any expert: no probability, no z term
    b = _run(L, l, idx, T)
    assert torch.isfinite(b.loss).all() and torch.isfinite(b.mean_prob).all()
    dl = torch.full((T, E), float("nan"), device="cuda")
    coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, None, b, torch.ones(2).cuda(), dl)
    assert torch.isfinite(dl).all() and (dl[3] == 0).all()


def _grad_scale(lh, idx, sig, renorm, scale, dw, bal, d_loss):
    """Sum of the absolute values of what each entry of d_logits is made of."""
    T, E = lh.shape
    S = np.zeros((T, E))
    p = tu.probs(lh, sig)
    sm = tu.probs(lh, False)
    if bal is not None:
        off, valid, counts, tokens = bal
        n_live, n_all = max(1, (tokens > 0).sum()), max(1, tokens.sum())
        for s in range(len(off) - 1):
            if not tokens[s]:
                continue
            f = E * counts[s] / (idx.shape[1] * tokens[s])
            r = slice(max(0, off[s]), off[s + 1])
            S[r] += abs(d_loss[0]) / (n_live * tokens[s]) * p[r] * (f + (f * p[r]).sum(1, keepdims=True))
            S[r] += 2 * abs(d_loss[1]) / n_all * np.abs(tu.lse(lh[r]))[:, None] * sm[r]
    if dw is not None:
        w = np.abs(tu.weights(lh, idx, sig, renorm, scale))
        part = w * (np.abs(dw) + ((w / abs(scale) * np.abs(dw)).sum(1, keepdims=True)
                                  if renorm else 0))
        np.add.at(S, (np.arange(T)[:, None], idx), part)
        if not sig and not renorm:
            S += p * (w * np.abs(dw)).sum(1, keepdims=True)
    return S


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (256, 8), (160, 6), (7, 3), (1, 1), (1024, 32),
                                 (30, 30), (16, 16)])
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_matches_reference(E, k, sig, renorm):
    scale = 2.5
    L = _layer(E, k, sig, renorm, scale)
    for i, (T, off) in enumerate(BATCHES):
        if (E == 1024 and T > 600) or T > 2500:
            continue
        print("route backward", E, k, sig, renorm, T, flush=True)
        l, idx = _inputs(T, E, k, seed=i)
        valid = None if i % 2 == 0 else (np.arange(T) * 7 % 5 != 1).astype(np.uint8)
        g = torch.Generator().manual_seed(i)
        dw = torch.randn(T, k, generator=g)
        d_loss = torch.tensor([0.7, -0.3])
        b = _run(L, l, idx, T, off, valid)
        lh, ih = tu.host(l), idx.numpy().astype(np.int64)
        o = [0, T] if off is None else off
        bal = (o, valid, b.counts.cpu().numpy(), b.tokens.cpu().numpy())
        D = np.max(np.max(lh, axis=1) - np.min(lh, axis=1))
        for use_w, use_b in ((True, True), (True, False), (False, True)):
            dl = torch.full((T, E), float("nan"), device="cuda")
            coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, dw.cuda() if use_w else None,
                                         b if use_b else None, d_loss.cuda() if use_b else None, dl)
            args = (sig, renorm, scale, tu.host(dw) if use_w else None, bal if use_b else None,
                    d_loss.double().numpy())
            ref = tu.route_backward(lh, ih, *args)
            S = _grad_scale(lh, ih, *args)
            bad = ~(np.abs(tu.host(dl) - ref) <= (4 * D + 2 * E + 64) * E24 * S + 1e-35)
            assert not bad.any(), (T, use_w, use_b, np.argwhere(bad)[:4])


def test_gradient_matches_differences():
    """The reference's gradient against central differences of the losses."""
    T, E, k = 6, 8, 3
    for sig in (False, True):
        for renorm in (False, True):
            l, idx = _inputs(T, E, k, seed=3)
            lh, ih = tu.host(l), idx.numpy().astype(np.int64)
            off, valid = [0, 4, 6], np.array([1, 0, 1, 1, 1, 1], np.uint8)
            _, counts, _, tokens, totals = tu.balance(lh, ih, off, valid, sig)
            rng = np.random.default_rng(1)
            dw, d_loss = rng.standard_normal((T, k)), np.array([0.8, 0.1])
            dw[1] = 0.0  # the row that does not count
            f = E * counts / (k * tokens[:, None])
            rows = [(t, s, 1 / (totals[1] * tokens[s]), 1 / totals[0])
                    for s in range(2) for t in range(off[s], off[s + 1]) if valid[t]]
            ref = tu.route_backward(lh, ih, sig, renorm, 1.5, dw, (off, valid, counts, tokens), d_loss)
            h = 1e-4  # truncation h^2 times third derivatives of order one
            for t in range(T):
                for e in range(E):
                    p, m = lh.copy(), lh.copy()
                    p[t, e] += h
                    m[t, e] -= h
                    d = (tu.losses_of(p, rows, f, sig, dw, ih, renorm, 1.5, d_loss) -
                         tu.losses_of(m, rows, f, sig, dw, ih, renorm, 1.5, d_loss)) / (2 * h)
                    assert abs(d - ref[t, e]) < 1e-6


def test_same_bits_twice_and_misaligned_rows():
    """Results do not depend on the run; logits that are not 16-byte aligned
    take the scalar loads and agree within the tolerance."""
    T, E, k = 900, 64, 8
    L = _layer(E, k, True, True)
    l, idx = _inputs(T, E, k)
    a, b = _run(L, l, idx, T), _run(L, l, idx, T)
    for n in ("counts", "mean_prob", "loss", "tokens"):
        assert torch.equal(getattr(a, n), getattr(b, n))
    buf = torch.empty(T * E + 1, device="cuda")
    odd = buf[1:].view(T, E)
    odd.copy_(l)
    c = _run(L, odd, idx, T)
    assert torch.equal(c.counts, a.counts)
    assert torch.allclose(c.mean_prob, a.mean_prob, rtol=(2 * 20 + E + T + 32) * E24, atol=0)


def test_captured_calls_replay():
    """Loss and gradient captured together and replayed with new logits."""
    T, E, k = 777, 64, 4
    L = _layer(E, k, True, True)
    off = torch.tensor([0, 100, 777], dtype=torch.int32).cuda()
    l, idx = _inputs(T, E, k)
    l, idx = l.cuda(), idx.cuda()
    b = coli.Balance(L, 2, off)
    ws = coli.balance_workspace(L, T, 2)
    dw, d_loss = torch.randn(T, k, device="cuda"), torch.rand(2, device="cuda")
    dl = torch.empty(T, E, device="cuda")

    def step():
        coli.coli_moe_balance_loss(L, l, idx, T, b, ws)
        coli.coli_moe_route_backward(L, l, idx, T, dw, b, d_loss, dl)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(5):
        l.copy_(_inputs(T, E, k, seed=50 + i)[0])
        idx.copy_(l.topk(k, dim=1).indices)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (b.loss, b.counts, b.mean_prob, b.tokens, dl)]
        for t in (b.loss, b.counts, b.mean_prob, b.tokens, dl):
            t.fill_(-1)
        ws.fill_(0xff)
        g.replay()
        torch.cuda.synchronize()
        for a, w in zip((b.loss, b.counts, b.mean_prob, b.tokens, dl), want):
            assert torch.equal(a, w), i


def test_an_expert_named_twice_counts_twice():
    T, E, k = 70, 16, 3
    L = _layer(E, k, False)
    l, idx = _inputs(T, E, k)
    idx[:, 2] = idx[:, 0]
    b = _run(L, l, idx, T)
    ih = idx.numpy().astype(np.int64)
    assert np.array_equal(b.counts.cpu().numpy()[0], np.bincount(ih.reshape(-1), minlength=E))
    dw = torch.randn(T, k)
    dl = torch.empty(T, E, device="cuda")
    coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, dw.cuda(), None, None, dl)
    ref = tu.route_backward(tu.host(l), ih, False, False, 1.0, tu.host(dw))
    S = _grad_scale(tu.host(l), ih, False, False, 1.0, tu.host(dw), None, None)
    assert (np.abs(tu.host(dl) - ref) <= (4 * 20 + 2 * E + 64) * E24 * S + 1e-35).all()
