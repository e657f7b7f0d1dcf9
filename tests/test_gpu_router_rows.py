"""Rows of the balance loss and the route's gradient at the edges of fp32's
exponentials, against float64 (tests/train_util.py; tolerances as in
test_gpu_balance.py): probabilities, losses and gradients of rows whose
largest logit is given."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import train_util as tu
from test_gpu_balance import E24, _check, _grad_scale, _inputs, _layer, _run

pytestmark = pytest.mark.gpu


def _rows(T, E, k, top, seed=0):
    """Logits of a spread of about 17 below a largest one of `top`."""
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * 3
    l = l - l.amax(dim=1, keepdim=True) + top
    return l, l.topk(k, dim=1).indices.to(torch.int32)


@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("top", [-88.0, -80.5, -79.5, -76.0, -72.0, -60.0, -20.5, -19.5, 0.0, 19.5,
                                 20.5, 60.0, 79.5, 80.5])
def test_rows_by_their_largest_logit(top, sig):
    T, E, k = 70, 256, 8
    print("largest logit", top, sig, flush=True)
    l, idx = _rows(T, E, k, top)
    lh, ih = tu.host(l), idx.numpy().astype(np.int64)
    dw, d_loss = torch.randn(T, k, generator=torch.Generator().manual_seed(1)), torch.tensor([0.7, -0.3])
    D = np.max(np.max(lh, axis=1) - np.min(lh, axis=1))
    for renorm in (False, True):
        L = _layer(E, k, sig, renorm)
        b = _run(L, l, idx, T)
        _check(L, l, idx, None, None, sig, b)
        bal = ([0, T], None, b.counts.cpu().numpy(), b.tokens.cpu().numpy())
        for use_w, use_b in ((True, True), (True, False), (False, True)):
            dl = torch.full((T, E), float("nan"), device="cuda")
            coli.coli_moe_route_backward(L, l.cuda(), idx.cuda(), T, dw.cuda() if use_w else None,
                                         b if use_b else None, d_loss.cuda() if use_b else None, dl)
            args = (sig, renorm, 1.0, tu.host(dw) if use_w else None, bal if use_b else None,
                    d_loss.double().numpy())
            ref, S = tu.route_backward(lh, ih, *args), _grad_scale(lh, ih, *args)
            bad = ~(np.abs(tu.host(dl) - ref) <= (4 * D + 2 * E + 64) * E24 * S + 1e-35)
            assert not bad.any(), (renorm, use_w, use_b, np.argwhere(bad)[:4])


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (256, 8), (7, 3), (1024, 32)])
@pytest.mark.parametrize("sig", [False, True])
@pytest.mark.parametrize("renorm", [False, True])
def test_rows_without_a_finite_logit(E, k, sig, renorm):
    """A counted row of -inf alone has no probabilities: its gradients are
    zero, also those of its routing weights, and other rows keep their bits."""
    T, gone = 37, [0, 5, 6, 36]
    print("rows of -inf", E, k, sig, renorm, flush=True)
    L = _layer(E, k, sig, renorm, 2.5)
    g = torch.Generator().manual_seed(E)
    l = torch.randn(T, E, generator=g)
    idx = l.topk(k, dim=1).indices.to(torch.int32)
    dw, d_loss = torch.randn(T, k, generator=g), torch.tensor([0.7, -0.3])
    b = _run(L, l, idx, T)  # the counts are inputs here, and the same for both
    rest = np.setdiff1d(np.arange(T), gone)
    for use_w, use_b in ((True, True), (True, False), (False, True)):
        got = []
        for rows in ([], gone):
            x = l.clone()
            x[rows] = float("-inf")
            dl = torch.full((T, E), float("nan"), device="cuda")
            coli.coli_moe_route_backward(L, x.cuda(), idx.cuda(), T, dw.cuda() if use_w else None,
                                         b if use_b else None, d_loss.cuda() if use_b else None, dl)
            got.append(tu.host(dl))
        assert np.array_equal(got[1][gone], np.zeros((len(gone), E))), (use_w, use_b)
        assert np.array_equal(got[1][rest], got[0][rest]), (use_w, use_b)


@pytest.mark.parametrize("E,k", [(8, 2), (256, 8)])
@pytest.mark.parametrize("n_seq", [1, 2, 9, 40, 3000])
def test_few_rows_in_many_sequences(E, k, n_seq):
    """A padded table of sequences, most of them empty: results, and that a
    single workgroup is left alone only with a few of them."""
    T = 40
    print("sequences", E, n_seq, flush=True)
    inner = np.sort(np.random.default_rng(n_seq).integers(0, T + 1, n_seq - 1))
    off = np.concatenate(([0], inner, [T])).tolist()
    valid = (np.arange(T) % 7 != 1).astype(np.uint8)
    l, idx = _inputs(T, E, k)
    L = _layer(E, k, True)
    _check(L, l, idx, off, valid, True, _run(L, l, idx, T, off, valid))
    with coli.KernelTimer() as timer:
        _run(L, l, idx, T, off, valid)
    names = [n for n, _ in timer.results()]
    timer.close()
    assert names == (["balance", "balance_finish"] if n_seq * -(-E // 16) > 8 else ["balance"])
