"""Rows sorted by expert and back with the routing weights, and the gradients
of both, against float64.

Tolerances.  Moved rows, and a row times its weight, are exact up to the one
rounding that torch makes too: equal bits.  A sum over k rows is k + 1 additions
and k products in fp32, k + 2 half steps 2^-24 of the sum of absolute values,
and the rounding of the result.  A dot over H goes through at most 96 additions
(64 values of a lane, six steps in a wavefront, its wavefronts)."""
import pytest
import torch

import int4_routed_expert_router_amd as coli

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H24 = 2.0 ** -24
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


class Case:
    """A routed batch: `drop` is the share of pairs without a row, `spare` rows
    that no pair owns."""

    def __init__(self, T, H, E, k, seed=0, drop=0.0, spare=0):
        self.T, self.H, self.k = T, H, k
        self.L = coli.Layer(H, 64, E, 0, k, coli.COLI_ROUTE_RENORM, None, None)
        self.r = coli.Route(self.L, T)
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        coli.coli_moe_route(self.L, torch.randn(T, E, generator=self.g, device="cuda"), None, T, self.r)
        self.n = T * k + spare
        pos = self.r.pair_pos.long()
        if spare:  # spread over the larger buffer
            pos = torch.randperm(self.n, generator=self.g, device="cuda")[:T * k][pos]
        if drop:
            bad = torch.tensor([-1, self.n, -2 ** 31, 2 ** 31 - 1], device="cuda")
            gone = torch.rand(T * k, generator=self.g, device="cuda") < drop
            pos = torch.where(gone, bad[torch.arange(T * k, device="cuda") % 4], pos)
        self.r.pair_pos.copy_(pos)
        self.pos = pos.view(T, k)
        self.has = (self.pos >= 0) & (self.pos < self.n)
        self.w = self.r.topk_w.view(T, k)

    def new(self, rows, dtype, scale=1.0):
        return (torch.randn(rows, self.H, generator=self.g, device="cuda") * scale).to(dtype)

    def owned(self):
        m = torch.zeros(self.n, dtype=torch.bool, device="cuda")
        m[self.pos[self.has]] = True
        return m

    def gather(self, rows):
        """[T, k, H] in 64 bits, zeros for pairs without a row."""
        return torch.where(self.has[:, :, None], rows[self.pos * self.has].double(), 0.0)


CASES = [(1, 64, 1, 1, 0, 0), (1, 6144, 256, 8, 0, 0), (4, 6144, 256, 8, 0.3, 3),
         (5, 16384, 8, 2, 0, 1), (17, 128, 8, 8, 0.5, 0), (64, 256, 64, 32, 0, 0),
         (65, 2048, 64, 8, 0.1, 100), (130, 1088, 33, 3, 0, 0), (517, 2048, 160, 6, 0.2, 9),
         (2051, 512, 256, 8, 0, 0), (700, 4160, 16, 4, 1.0, 0), (33, 8256, 8, 2, 0, 5)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H,E,k,drop,spare", CASES)
def test_dispatch(T, H, E, k, drop, spare, dtype):
    c = Case(T, H, E, k, drop=drop, spare=spare)
    x = c.new(T, dtype)
    rows = torch.full((c.n, H), 7.0, dtype=dtype, device="cuda")
    coli.coli_moe_dispatch(c.L, c.r, x, T, rows)
    torch.cuda.synchronize()
    ref = torch.full_like(rows, 7.0)
    token = torch.arange(T, device="cuda")[:, None].expand(T, k)
    ref[c.pos[c.has]] = x[token[c.has]]
    assert torch.equal(rows, ref)  # rows without an owner too


def _check_sum(c, rows, weights, beside, out):
    v = c.gather(rows) * (1.0 if weights is None else weights.double()[:, :, None])
    ref, a = v.sum(dim=1), v.abs().sum(dim=1)
    if beside is not None:
        ref, a = ref + beside.double(), a + beside.double().abs()
    tol = ref.abs() * HALF[out.dtype] + (c.k + 2) * H24 * a
    assert ((out.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype,out_dtype,beside", [(BF, BF, True), (BF, F32, False),
                                                    (F32, BF, False), (F32, F32, True)])
@pytest.mark.parametrize("T,H,E,k,drop,spare", CASES)
def test_sums(T, H, E, k, drop, spare, dtype, out_dtype, beside, weighted):
    """Combine, and dispatch's gradient."""
    c = Case(T, H, E, k, seed=1, drop=drop, spare=spare)
    rows = c.new(c.n, dtype)
    rows[~c.owned()] = float("nan")  # not read
    b = c.new(T, dtype) if beside else None
    out = torch.full((T, H), 7.0, dtype=out_dtype, device="cuda")
    f = coli.coli_moe_combine if weighted else coli.coli_moe_dispatch_backward
    f(c.L, c.r, rows, b, T, out)
    torch.cuda.synchronize()
    _check_sum(c, rows, c.w if weighted else None, b, out)
    if beside and dtype == out_dtype:  # onto beside itself
        f(c.L, c.r, rows, b, T, b)
        torch.cuda.synchronize()
        assert torch.equal(b, out)


def _check_backward(c, rows, dy, d_rows, d_w, before):
    T, k = c.T, c.k
    if d_rows is not None:
        ref = before.clone()
        v = (c.w[:, :, None] * dy.float()[:, None, :]).to(d_rows.dtype)
        ref[c.pos[c.has]] = v[c.has]
        assert torch.equal(d_rows, ref)
    if d_w is not None:
        v = c.gather(rows) * dy.double()[:, None, :]
        err = (d_w.view(T, k).double() - v.sum(dim=2)).abs()
        assert (err <= 100 * H24 * v.abs().sum(dim=2)).all()
        assert (d_w.view(T, k)[~c.has] == 0).all()


@pytest.mark.parametrize("dtype,dy_dtype", [(BF, BF), (BF, F32), (F32, BF), (F32, F32)])
@pytest.mark.parametrize("T,H,E,k,drop,spare", CASES)
def test_combine_backward(T, H, E, k, drop, spare, dtype, dy_dtype):
    c = Case(T, H, E, k, seed=2, drop=drop, spare=spare)
    rows, dy = c.new(c.n, dtype), c.new(T, dy_dtype, 1e-2)
    rows[~c.owned()] = float("nan")  # not read
    before = torch.full_like(rows, 7.0)

    def run(d_rows, d_w, r=rows):
        coli.coli_moe_combine_backward(c.L, c.r, r, dy, T, d_rows, d_w)
        torch.cuda.synchronize()
        return d_rows, d_w

    new_w = lambda: torch.full((T * k,), 7.0, device="cuda")  # noqa: E731
    d_rows, d_w = run(before.clone(), new_w())
    _check_backward(c, rows, dy, d_rows, d_w, before)
    assert torch.equal(run(before.clone(), None, None)[0], d_rows)
    assert torch.equal(run(None, new_w())[1], d_w)
    mine = rows.clone()  # the gradient onto the rows themselves
    assert torch.equal(run(mine, new_w(), mine)[1], d_w)
    own = c.owned()
    assert torch.equal(mine[own], d_rows[own]) and mine[~own].isnan().all()


def test_gradients_are_those_of_the_forward_calls():
    """Dispatch, a product per row, combine: gradients against differences of
    the whole in float64 along a direction."""
    c = Case(9, 128, 8, 3, drop=0.2, seed=3)
    x, dy = c.new(9, F32), c.new(9, F32)
    f = torch.randn(c.n, 1, generator=c.g, device="cuda")
    rows = torch.zeros(c.n, 128, device="cuda")
    coli.coli_moe_dispatch(c.L, c.r, x, 9, rows)
    mid = rows * f
    d_mid, d_w = torch.zeros_like(rows), torch.empty(27, device="cuda")
    coli.coli_moe_combine_backward(c.L, c.r, mid, dy, 9, d_mid, d_w)
    dx = torch.empty(9, 128, device="cuda")
    coli.coli_moe_dispatch_backward(c.L, c.r, d_mid * f, None, 9, dx)
    torch.cuda.synchronize()
    ax = torch.randn(9, 128, generator=c.g, device="cuda").double()
    aw = torch.randn(9, 3, generator=c.g, device="cuda").double()
    scale = torch.where(c.has, f.double()[:, 0][c.pos * c.has], 0.0)

    def value(e, d):
        w = (c.w.double() + d * aw) * scale
        return (dy.double() * ((x.double() + e * ax) * w.sum(dim=1, keepdim=True))).sum()

    # both are linear in what moves, so the differences are exact up to 2^-52 / 1e-3
    for got, along, num in ((dx, ax, (value(1e-3, 0) - value(-1e-3, 0)) / 2e-3),
                            (d_w.view(9, 3), aw, (value(0, 1e-3) - value(0, -1e-3)) / 2e-3)):
        a = float((got.double() * along).abs().sum())
        absolute = float((dy.double().abs()[:, None, :] * (x.double().abs()[:, None, :])
                          * scale.abs()[:, :, None]).sum()) * float(along.abs().max())
        assert abs(float((got.double() * along).sum() - num)) <= 110 * H24 * absolute + 1e-9 * a


def test_a_route_of_other_tensors():
    """Positions and weights that the caller put in place of the route's own;
    what the forward calls read stays the route's."""
    c = Case(20, 256, 8, 2, seed=9)
    own = c.r.pair_pos, c.r.topk_w
    x, y = c.new(20, F32), torch.empty(20, 256, device="cuda")
    c.r.pair_pos = torch.randperm(40, generator=c.g, device="cuda").to(torch.int32)
    c.r.topk_w = torch.rand(40, generator=c.g, device="cuda")
    c.pos, c.w = c.r.pair_pos.long().view(20, 2), c.r.topk_w.view(20, 2)
    c.has = torch.ones_like(c.has)
    rows = torch.empty(40, 256, device="cuda")
    coli.coli_moe_dispatch(c.L, c.r, x, 20, rows)
    coli.coli_moe_combine(c.L, c.r, rows, None, 20, y)
    torch.cuda.synchronize()
    assert torch.equal(rows[c.pos], x[:, None, :].expand(20, 2, 256))
    _check_sum(c, rows, c.w, None, y)
    assert (c.r.c.pair_pos, c.r.c.topk_w) == tuple(t.data_ptr() for t in own)


def test_with_nothing_but_missing_pairs():
    c = Case(6, 256, 8, 2, drop=1.1)
    rows, b = c.new(c.n, BF), c.new(6, BF)
    y = torch.empty(6, 256, dtype=BF, device="cuda")
    coli.coli_moe_combine(c.L, c.r, rows, None, 6, y)
    assert (y == 0).all()
    coli.coli_moe_combine(c.L, c.r, rows, b, 6, y)
    assert torch.equal(y, b)


def test_infinities_stay_in_their_token():
    c = Case(50, 512, 8, 2, seed=4)
    rows, dy = c.new(c.n, BF), c.new(50, BF)
    y0, y1 = (torch.empty(50, 512, dtype=BF, device="cuda") for _ in range(2))
    d0, d1 = (torch.empty(100, device="cuda") for _ in range(2))
    coli.coli_moe_combine(c.L, c.r, rows, None, 50, y0)
    coli.coli_moe_combine_backward(c.L, c.r, rows, dy, 50, None, d0)
    rows[int(c.pos[7, 1]), 3] = float("inf")
    coli.coli_moe_combine(c.L, c.r, rows, None, 50, y1)
    coli.coli_moe_combine_backward(c.L, c.r, rows, dy, 50, None, d1)
    torch.cuda.synchronize()
    keep = torch.arange(50, device="cuda") != 7
    assert torch.equal(y0[keep], y1[keep]) and not y1[7].isfinite().all()
    keep = torch.arange(100, device="cuda") != 15
    assert torch.equal(d0[keep], d1[keep]) and not d1[15].isfinite()


def test_largest():
    """All 2^20 pairs, 65,536 tokens, and row buffers past 4 GiB."""
    c = Case(65536, 2304, 16, 16, seed=5)
    x = c.new(65536, BF)
    rows = torch.empty(c.n, 2304, dtype=BF, device="cuda")
    coli.coli_moe_dispatch(c.L, c.r, x, 65536, rows)
    y = torch.empty(65536, 2304, device="cuda")
    d_w = torch.empty(1 << 20, device="cuda")
    coli.coli_moe_combine(c.L, c.r, rows, None, 65536, y)
    d_rows = torch.empty_like(rows)
    coli.coli_moe_combine_backward(c.L, c.r, rows, x, 65536, d_rows, d_w)
    torch.cuda.synchronize()
    for a in range(0, 65536, 8192):
        at = torch.arange(a, a + 64, device="cuda")
        pos = c.pos[at]
        assert torch.equal(rows[pos], x[at][:, None, :].expand(64, 16, 2304))
        # weights are renormalised: y = x up to their sum
        v = c.w[at].double()[:, :, None] * x[at].double()[:, None, :]
        err = (y[at].double() - v.sum(dim=1)).abs()
        assert (err <= 19 * H24 * v.abs().sum(dim=1)).all()
        assert torch.equal(d_rows[pos], (c.w[at][:, :, None] * x[at].float()[:, None, :]).to(BF))
        sq = x[at].double().square().sum(dim=1, keepdim=True)
        assert ((d_w.view(65536, 16)[at].double() - sq).abs() <= 100 * H24 * sq).all()


@pytest.mark.parametrize("H,dtype", [(64, F32), (128, BF), (256, BF), (256, F32), (512, BF)])
def test_many_short_rows(H, dtype):
    """Rows of few lanes in buffers that go past the caches, some pairs without."""
    c = Case(65536, H, 64, 16, seed=10, drop=0.01)
    x, rows = c.new(65536, dtype), c.new(c.n, dtype)
    before = rows.clone()
    coli.coli_moe_dispatch(c.L, c.r, x, 65536, rows)
    torch.cuda.synchronize()
    token = torch.arange(65536, device="cuda")[:, None].expand(65536, 16)
    before[c.pos[c.has]] = x[token[c.has]]
    assert torch.equal(rows, before)
    rows = c.new(c.n, dtype)
    y, dx = torch.empty(65536, H, dtype=BF, device="cuda"), torch.empty(65536, H, device="cuda")
    coli.coli_moe_combine(c.L, c.r, rows, x, 65536, y)
    coli.coli_moe_dispatch_backward(c.L, c.r, rows, None, 65536, dx)
    torch.cuda.synchronize()
    _check_sum(c, rows, c.w, x, y)
    _check_sum(c, rows, None, None, dx)


def test_captured():
    c = Case(300, 1024, 64, 8, seed=6)
    x, dy = c.new(300, BF), c.new(300, BF)
    rows, d_rows = (torch.empty(c.n, 1024, dtype=BF, device="cuda") for _ in range(2))
    y, dx, d_w = torch.empty_like(x), torch.empty_like(x), torch.empty(2400, device="cuda")

    def step():
        coli.coli_moe_dispatch(c.L, c.r, x, 300, rows)
        coli.coli_moe_combine(c.L, c.r, rows, x, 300, y)
        coli.coli_moe_combine_backward(c.L, c.r, rows, dy, 300, d_rows, d_w)
        coli.coli_moe_dispatch_backward(c.L, c.r, d_rows, dy, 300, dx)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    outs = (rows, y, d_rows, d_w, dx)
    for seed in range(3):
        x.copy_(c.new(300, BF)), dy.copy_(c.new(300, BF))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


def test_two_streams():
    c, d = Case(400, 2048, 64, 8, seed=7), Case(300, 2048, 64, 8, seed=8)
    xc, xd = c.new(400, BF), d.new(300, BF)
    out = {}
    torch.cuda.synchronize()
    for name, k, x in (("c", c, xc), ("d", d, xd)):
        s = torch.cuda.Stream()
        rows = torch.empty(k.n, 2048, dtype=BF, device="cuda")
        y = torch.empty_like(x)
        for _ in range(5):
            coli.coli_moe_dispatch(k.L, k.r, x, k.T, rows, stream=s)
            coli.coli_moe_combine(k.L, k.r, rows, None, k.T, y, stream=s)
        out[name] = (s, rows, y)
    for name, k, x in (("c", c, xc), ("d", d, xd)):
        s, rows, y = out[name]
        s.synchronize()
        _check_sum(k, rows, k.w, None, y)
        assert torch.equal(rows[k.pos], x[:, None, :].expand(k.T, k.k, 2048))
