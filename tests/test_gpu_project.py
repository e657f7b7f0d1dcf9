"""A projection with the adapters of many requests, and its backward pass,
against float64 references (tests/train_util.py).

Tolerances.  Products of bf16 values are exact in fp32, and every sum of n
terms in fp32, in any order, is off by at most n half steps (2^-24) of the sum
of its terms' absolute values; a sum over rounded sums adds up both counts.
With S the sum of the absolute products:
  y  : K terms, one rounding per 64-wide group's scaling, the adapter's K + R
       terms, its scale and the parts of u (2^-24 each; 2^-16 where two parts
       are kept, for bf16 results) -- (2K + R + 8) * 2^-24 * S, plus half a
       step of a bf16 result;
  dx : the same with N for K, against W rounded to bf16;
  dA : N terms of v and T of the sum, dB: K and T."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import synth
import train_util as tu

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def _spec(fmt, H=256, I=128):
    return synth.LayerSpec(H, I, 2, 1, 1, sigmoid=False, renorm=False, int8=fmt == "int8",
                           mxfp4=fmt == "mxfp4")


class Case:
    """One batch on the device and on the host."""

    def __init__(self, spec, matrix, T, offsets, adapter, low, expert=None, seed=0):
        self.spec, self.matrix, self.T, self.low = spec, matrix, T, low
        self.expert = spec.n_experts if expert is None else expert
        q4, sc = synth.make_weights(spec, seed=seed)
        self.w = tu.dense(spec, q4, sc, self.expert, matrix)
        self.q4, self.sc = q4.cuda(), sc.cuda()
        self.L = coli.Layer.from_spec(spec, self.q4, self.sc)
        self.N, self.K = self.w.shape
        g = torch.Generator().manual_seed(seed + 5)
        self.x = torch.randn(T, self.K, generator=g).to(torch.bfloat16)
        self.dy = torch.randn(T, self.N, generator=g).to(torch.bfloat16)
        self.own = np.full(T, -1)
        self.ad = self.rq = None
        if low is not None:
            self.own = tu.owners(offsets, adapter, low.n, T)
            self.ad = low.device()
            self.rq = coli.Requests(torch.tensor(offsets, dtype=torch.int32).cuda(),
                                    torch.tensor(adapter, dtype=torch.int32).cuda())

    def forward(self, f32=True, ws=None):
        dt = torch.float32 if f32 else torch.bfloat16
        y = torch.full((self.T, self.N), float("nan"), dtype=dt, device="cuda")
        if ws is None:
            ws = coli.project_workspace(self.L, self.matrix, self.ad, self.T)
            ws.fill_(0xff)  # NaN patterns: nothing may come out of unwritten scratch
        coli.coli_moe_project(self.L, self.expert, self.matrix, self.ad, self.rq, self.x.cuda(),
                              self.T, y, coli.COLI_OUT_F32 if f32 else coli.COLI_OUT_BF16, ws)
        torch.cuda.synchronize()
        return y

    def backward(self, want_dx=True, want_grads=True):
        nan = float("nan")
        dx = torch.full((self.T, self.K), nan, dtype=torch.bfloat16, device="cuda")
        da = db = None
        if self.low is not None and want_grads:
            da = torch.full(self.low.a.shape, nan, device="cuda")
            db = torch.full(self.low.b.shape, nan, device="cuda")
        ws = coli.project_workspace(self.L, self.matrix, self.ad, self.T, True)
        ws.fill_(0xff)
        coli.coli_moe_project_backward(self.L, self.expert, self.matrix, self.ad, self.rq,
                                       self.x.cuda(), self.dy.cuda(), self.T,
                                       dx if want_dx else None, da, db, ws)
        torch.cuda.synchronize()
        return (dx if want_dx else None), da, db

    def check_forward(self):
        y, S = tu.project(self.w, self.low, self.own, tu.host(self.x))
        R = 0 if self.low is None else self.low.R
        tol = (2 * self.K + R + 8) * E24 * S
        got = tu.host(self.forward(True))
        bad = np.abs(got - y) > tol
        assert not bad.any(), (np.argwhere(bad)[:5], np.nanmax(np.abs(got - y) / tol))
        got = tu.host(self.forward(False))
        tol = tol + 2.0 ** -16 * (S - np.abs(tu.host(self.x)) @ np.abs(self.w).T)
        bad = np.abs(got - y) > tol + tu.HALF[torch.bfloat16] * (np.abs(y) + tol)
        assert not bad.any(), np.argwhere(bad)[:5]

    def check_backward(self):
        x, dy = tu.host(self.x), tu.host(self.dy)
        (dx, Sx), ga, gb = tu.project_backward(tu.bf16_round(self.w), self.low, self.own, x, dy)
        R = 0 if self.low is None else self.low.R
        gx, da, db = self.backward()
        tol = ((2 * self.N + R + 8) * E24 + 2.0 ** -16) * Sx
        bad = ~(np.abs(tu.host(gx) - dx) <= tol + tu.HALF[torch.bfloat16] * (np.abs(dx) + tol))
        assert not bad.any(), ("dx", np.argwhere(bad)[:5])
        if self.low is None:
            return
        for name, got, (ref, S), n in (("da", da, ga, self.N), ("db", db, gb, self.K)):
            bad = ~(np.abs(tu.host(got) - ref) <= (n + self.T + 8) * E24 * S)
            assert not bad.any(), (name, np.argwhere(bad)[:5])


# T, offsets, adapters of the requests: single tokens, tiles cut at odd rows,
# empty requests, rows outside every request, the same adapter several times,
# ids that mean "none", one long request
BATCHES = [
    (1, [0, 1], [0]),
    (1, [0, 1], [-1]),
    (3, [0, 1, 2, 3], [2, 0, 2]),
    (16, list(range(17)), [i % 3 for i in range(16)]),
    (37, [2, 2, 9, 10, 30, 30, 33], [1, 0, 5, 2, 1, 0]),
    (64, list(range(65)), [(7 * i) % 4 - 1 for i in range(64)]),
    (65, [0, 64, 65], [0, 1]),
    (130, [0, 1, 2, 67, 129], [0, 1, 2, 1]),
    (200, [0, 200], [2]),
    (257, [5, 100, 100, 101, 250], [-1, 1, 1, 0]),
]


@pytest.mark.parametrize("fmt", ["int4", "int8", "mxfp4"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_project_matches_reference(fmt, i):
    T, off, who = BATCHES[i]
    print("project", fmt, i, flush=True)
    spec = _spec(fmt)
    for matrix in range(3):
        N, K = (256, 128) if matrix == 2 else (128, 256)
        low = tu.Low(3, 16, N, K, ranks=(16, 1, 11), seed=i)
        Case(spec, matrix, T, off, who, low, seed=i).check_forward()


@pytest.mark.parametrize("fmt", ["int4", "int8", "mxfp4"])
@pytest.mark.parametrize("i", range(len(BATCHES)))
def test_project_backward_matches_reference(fmt, i):
    T, off, who = BATCHES[i]
    print("project backward", fmt, i, flush=True)
    spec = _spec(fmt)
    for matrix in (0, 2):
        N, K = (256, 128) if matrix == 2 else (128, 256)
        low = tu.Low(3, 16, N, K, ranks=(16, 1, 11), seed=i)
        Case(spec, matrix, T, off, who, low, seed=i).check_backward()


@pytest.mark.parametrize("R,ranks", [(8, (8, 3)), (24, (24, 17)), (40, (40, 0)), (64, (33, 64)),
                                     (72, (72, 65)), (128, (128, 97))])
def test_ranks(R, ranks):
    print("ranks", R, ranks, flush=True)
    spec = _spec("int4", 320, 192)  # neither a multiple of the tiles
    for matrix in (1, 2):
        N, K = (320, 192) if matrix == 2 else (192, 320)
        low = tu.Low(2, R, N, K, ranks=ranks, seed=R)
        c = Case(spec, matrix, 150, [0, 70, 71, 150], [0, 1, 0], low, seed=R)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("shape", [(64, 64), (64, 128), (576, 64), (2048, 512), (6144, 2048)])
@pytest.mark.parametrize("T", [1, 5, 70])
def test_layer_shapes(shape, T):
    print("shape", shape, T, flush=True)
    spec = _spec("int4", *shape)
    for matrix in (0, 2):
        N, K = (shape[0], shape[1]) if matrix == 2 else (shape[1], shape[0])
        low = tu.Low(2, 8, N, K, seed=T)
        c = Case(spec, matrix, T, [0, T // 2, T], [1, 0], low, seed=T)
        c.check_forward()
        c.check_backward()


@pytest.mark.parametrize("fmt", ["int4", "mxfp4"])
def test_without_adapters_and_of_a_routed_expert(fmt):
    spec = _spec(fmt)
    for T in (1, 17, 300):
        c = Case(spec, 0, T, None, None, None, expert=1, seed=T)
        c.check_forward()
        c.check_backward()


def test_scale_and_rank_tables_are_optional():
    low = tu.Low(2, 16, 128, 256, scaled=False)
    c = Case(_spec("int4"), 0, 40, [0, 20, 40], [0, 1], low)
    assert c.ad.rank is None and c.ad.scale is None
    c.check_forward()
    c.check_backward()


def test_long_batch():
    """Several row ranges per adapter, tiles of every kind, a tail row."""
    T = 1111
    off = [0, 3, 500, 501, 640, 1100]
    low = tu.Low(3, 32, 128, 256, ranks=(32, 30, 8))
    c = Case(_spec("int4"), 0, T, off, [0, 1, 2, 0, 1], low)
    c.check_forward()
    c.check_backward()


def test_other_rows_do_not_leak():
    """NaN and infinities in rows without an adapter, and in other requests,
    stay in their own rows and out of other adapters' gradients."""
    low = tu.Low(2, 16, 128, 256)
    off, who = [0, 10, 40, 41, 90], [0, -1, 1, 0]
    c = Case(_spec("int4"), 0, 100, off, who, low)
    ref = [tu.host(t) for t in (c.forward(), *c.backward())]
    x, dy = c.x.clone(), c.dy.clone()
    bad = list(range(10, 40)) + [40, 95, 99]  # request 1, adapter 1's only row, rows outside
    for t in bad:
        c.x[t, ::3] = float("nan")
        c.x[t, 1::3] = float("inf")
        c.dy[t, ::2] = float("nan")
    got = [tu.host(t) for t in (c.forward(), *c.backward())]
    ok = np.setdiff1d(np.arange(100), bad)
    assert np.array_equal(got[0][ok], ref[0][ok]) and np.array_equal(got[1][ok], ref[1][ok])
    assert np.array_equal(got[2][0], ref[2][0]) and np.array_equal(got[3][0], ref[3][0])
    assert np.isnan(got[0][bad]).all()


@pytest.mark.parametrize("R", [8, 24, 40, 64, 72, 128])
@pytest.mark.parametrize("rows", [1, 2, 3, 7, 9, 21, 33])
def test_request_lengths_and_ranks(R, rows):
    """Requests of a few rows each, at ranks on both sides of where the second
    launch goes row by row; the tables of offsets below and above 64 entries."""
    n = max(2, 100 // rows)
    off = [rows * i for i in range(n + 1)]
    low = tu.Low(5, R, 128, 192, ranks=(R, 1, max(1, R - 3), R, R // 2))
    Case(_spec("int4", 192, 128), 0, rows * n + 3, off, [(3 * i) % 6 - 1 for i in range(n)],
         low).check_forward()


@pytest.mark.parametrize("T,H,I,fmt", [(60, 256, 128, "int4"), (60, 4160, 128, "int4"),
                                       (300, 256, 128, "int8"), (1100, 512, 4096, "int4"),
                                       (1100, 512, 4096, "mxfp4"), (1100, 4096, 512, "int8")])
def test_broken_adapters_and_rows_stay_alone(T, H, I, fmt):
    """An adapter full of NaN and infinities, and a row that is not finite,
    leave the rows of other requests in the same tiles and other adapters'
    gradients as they are; gradients past a rank stay zero."""
    low = tu.Low(3, 16, I, H, ranks=(13, 16, 5))
    off, who = [0, 3, 10, 21, 22, 37, T - 5], [0, 1, 2, 1, 0, 2]
    c = Case(_spec(fmt, H, I), 0, T, off, who, low)
    ref = [tu.host(t) for t in (c.forward(), c.forward(False), *c.backward())]
    low.a[1], low.b[1] = float("nan"), float("inf")
    c.ad = low.device()
    c.x[37], c.dy[37] = float("inf"), float("inf")  # request 5's first row, adapter 2
    got = [tu.host(t) for t in (c.forward(), c.forward(False), *c.backward())]
    own = c.own.copy()
    own[37] = 1
    ok = own != 1
    for g, r in zip(got[:3], ref[:3]):
        assert np.array_equal(g[ok], r[ok])
        assert not np.isfinite(g[own == 1]).any()
    assert np.array_equal(got[3][0], ref[3][0]) and np.array_equal(got[4][0], ref[4][0])
    assert not got[3][2, 5:].any() and not got[4][2, :, 5:].any()


def test_rows_do_not_depend_on_their_batch():
    """Same bits twice, and outputs wanted one at a time are the same bits."""
    low = tu.Low(2, 16, 128, 256)
    c = Case(_spec("int8"), 0, 77, [0, 30, 77], [1, 0], low)
    a, b = c.forward(), c.forward()
    assert torch.equal(a, b)
    full, again = c.backward(), c.backward()
    for p, q in zip(full, again):
        assert torch.equal(p, q)
    dx, _, _ = c.backward(want_grads=False)
    _, da, db = c.backward(want_dx=False)
    assert torch.equal(dx, full[0]) and torch.equal(da, full[1]) and torch.equal(db, full[2])


def test_gradients_match_differences():
    """The formulas of the backward pass against central differences of the
    float64 projection, at a few entries; and the device against the formulas."""
    low = tu.Low(2, 8, 128, 256, ranks=(8, 5))
    c = Case(_spec("int4"), 0, 21, [0, 8, 20], [0, 1], low)
    c.check_backward()
    x, dy = tu.host(c.x), tu.host(c.dy)
    (dx, _), (da, _), (db, _) = tu.project_backward(c.w, low, c.own, x, dy)
    rng = np.random.default_rng(0)

    def loss(x, i=None, a=None, b=None):
        y = x @ c.w.T
        for j in range(low.n):
            A, B, s = low.of(j)
            if j == i:
                A, B = (A if a is None else a), (B if b is None else b)
            at = c.own == j
            y[at] += s * (x[at] @ A.T) @ B.T
        return np.sum(y * dy)

    h = 1e-3  # the loss is quadratic at most along one entry: differences are exact
    for _ in range(6):
        t, k, n = rng.integers(21), rng.integers(256), rng.integers(128)
        p, m = x.copy(), x.copy()
        p[t, k] += h
        m[t, k] -= h
        assert abs((loss(p) - loss(m)) / (2 * h) - dx[t, k]) < 1e-6 * (1 + abs(dx[t, k]))
        i = int(rng.integers(2))
        A, B, _s = low.of(i)
        r = rng.integers(A.shape[0])
        for M, G, at in ((A, da[i], (r, k)), (B, db[i], (n, r))):
            p, m = M.copy(), M.copy()
            p[at] += h
            m[at] -= h
            kw = "a" if M is A else "b"
            d = (loss(x, i, **{kw: p}) - loss(x, i, **{kw: m})) / (2 * h)
            assert abs(d - G[at]) < 1e-6 * (1 + abs(G[at]))


@pytest.mark.parametrize("T", [7, 70, 1300])
def test_extreme_weight_scales(T):
    """fp16 scales down to the smallest subnormal, E8M0 scales near both ends."""
    print("extreme scales", T, flush=True)
    for fmt, lo, hi, shift in (("int4", 0, 0, 0), ("int8", 0, 0, 0), ("mxfp4", 1, 12, 90),
                               ("mxfp4", 240, 251, -100)):
        spec = _spec(fmt, 2048, 512)
        c = Case(spec, 2, T, [0, T], [0], tu.Low(1, 8, 2048, 512), seed=3)
        g = torch.Generator().manual_seed(T)
        if fmt == "mxfp4":
            sc = torch.randint(lo, hi, c.sc.shape, generator=g, dtype=torch.uint8)
        else:
            bits = torch.randint(1, 0x0420, c.sc.shape, generator=g, dtype=torch.int32)
            sc = bits.to(torch.int16).view(torch.float16)  # subnormals and the first normals
        c.sc.copy_(sc)
        c.w = tu.dense(spec, c.q4.cpu(), sc, c.expert, 2)
        c.x = (c.x.double() * 2.0 ** shift).to(torch.bfloat16)
        c.low.a = (c.low.a.double() * 2.0 ** -shift).to(torch.bfloat16)
        c.ad = c.low.device()
        c.check_forward()


def _captured(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()  # the first launches outside the capture
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    torch.cuda.synchronize()
    return g


@pytest.mark.parametrize("T", [5, 90, 1500])
def test_captured_calls_replay(T):
    """Forward and backward captured into two graphs that share a workspace,
    replayed in turn with new inputs and eager calls in between."""
    print("graphs", T, flush=True)
    N = 2048 if T > 1000 else 128
    spec = _spec("int4", 256, N)
    low = tu.Low(2, 16, N, 256, ranks=(16, 7))
    c = Case(spec, 0, T, [0, T // 2, T], [1, 0], low)
    x, dy = c.x.cuda(), c.dy.cuda()
    y = torch.empty(T, N, device="cuda")
    dx = torch.empty(T, 256, dtype=torch.bfloat16, device="cuda")
    da, db = torch.empty(low.a.shape, device="cuda"), torch.empty(low.b.shape, device="cuda")
    ws = coli.project_workspace(c.L, 0, c.ad, T, True)
    wf = coli.project_workspace(c.L, 0, c.ad, T)
    ws = ws if ws.numel() > wf.numel() else wf

    def forward():
        coli.coli_moe_project(c.L, c.expert, 0, c.ad, c.rq, x, T, y, coli.COLI_OUT_F32, ws)

    def backward():
        coli.coli_moe_project_backward(c.L, c.expert, 0, c.ad, c.rq, x, dy, T, dx, da, db, ws)

    gf, gb = _captured(forward), _captured(backward)
    for i in range(4):
        g = torch.Generator().manual_seed(100 + i)
        x.copy_(torch.randn(T, 256, generator=g))
        dy.copy_(torch.randn(T, N, generator=g))
        forward()
        backward()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, dx, da, db)]
        for t in (y, dx, da, db):
            t.fill_(-1.0)
        if i % 2:
            ws.fill_(0xff)
        gb.replay()
        gf.replay()
        torch.cuda.synchronize()
        for a, b in zip((y, dx, da, db), want):
            assert torch.equal(a, b), i


def test_two_streams_at_once():
    """Calls on two streams with a workspace each do not disturb each other."""
    cases = [Case(_spec(f), 0, 300, [0, 100, 300], [0, 1], tu.Low(2, 16, 128, 256, seed=i), seed=i)
             for i, f in enumerate(("int4", "mxfp4"))]
    ref = [c.forward() for c in cases]
    st = [torch.cuda.Stream() for _ in cases]
    xs = [c.x.cuda() for c in cases]
    ys = [torch.empty_like(r) for r in ref]
    ws = [coli.project_workspace(c.L, 0, c.ad, 300) for c in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate(cases):
            coli.coli_moe_project(c.L, c.expert, 0, c.ad, c.rq, xs[i], 300, ys[i],
                                  coli.COLI_OUT_F32, ws[i], stream=st[i])
    torch.cuda.synchronize()
    for y, r in zip(ys, ref):
        assert torch.equal(y, r)


@pytest.mark.parametrize("T", [1, 33, 129, 600])
def test_workspace_for_more_rows_serves_fewer(T):
    low = tu.Low(2, 16, 128, 256)
    c = Case(_spec("int4"), 0, T, [0, T], [1], low)
    ws = coli.project_workspace(c.L, 0, c.ad, 5000)
    assert torch.equal(c.forward(ws=ws), c.forward())


@pytest.mark.parametrize("fmt", ["int4", "int8", "mxfp4"])
def test_long_batches_match_reference(fmt):
    """Batches that take the tiled product: whole and cut tiles, an odd number
    of 64-wide stages, many short requests between long ones."""
    print("long", fmt, flush=True)
    for (H, I), T in (((320, 4096), 700), ((192, 2112), 1555)):
        spec = _spec(fmt, H, I)
        off = [0, 3, 300] + list(range(301, 340)) + [600, T - 7]
        who = [(5 * i) % 4 - 1 for i in range(len(off) - 1)]
        low = tu.Low(3, 24, I, H, ranks=(24, 9, 17))
        c = Case(spec, 0, T, off, who, low, seed=T)
        c.check_forward()
        c.check_backward()
        low = tu.Low(3, 24, H, I, ranks=(24, 9, 17))
        c = Case(spec, 2, T, off, who, low, seed=T)
        c.check_forward()
        c.check_backward()  # dx [T, I] of the wide side


def test_thousands_of_requests():
    """More requests than the backward pass looks through per adapter."""
    T = 2000
    off = list(range(0, T + 1))
    who = [(7 * i) % 9 - 1 for i in range(T)]
    low = tu.Low(8, 8, 128, 256)
    c = Case(_spec("int4"), 0, T, off, who, low)
    c.check_forward()
    c.check_backward()
