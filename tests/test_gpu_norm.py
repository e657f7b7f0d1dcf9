"""The norm with residual and codes, and its backward pass, against float64.

Tolerances.  A row's sum of squares goes through at most 96 fp32 additions in
any of the layouts (up to 64 values of a lane one after another, six steps in a
wavefront, its wavefronts), each off by half a step 2^-24; the mean, the
reciprocal root (half of the mean's error) and three products add a few more:
REL = 64 half steps on y before its rounding to bf16, 2^-8.  Gradients are sums
of products: 128 half steps of the sum of the absolute values of their terms,
mean(n h) with that of |n h|.  d_weight adds rows one after another, spread over
256 groups or more (T / 256 + 1 additions), up to 32 of them side by side, and
up to 1,536 groups, every 64th one after another (24) and then 64 sums; or, for
a few rows, four and up to 128 side by side.  DW = 193 half steps beside T /
256, of which 64 are those of each h, is over both."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli
import synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
H24 = 2.0 ** -24
DW = 1 + 32 + 24 + 64 + 64 + 8
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}
TYPES = {"none": None, "bf16": BF, "f32": F32}


def _inputs(T, H, residual, weight, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, H, generator=g) * scale).to(BF).cuda()
    res = None if residual is None else (torch.randn(T, H, generator=g) * 3 * scale).to(residual).cuda()
    w = None if weight is None else (torch.randn(H, generator=g) * 0.3 + 1).to(weight).cuda()
    return x, res, w


def _run(x, res, w, fmt=coli.COLI_NORM_PLAIN, y=True, eps=1e-6):
    T, H = x.shape
    n = coli.Norm(H, w, eps)
    out = dict(total=None if res is None else torch.full_like(res, 7.0),
               y=torch.full_like(x, 7.0) if y else None, q=None, scales=None)
    if fmt == coli.COLI_NORM_Q8_0:
        out["q"] = torch.full((T, H), 99, dtype=torch.int8, device="cuda")
        out["scales"] = torch.full((T, H // 32), 7.0, dtype=torch.float16, device="cuda")
    elif fmt == coli.COLI_NORM_MXFP8:
        out["q"] = torch.full((T, H), 99, dtype=torch.uint8, device="cuda")
        out["scales"] = torch.full((T, H // 32), 99, dtype=torch.uint8, device="cuda")
    coli.coli_moe_norm(n, x, res, out["total"], T, out["y"], fmt, out["q"], out["scales"])
    torch.cuda.synchronize()
    return out


def _check(x, res, w, out, eps=1e-6):
    total = x if res is None else (res.float() + x.float()).to(res.dtype)
    if res is not None:  # one addition and one rounding: no room
        assert torch.equal(out["total"], total)
    s = total.double()
    ref = s / torch.sqrt(s.square().mean(dim=1, keepdim=True) + eps)
    if w is not None:
        ref = ref * w.double()
    err = (out["y"].double() - ref).abs()
    # below the normal range a step is absolute
    assert (err <= ref.abs() * (2.0 ** -8 + 64 * H24) + 2.0 ** -134).all()
    return ref


def _codes(y, fmt):
    n = y.numel()
    if fmt == coli.COLI_NORM_Q8_0:
        q = torch.empty(y.shape, dtype=torch.int8, device="cuda")
        d = torch.empty(n // 32, dtype=torch.float16, device="cuda")
        coli.coli_moe_quantize_q8_0(y, coli.COLI_SRC_BF16, n, q, d)
    else:
        q = torch.empty(y.shape, dtype=torch.uint8, device="cuda")
        d = torch.empty(n // 32, dtype=torch.uint8, device="cuda")
        coli.coli_moe_quantize_mxfp8(y, coli.COLI_SRC_BF16, n, q, d)
    torch.cuda.synchronize()
    return q, d


SIZES = [(1, 8), (1, 6144), (2, 16384), (3, 16), (5, 520), (4, 2048), (7, 2056), (64, 256),
         (65, 1024), (33, 4104), (130, 128), (517, 2048), (2051, 6144), (1025, 8192), (600, 16384)]


@pytest.mark.parametrize("residual", ["none", "bf16", "f32"])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm(T, H, residual):
    weight = (BF, F32, None)[(T + H // 8) % 3]
    x, res, w = _inputs(T, H, TYPES[residual], weight, seed=T + H)
    _check(x, res, w, _run(x, res, w))


@pytest.mark.parametrize("fmt", [coli.COLI_NORM_Q8_0, coli.COLI_NORM_MXFP8])
@pytest.mark.parametrize("T,H", [(1, 32), (1, 6144), (3, 96), (5, 544), (9, 2048), (64, 256),
                                 (517, 2048), (33, 4128), (1100, 6144), (2, 16384), (700, 16384)])
def test_codes_are_those_of_the_quantiser(T, H, fmt):
    x, res, w = _inputs(T, H, (BF, F32, None)[T % 3], BF, seed=T)
    out = _run(x, res, w, fmt)
    _check(x, res, w, out)
    q, d = _codes(out["y"], fmt)
    assert torch.equal(out["q"], q)
    assert torch.equal(out["scales"].view(-1).view(torch.uint8), d.view(torch.uint8))
    # and without y
    again = _run(x, res, w, fmt, y=False)
    assert torch.equal(again["q"], q) and torch.equal(again["scales"], out["scales"])


@pytest.mark.parametrize("fmt", [coli.COLI_NORM_Q8_0, coli.COLI_NORM_MXFP8])
def test_codes_of_ragged_blocks(fmt):
    """Blocks of zeros and of very unequal values, steps and halves: a weight
    that is a table of magnitudes makes y what the test wants, as a row of equal
    values has y = +-weight up to eps."""
    H, T = 8192, 4
    g = torch.Generator().manual_seed(5)
    m = torch.randint(0, 255, (H,), generator=g).float() / 2
    m[:512] = 0
    m[512:1024] *= 1e-30
    m[1024:1536] *= 1e30
    m[1536:2048] *= 2.0 ** -126
    m[2048:2560] = 0.0
    m[2048:2560:32] = 448.0
    m[2560:3584] = torch.rand(1024, generator=g) * 2.0 ** torch.randint(-20, 9, (1024,), generator=g)
    m[3584:4096] = torch.arange(512) / 512 * 127.5
    m[4096:4128] = 2.0 ** -133
    w = m.cuda()
    x = torch.where(torch.rand(T, H, generator=g) < 0.5, -1.0, 1.0).to(BF).cuda()
    out = _run(x, None, w, fmt, eps=1e-30)
    q, d = _codes(out["y"], fmt)
    assert torch.equal(out["q"], q)
    assert torch.equal(out["scales"].view(-1).view(torch.uint8), d.view(torch.uint8))


def test_in_place_and_streams():
    T, H = 300, 2048
    x, res, w = _inputs(T, H, F32, BF)
    ref = _run(x, res, w)
    n = coli.Norm(H, w)
    s = torch.cuda.Stream()
    x2, r2 = x.clone(), res.clone()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        coli.coli_moe_norm(n, x2, r2, r2, T, x2)  # total over residual, y over x
    s.synchronize()
    assert torch.equal(r2, ref["total"]) and torch.equal(x2, ref["y"])
    x3 = x.clone()
    torch.cuda.synchronize()
    coli.coli_moe_norm(n, x3, res, ref["total"], T, x3, stream=s)
    s.synchronize()
    assert torch.equal(x3, ref["y"])


def test_rows_stand_alone():
    T, H = 40, 2048
    x, res, w = _inputs(T, H, BF, BF)
    clean = _run(x, res, w, coli.COLI_NORM_MXFP8)
    x[3, 5], x[20, 100], res[31, 0] = float("nan"), float("inf"), float("-inf")
    x[10], res[10] = 0, 0  # a row of nothing
    out = _run(x, res, w, coli.COLI_NORM_MXFP8)
    keep = [t for t in range(T) if t not in (3, 10, 20, 31)]
    for name in ("total", "y", "q", "scales"):
        assert torch.equal(out[name][keep], clean[name][keep])
    assert out["y"][3].isnan().all()
    assert not out["y"][20].isfinite().all() and not out["y"][31].isfinite().all()
    for name in ("total", "y", "q", "scales"):
        assert (out[name][10].float() == 0).all()


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** -10, 2.0 ** 50])
def test_scale(scale):
    x, res, w = _inputs(17, 4096, F32, F32, scale=scale)
    _check(x, res, w, _run(x, res, w, eps=1e-30), eps=1e-30)


def test_every_bf16_value():
    """The stored sum for every finite bf16 x, subnormal ones among them, beside
    nothing, a value of its own size and a tiny one."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    x = x[x.isfinite()].view(255, 256).cuda()
    g = torch.Generator(device="cuda").manual_seed(6)
    near = (x.float() * (torch.rand(x.shape, generator=g, device="cuda") * 2 - 1)).to(BF)
    for res in (torch.zeros_like(x), near, torch.full_like(x, 1e-40)):
        out = _run(x, res, None)
        # -0 + 0 is +0 in both
        assert torch.equal(out["total"].view(torch.int16), (x.float() + res.float()).to(BF).view(torch.int16))


def test_many_rows():
    """More rows than a launch has workgroups, and buffers past 2 GiB."""
    g = torch.Generator(device="cuda").manual_seed(1)
    for T, H in (((1 << 18) + 3, 16), ((1 << 17) + 1, 16384)):
        x = torch.randn(T, H, generator=g, device="cuda").to(BF)
        out = _run(x, None, None, coli.COLI_NORM_PLAIN if H < 32 else coli.COLI_NORM_Q8_0)
        for at in (slice(0, 64), slice(T // 2, T // 2 + 64), slice(T - 64, T)):
            _check(x[at], None, None, {"y": out["y"][at]})
            if out["q"] is not None:
                q, d = _codes(out["y"][at].contiguous(), coli.COLI_NORM_Q8_0)
                assert torch.equal(out["q"][at], q) and torch.equal(out["scales"][at].reshape(-1), d)


@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("T,H", [(40001, 2048), (14001, 6144), (200001, 416)])
def test_large_streams(T, H, residual):
    """Calls of over 384 MB, which go past the caches."""
    g = torch.Generator(device="cuda").manual_seed(3)
    new = lambda dt, s: (torch.randn(T, H, generator=g, device="cuda") * s).to(dt)  # noqa: E731
    x, res, w = new(BF, 1.0), new(TYPES[residual], 3.0), torch.rand(H, generator=g, device="cuda")
    out = _run(x, res, w, coli.COLI_NORM_MXFP8)
    _check(x, res, w, out)
    q, d = _codes(out["y"], coli.COLI_NORM_MXFP8)
    assert torch.equal(out["q"], q) and torch.equal(out["scales"].view(-1), d)
    dy, d_total = new(BF, 1e-2), new(TYPES[residual], 1e-2)
    _check_backward(out["total"], dy, w, d_total, _backward(out["total"], dy, w, d_total))


# ------------------------------------------------------------------ the path

@pytest.mark.parametrize("H,I,kind,act", [
    (256, 256, "int4", False), (512, 256, "int4", False), (192, 128, "int4", False),
    (256, 128, "int8", False), (512, 256, "mxfp4", False), (512, 256, "mxfp4", True)])
def test_prefill_of_codes_is_prefill_of_y(H, I, kind, act):
    spec = synth.LayerSpec(H, I, 8, 1, 2, sigmoid=True, renorm=True, int8=kind == "int8",
                           mxfp4=kind == "mxfp4")
    T = 77
    q4, sc = synth.make_weights(spec, device="cuda")
    flags = spec.flags | (coli.COLI_ACT_MXFP8 if act else 0)
    L = coli.Layer(H, I, 8, 1, 2, flags, q4, sc, int8=spec.int8, mxfp4=spec.mxfp4)
    x, res, w = _inputs(T, H, BF, BF)
    out = _run(x, res, w, coli.COLI_NORM_MXFP8 if act else coli.COLI_NORM_Q8_0)
    r = coli.Route(L, T)
    coli.coli_moe_route(L, synth.make_logits(spec, T).cuda(), None, T, r)
    ws = coli.workspace(L, T, coli.COLI_ENTRY_PREFILL)
    for dt, t in ((coli.COLI_OUT_F32, F32), (coli.COLI_OUT_BF16, BF)):
        a, b = (torch.zeros(T, H, dtype=t, device="cuda") for _ in range(2))
        ws.fill_(0xff)
        coli.coli_moe_forward_prefill(L, r, out["y"], T, a, dt, ws)
        ws.fill_(0xff)
        coli.coli_moe_forward_prefill_quantized(L, r, out["q"], out["scales"], T, b, dt, ws)
        torch.cuda.synchronize()
        assert torch.equal(a, b) and a.float().abs().max() > 0


# ------------------------------------------------------------------ backward

def _reference(total, dy, w, d_total, eps=1e-6):
    s, g = total.double(), dy.double()
    n = g if w is None else g * w.double()
    r = 1 / torch.sqrt(s.square().mean(dim=1, keepdim=True) + eps)
    h = s * r
    m, ma = (n * h).mean(dim=1, keepdim=True), (n * h).abs().mean(dim=1, keepdim=True)
    d, a = r * (n - h * m), r * (n.abs() + h.abs() * ma)
    if d_total is not None:
        d, a = d + d_total.double(), a + d_total.double().abs()
    return d, a, (g * h).sum(dim=0), (g * h).abs().sum(dim=0)


def _backward(total, dy, w, d_total, eps=1e-6, dx=True, dr=True, dw=True):
    T, H = total.shape
    n = coli.Norm(H, w, eps)
    out = dict(dx=torch.full((T, H), 7.0, dtype=BF, device="cuda") if dx else None,
               d_residual=torch.full_like(total, 7.0) if dr else None,
               d_weight=torch.full((H,), 7.0, device="cuda") if dw else None)
    ws = None
    if dw:
        ws = coli.norm_workspace(n, T)
        ws.fill_(0xff)
    coli.coli_moe_norm_backward(n, total, T, dy, d_total, out["dx"], out["d_residual"],
                                out["d_weight"], ws)
    torch.cuda.synchronize()
    return out


def _check_backward(total, dy, w, d_total, out):
    T = total.shape[0]
    d, a, dw, aw = _reference(total, dy, w, d_total)
    for name in ("dx", "d_residual"):
        if out[name] is not None:
            tol = d.abs() * HALF[out[name].dtype] + 130 * H24 * a
            assert ((out[name].double() - d).abs() <= tol).all(), name
    if out["d_weight"] is not None:
        tol = (T / min(T, 256) + DW) * H24 * aw
        assert ((out["d_weight"].double() - dw).abs() <= tol).all()


def _back_inputs(T, H, dtype, weight, through, seed):
    g = torch.Generator().manual_seed(seed)
    total = (torch.randn(T, H, generator=g) * 3).to(dtype).cuda()
    dy = (torch.randn(T, H, generator=g) * 1e-2).to(BF).cuda()
    w = None if weight is None else (torch.randn(H, generator=g) * 0.3 + 1).to(weight).cuda()
    d_total = (torch.randn(T, H, generator=g) * 1e-2).to(dtype).cuda() if through else None
    return total, dy, w, d_total


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,H", SIZES)
def test_norm_backward(T, H, dtype):
    total, dy, w, d_total = _back_inputs(T, H, dtype, (BF, F32, None)[T % 3], T % 2 == 0, T + H)
    _check_backward(total, dy, w, d_total, _backward(total, dy, w, d_total))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,few", [(64, 512), (128, 256), (256, 128), (512, 64), (520, 32),
                                   (2048, 16), (4096, 8), (6144, 4), (8192, 4), (16384, 2)])
def test_backward_few_rows(H, few, dtype):
    """On both sides of the number of rows that one workgroup takes."""
    for T in (2, 3, few - 1, few, few + 1):
        total, dy, w, d_total = _back_inputs(T, H, dtype, BF, True, T)
        _check_backward(total, dy, w, d_total, _backward(total, dy, w, d_total))


@pytest.mark.parametrize("asked", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1)])
def test_backward_parts(asked):
    total, dy, w, d_total = _back_inputs(70, 1024, F32, BF, True, 1)
    whole = _backward(total, dy, w, d_total)
    part = _backward(total, dy, w, d_total, dx=asked[0], dr=asked[1], dw=asked[2])
    for name, a in zip(("dx", "d_residual", "d_weight"), asked):
        assert (part[name] is None) == (not a)
        assert part[name] is None or torch.equal(part[name], whole[name])


def test_backward_in_place_and_repeated():
    total, dy, w, d_total = _back_inputs(1500, 2048, BF, BF, True, 2)
    one = _backward(total, dy, w, d_total)
    two = _backward(total, dy, w, d_total)
    assert all(torch.equal(one[k], two[k]) for k in one)  # the same bits
    n = coli.Norm(2048, w)
    dw = torch.empty(2048, device="cuda")
    dy2, dt2 = dy.clone(), d_total.clone()
    coli.coli_moe_norm_backward(n, total, 1500, dy2, dt2, dy2, dt2, dw, coli.norm_workspace(n, 1500))
    torch.cuda.synchronize()
    assert torch.equal(dy2, one["dx"]) and torch.equal(dt2, one["d_residual"])
    assert torch.equal(dw, one["d_weight"])


def test_backward_rows_stand_alone():
    total, dy, w, d_total = _back_inputs(30, 512, BF, BF, True, 3)
    clean = _backward(total, dy, w, d_total)
    total[4, 7], dy[9, 0] = float("nan"), float("inf")
    total[15] = 0
    out = _backward(total, dy, w, d_total)
    keep = [t for t in range(30) if t not in (4, 9, 15)]
    assert torch.equal(out["dx"][keep], clean["dx"][keep])
    assert out["dx"][15].isfinite().all()  # a row of zeros: r dy w, r = 1 / sqrt(eps)


def test_backward_against_differences():
    """The gradient along a direction against central differences of the norm
    itself in float64."""
    total, dy, w, _ = _back_inputs(6, 264, F32, F32, False, 4)
    out = _backward(total, dy, w, None)
    g = torch.Generator().manual_seed(9)
    along = torch.randn(6, 264, generator=g).double().cuda()
    along_w = torch.randn(264, generator=g).double().cuda()
    s, wd = total.double(), w.double()

    def value(a, b):
        v, u = s + a * along, wd + b * along_w
        return (dy.double() * u * v / torch.sqrt(v.square().mean(dim=1, keepdim=True) + 1e-6)).sum()

    eps = 1e-5
    num = (value(eps, 0) - value(-eps, 0)) / (2 * eps)
    num_w = (value(0, eps) - value(0, -eps)) / (2 * eps)
    _, a, _, aw = _reference(total, dy, w, None)
    # the device's error along the direction, and the differences' own (their
    # third derivatives are of the order of the terms over |s|^2 = 9)
    tol = float((along.abs() * a).sum()) * (131 * H24 + 1e-9)
    assert abs(float((out["d_residual"].double() * along).sum() - num)) <= tol
    tol = float((along_w.abs() * aw).sum()) * ((1 + DW) * H24 + 1e-9)
    assert abs(float((out["d_weight"].double() * along_w).sum() - num_w)) <= tol


def test_backward_many_rows():
    """Buffers past 2 GiB, and more rows than workgroups by far."""
    g = torch.Generator(device="cuda").manual_seed(2)
    for T, H in ((300007, 64), (70001, 16384)):
        total = torch.randn(T, H, generator=g, device="cuda").to(BF)
        dy = (torch.randn(T, H, generator=g, device="cuda") * 1e-2).to(BF)
        out = _backward(total, dy, None, None, dr=False)
        aw, dw = (torch.zeros(H, dtype=torch.float64, device="cuda") for _ in range(2))
        for at in torch.arange(T, device="cuda").split(4096):
            d, a, w, b = _reference(total[at], dy[at], None, None)
            dw, aw = dw + w, aw + b
            tol = d.abs() * 2.0 ** -8 + 130 * H24 * a
            assert ((out["dx"][at].double() - d).abs() <= tol).all()
        assert ((out["d_weight"].double() - dw).abs() <= (T / 256 + DW) * H24 * aw).all()


def test_captured():
    """Forward and backward in one graph, replayed with eager work between."""
    T, H = 200, 1024
    x, res, w = _inputs(T, H, BF, BF)
    n, dw = coli.Norm(H, w), torch.empty(H, device="cuda")
    total, y, dx = torch.empty_like(res), torch.empty_like(x), torch.empty_like(x)
    ws = coli.norm_workspace(n, T)

    def step():
        coli.coli_moe_norm(n, x, res, total, T, y)
        coli.coli_moe_norm_backward(n, total, T, y, None, dx, None, dw, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x2, r2, _ = _inputs(T, H, BF, BF, seed=seed + 10)
        x.copy_(x2), res.copy_(r2)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (total, y, dx, dw)]
        for t in (total, y, dx, dw):
            t.fill_(3.0)
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (total, y, dx, dw)))
