"""The norm over many gradients, and clipping, against float64.

Tolerances.  Squares are exact in 64 bits and summed there; the norm is rounded
to fp32 once: half a step 2^-24 (and 1e-12 for the sums).  The factor is one
fp32 division of what is reported, and a clipped value one fp32 product and one
rounding: equal bits."""
import numpy as np
import pytest
import torch

import int4_routed_expert_router_amd as coli

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def _make(sizes, seed=0, out="same", shift=False):
    """Gradients and their outputs; `shift`: at any element instead of at 16 bytes."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    grads, outs = [], []
    for i, n in enumerate(sizes):
        dt = (F32, BF, F32, F32)[(i + seed) % 4]
        a = (1 + i) % 9 if shift else 0
        grads.append((torch.randn(n + a, generator=g, device="cuda") * 10 ** (i % 3 - 1)).to(dt)[a:])
        if out == "same":
            outs.append(grads[-1])
        else:
            od = (F32, BF, BF)[(i + seed) % 3] if out == "mixed" else dt
            b = (3 * i) % 8 if shift else 0
            outs.append(torch.full((n + b,), 7.0, dtype=od, device="cuda")[b:])
    return grads, outs


def _clip(grads, outs, max_norm, ws=None):
    p = coli.Gradients(grads, outs)
    norm = torch.full((2,), 7.0, device="cuda")
    if ws is None:
        ws = coli.clip_workspace()
        ws.fill_(0xff)
    coli.coli_moe_clip_gradients(p, max_norm, norm, ws)
    torch.cuda.synchronize()
    return norm.cpu().numpy()


def _check(before, outs, norm, max_norm):
    ref = float(np.sqrt(sum(float(t.double().square().sum()) for t in before)))
    assert abs(norm[0] - ref) <= ref * (2.0 ** -24 + 1e-12)
    want = np.float32(max_norm) / norm[0] if norm[0] > np.float32(max_norm) else np.float32(1)
    assert norm[1] == want
    f = torch.tensor(norm[1], device="cuda")
    for b, o in zip(before, outs):
        assert torch.equal(o, (b.float() * f).to(o.dtype))
    return ref


SIZES = [[1], [7], [8], [2048], [2049, 1, 5, 4097], [100, 3, 0, 31, 70000, 8, 0, 2047, 6144 * 7],
         [5] * 300, [1 << 20, 3, 12345, 1 << 18]]


@pytest.mark.parametrize("share", [0.01, 0.999, 1.5])
@pytest.mark.parametrize("shift", [False, True])
@pytest.mark.parametrize("out", ["same", "other", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "%dx%d" % (len(s), max(s)))
def test_clip(sizes, out, shift, share):
    grads, outs = _make(sizes, len(sizes), out, shift)
    before = [t.clone() for t in grads]
    size = float(np.sqrt(sum(float(t.double().square().sum()) for t in before)))
    norm = _clip(grads, outs, share * size)
    _check(before, outs, norm, share * size)
    if out != "same":
        assert all(torch.equal(a, b) for a, b in zip(before, grads))


def test_neighbours_stay():
    """Values in front of and behind the gradients in the same buffer."""
    buf = torch.ones(5000, device="cuda")
    grads = [buf[3:1001], buf[1002:1003], buf[1010:4990]]
    norm = _clip(grads, grads, 0.5)
    keep = torch.ones(5000, dtype=torch.bool)
    keep[3:1001] = keep[1002:1003] = keep[1010:4990] = False
    b = buf.cpu()
    assert (b[keep] == 1).all() and (b[~keep] == torch.tensor(norm[1])).all()


def test_nothing_to_clip():
    e = torch.empty(0, device="cuda")
    assert _clip([e], [e], 1.0).tolist() == [0.0, 1.0]
    z = torch.zeros(1000, device="cuda")
    assert _clip([z], [z], 0.0).tolist() == [0.0, 1.0]
    t = torch.ones(4, device="cuda")
    assert _clip([t], [t], 0.0).tolist() == [2.0, 0.0] and (t == 0).all()
    t = torch.ones(4, device="cuda")
    assert _clip([t], [t], float("inf")).tolist() == [2.0, 1.0] and (t == 1).all()


@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_squares_outside_fp32(scale):
    t = torch.full((3000,), scale, device="cuda")
    u = torch.full((1000,), scale, device="cuda").to(BF)
    before = [t.clone(), u.clone()]
    _check(before, [t, u], _clip([t, u], [t, u], scale), scale)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_not_finite(bad):
    grads, outs = _make([1000, 33], 1, "other")
    grads[1][7] = bad
    norm = _clip(grads, outs, 0.1)
    assert not np.isfinite(norm[0]) and norm[1] == 1.0
    for g, o in zip(grads, outs):
        assert torch.equal(g.nan_to_num(7, 8, 9), o.nan_to_num(7, 8, 9))


def test_norm_past_fp32():
    t = torch.full((200,), 3e38, device="cuda")
    norm = _clip([t], [t], 1.0)
    assert norm[0] == np.inf and norm[1] == 1.0 and (t == 3e38).all()


def test_repeated_captured_and_streams():
    grads, outs = _make([70000, 513, 2048, 9], 2, "other")
    p, norm, ws = coli.Gradients(grads, outs), torch.empty(2, device="cuda"), coli.clip_workspace()
    coli.coli_moe_clip_gradients(p, 3.0, norm, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        coli.coli_moe_clip_gradients(p, 3.0, norm, ws)
    for i in range(3):
        for g in grads:
            g.mul_(1.7)
        want = _clip(grads, outs, 3.0)
        kept = [o.clone() for o in outs]
        for o in outs:
            o.fill_(5.0)
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(norm.cpu().numpy(), want)
        assert all(torch.equal(a, b) for a, b in zip(kept, outs))
        s = torch.cuda.Stream()
        coli.coli_moe_clip_gradients(p, 3.0, norm, ws, stream=s)
        s.synchronize()
        assert np.array_equal(norm.cpu().numpy(), want)


@pytest.mark.parametrize("out,shift", [("same", False), ("other", True), ("mixed", False),
                                       ("mixed", True)])
@pytest.mark.parametrize("n", [20000003, 90000001])
def test_large(n, out, shift):
    """Gradients of 80 and 360 MB and more, which go past the caches."""
    sizes = [n, 5, n // 3, 100000]
    grads, outs = _make(sizes, 0, out, shift)
    before = [t.clone() for t in grads]
    size = float(np.sqrt(sum(float(t.double().square().sum()) for t in before)))
    _check(before, outs, _clip(grads, outs, 1.5 * size), 1.5 * size)  # nothing to clip
    _check(before, outs, _clip(grads, outs, 0.3 * size), 0.3 * size)


def test_largest():
    """A gradient of over 2^31 values, in bf16, and many beside it."""
    big = torch.full(((1 << 31) + 77,), 0.5, dtype=BF, device="cuda")
    small = [torch.ones(1000 + i, device="cuda") for i in range(2000)]
    want = np.sqrt(big.numel() * 0.25 + sum(t.numel() for t in small))
    norm = _clip([big] + small, None, want / 2)
    assert abs(norm[0] - want) <= want * (2.0 ** -24 + 1e-12)
    f = torch.tensor(norm[1], device="cuda")
    v = (0.5 * f).to(BF)
    for a in range(0, big.numel(), 1 << 28):
        assert (big[a:a + (1 << 28)] == v).all()
    assert all((t == f).all() for t in small)
