"""Cases, plain forms and calls of the layer library's norm, row and gradient operators.

Operators: the root-mean-square norm in front of the layer (with the residual's
addition, and codes for the prefill path) and its backward pass; a batch's rows
sorted by expert and the gradient of that; the experts' rows weighted and added
up per token and the gradient of that; the global norm of many gradients, and
clipping.  `run` computes each either with elementary torch operations in 32
bits (own = False) or through the library (own = True).
"""
import math

import numpy as np
import torch

own = False

# (hidden, inter), and (experts, top_k), of the layer shapes the library is tested and benchmarked on
SHAPES = ((256, 128), (2048, 512), (2048, 1024), (6144, 2048))
ROUTERS = ((8, 2), (64, 8), (256, 8), (160, 6))
LARGEST_NORM = 16384 * 6144
LARGEST_ROWS = 8192 * 8 * 6144


# ------------------------------------------------------------------ cases
def _norm(name, op, hidden, tokens, residual, fmt="none", weight="bf16", y=True, through=True):
    return dict(name=name, op=op, hidden=hidden, tokens=tokens, residual=residual, fmt=fmt,
                weight=weight, y=y, through=through)


def _rows(name, op, hidden, router, tokens, rows="bf16", out="bf16", beside=False, capacity=0.0):
    return dict(name=name, op=op, hidden=hidden, experts=router[0], top_k=router[1],
                tokens=tokens, rows=rows, out=out, beside=beside, capacity=capacity)


def _clip(name, hidden, inter, layers, adapters, rank, experts, share):
    return dict(name=name, op="clip", hidden=hidden, inter=inter, layers=layers,
                adapters=adapters, rank=rank, experts=experts, share=share)


def listed():
    return [
        # one decoded token in front of the router and the experts
        _norm("norm_1_token", "norm", 6144, 1, "bf16"),
        # a step of short prompts, fp32 residual stream, Q8_0 codes for the integer path
        _norm("norm_517_q8_0", "norm", 2048, 517, "f32", "q8_0"),
        # a long prompt, MXFP8 codes for the MX path
        _norm("norm_16384_mxfp8", "norm", 6144, 16384, "bf16", "mxfp8"),
        # a training step on a few short sequences, the first norm of a stack
        _norm("norm_backward_65", "norm_backward", 2048, 65, "none", through=False),
        # a training step on full sequences, fp32 residual stream
        _norm("norm_backward_8192", "norm_backward", 6144, 8192, "f32"),
        # a prompt's tokens laid out for the experts' products
        _rows("dispatch_16384", "dispatch", 2048, (256, 8), 16384),
        # a ragged micro-batch's gradient back to its tokens, the shared expert's beside it
        _rows("dispatch_backward_517", "dispatch_backward", 2048, (64, 8), 517, beside=True),
        # four verified tokens of a large layer, fp32 rows of its products
        _rows("combine_4", "combine", 6144, (256, 8), 4, rows="f32", beside=True),
        # a full batch's rows back to its tokens
        _rows("combine_8192", "combine", 6144, (256, 8), 8192),
        # a ragged training batch with a limit per expert, so that some pairs have no row
        _rows("combine_backward_2051", "combine_backward", 2048, (160, 6), 2051, capacity=1.25),
        # the gradients of one small layer's adapters and router
        _clip("clip_small", 256, 128, 1, 2, 8, 8, 0.5),
        # those of a stack of twelve large layers, as the adapters of many users train at once
        _clip("clip_stack", 6144, 2048, 12, 8, 64, 256, 0.1),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(("norm", "norm_backward", "dispatch", "dispatch_backward", "combine",
                     "combine_backward", "clip"))
    if op in ("norm", "norm_backward"):
        h = rng.choice((rng.choice(SHAPES)[0], 32 * log(1, 512)))
        most = LARGEST_NORM if op == "norm" else LARGEST_NORM // 2
        t = log(1, min(65536, most // h))
        fmt = rng.choice(("none", "q8_0", "mxfp8")) if op == "norm" else "none"
        c = _norm("", op, h, t, rng.choice(("none", "bf16", "f32")), fmt,
                  rng.choice(("bf16", "f32", "none")), fmt == "none" or rng.random() < 0.8,
                  rng.random() < 0.7)
    elif op == "clip":
        h, i = rng.choice(SHAPES)
        c = _clip("", h, i, log(1, 12), log(1, 8), 8 * rng.randrange(1, 9),
                  rng.choice(ROUTERS)[0], rng.choice((0.01, 0.5, 2.0)))
    else:
        router = rng.choice(ROUTERS)
        h = rng.choice((rng.choice(SHAPES)[0], 64 * log(1, 128)))
        t = log(1, min(65536, LARGEST_ROWS // (4 * h * router[1])))
        c = _rows("", op, h, router, t, rng.choice(("bf16", "f32")), rng.choice(("bf16", "f32")),
                  rng.random() < 0.5, rng.choice((0.0, 0.0, 1.0, 1.5)))
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


def _normal(g, *shape, std=1.0, dtype="bf16"):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(DTYPES[dtype])


def _prepare_norm(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 41)
    h, t, res = case["hidden"], case["tokens"], case["residual"]
    s = dict(case=case, weight=None, residual=None)
    if case["weight"] != "none":
        s["weight"] = (torch.randn(h, generator=g, device="cuda") * 0.2 + 1).to(DTYPES[case["weight"]])
    if case["op"] == "norm":
        s["x"] = _normal(g, t, h, std=0.7)
        if res != "none":
            # the stream that many layers have added to, with a few large channels
            s["residual"] = ((torch.randn(t, h, generator=g, device="cuda") * 3)
                             * (1 + 20 * (torch.rand(h, generator=g, device="cuda") < 0.002))
                             ).to(DTYPES[res])
    else:
        s["total"] = _normal(g, t, h, std=3.0, dtype="bf16" if res == "none" else res)
        s["dy"] = _normal(g, t, h, std=1e-2)
        # the gradient that reaches the stream past the layer
        s["d_total"] = (_normal(g, t, h, std=1e-2, dtype="bf16" if res == "none" else res)
                        if case["through"] else None)
    if own:
        _handles_norm(s)
    return s


def _handles_norm(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    t, h = c["tokens"], c["hidden"]
    new = lambda dtype, *shape: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s["norm"] = coli.Norm(h, s["weight"], EPS)
    if c["op"] == "norm":
        s["total"] = None if s["residual"] is None else torch.empty_like(s["residual"])
        s["y"] = new(torch.bfloat16, t, h) if c["y"] else None
        s["format"] = {"none": coli.COLI_NORM_PLAIN, "q8_0": coli.COLI_NORM_Q8_0,
                       "mxfp8": coli.COLI_NORM_MXFP8}[c["fmt"]]
        s["q"] = s["scales"] = None
        if c["fmt"] == "q8_0":
            s["q"], s["scales"] = new(torch.int8, t, h), new(torch.float16, t, h // 32)
        elif c["fmt"] == "mxfp8":
            s["q"], s["scales"] = new(torch.uint8, t, h), new(torch.uint8, t, h // 32)
        return
    s["dx"] = new(torch.bfloat16, t, h)
    s["d_residual"] = torch.empty_like(s["total"]) if c["residual"] == "f32" else None
    s["d_weight"] = None if s["weight"] is None else new(torch.float32, h)
    s["ws"] = coli.norm_workspace(s["norm"], t)


def _prepare_rows(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 53)
    h, e, k, t = (case[n] for n in ("hidden", "experts", "top_k", "tokens"))
    # a few hot experts; the routing weights are renormalised
    logits = _normal(g, t, e, dtype="f32") * 1.5 + _normal(g, e, dtype="f32") * 0.7
    best = logits.topk(k, dim=1)
    idx = best.indices.reshape(-1)
    s = dict(case=case, weights=torch.softmax(best.values, dim=1).reshape(-1).contiguous())
    order = torch.argsort(idx, stable=True)
    count = torch.bincount(idx, minlength=e)
    rank = torch.arange(t * k, device="cuda") - (count.cumsum(0) - count)[idx[order]]
    if case["capacity"]:
        most = max(1, int(case["capacity"] * t * k / e))
        s["n_rows"] = e * most
        pos = torch.where(rank < most, idx[order] * most + rank, -1)
    else:
        s["n_rows"] = t * k
        pos = torch.arange(t * k, device="cuda")
    # row of each pair (-1: none), and pair of each row (-1: none)
    s["pair_pos"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
    s["pair_pos"][order] = pos.to(torch.int32)
    table = torch.full((s["n_rows"] + 1,), -1, dtype=torch.int64, device="cuda")
    table[torch.where(pos >= 0, pos, s["n_rows"])] = order
    s["pair_of_row"] = table[:-1].contiguous()
    if case["op"] == "dispatch":
        s["x"] = _normal(g, t, h, dtype=case["rows"])
    else:
        s["rows"] = _normal(g, s["n_rows"], h, dtype=case["rows"])
        if case["op"] == "combine_backward":
            s["dy"] = _normal(g, t, h, std=1e-2, dtype=case["out"])
        else:
            s["beside"] = _normal(g, t, h, dtype=case["rows"]) if case["beside"] else None
    if case["op"] in ("dispatch", "combine_backward"):
        s["empty"] = torch.zeros(s["n_rows"], h, dtype=DTYPES[case["rows"]], device="cuda")
    if own:
        _handles_rows(s)
    return s


def _handles_rows(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    t, h = c["tokens"], c["hidden"]
    s["layer"] = coli.Layer(h, 64, c["experts"], 0, c["top_k"], coli.COLI_ROUTE_RENORM, None, None)
    s["route"] = coli.Route(s["layer"], t)
    s["route"].pair_pos.copy_(s["pair_pos"])
    s["route"].topk_w.copy_(s["weights"])
    if c["op"] in ("combine", "dispatch_backward"):
        s["y"] = torch.empty(t, h, dtype=DTYPES[c["out"]], device="cuda")
    elif c["op"] == "combine_backward":
        s["d_topk_w"] = torch.empty(t * c["top_k"], dtype=torch.float32, device="cuda")


def _prepare_clip(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 61)
    h, i, n, r, e = (case[k] for k in ("hidden", "inter", "adapters", "rank", "experts"))
    # a layer's adapters of gate, up and down; its router (bf16) and a gate of odd size; its norm
    shapes = [(n, r, h), (n, i, r), (n, r, h), (n, i, r), (n, r, i), (n, h, r), (e, h), (h,), (h + 1,)]
    s = dict(case=case, grads=[], at=[])
    total = 0
    for _ in range(case["layers"]):
        for j, shape in enumerate(shapes):
            s["grads"].append(_normal(g, *shape, std=1e-3 * (1 + j), dtype="bf16" if j == 6 else "f32"))
            s["at"].append(total)
            total += (s["grads"][-1].numel() + 63) // 64 * 64
    # one flat buffer takes all clipped gradients, each from a multiple of 64 on
    s["flat"] = torch.zeros(total, dtype=torch.float32, device="cuda")
    expect = math.sqrt(sum((1e-3 * (1 + j % len(shapes))) ** 2 * t.numel()
                           for j, t in enumerate(s["grads"])))
    s["max_norm"] = case["share"] * expect
    if own:
        _handles_clip(s)
    return s


def _handles_clip(s):
    import int4_routed_expert_router_amd as coli
    out = [s["flat"][a:a + t.numel()] for a, t in zip(s["at"], s["grads"])]
    s["gradients"] = coli.Gradients(s["grads"], out)
    s["norm"] = torch.empty(2, dtype=torch.float32, device="cuda")
    s["ws"] = coli.clip_workspace()


def prepare(case, seed):
    if case["op"] in ("norm", "norm_backward"):
        return _prepare_norm(case, seed)
    if case["op"] == "clip":
        return _prepare_clip(case, seed)
    return _prepare_rows(case, seed)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _RUN_OWN[op](s)
    return _RUN_PLAIN[op](s)


def _out_norm(c, y, q, scales, total):
    """MXFP8 as its E4M3 and E8M0 values, Q8_0 as code times scale (fp16)."""
    r = {} if y is None else {"y": y}
    if c["fmt"] == "mxfp8":
        r["q"], r["scales"] = q.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu)
    elif c["fmt"] == "q8_0":
        r["q"] = q.view(-1, 32) * scales.view(-1, 1)
    return r if total is None else {**r, "total": total}


def _own_norm(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    coli.coli_moe_norm(s["norm"], s["x"], s["residual"], s["total"], c["tokens"], s["y"],
                       s["format"], s["q"], s["scales"])
    return _out_norm(c, s["y"], s["q"], s["scales"], s["total"])


def _own_norm_backward(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_norm_backward(s["norm"], s["total"], s["case"]["tokens"], s["dy"], s["d_total"],
                                s["dx"], s["d_residual"], s["d_weight"], s["ws"])
    return {"dx": s["dx"], "d_residual": s["d_residual"], "d_weight": s["d_weight"]}


def _own_dispatch(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_dispatch(s["layer"], s["route"], s["x"], s["case"]["tokens"], s["empty"])
    return {"rows": s["empty"]}


def _own_dispatch_backward(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_dispatch_backward(s["layer"], s["route"], s["rows"], s["beside"],
                                    s["case"]["tokens"], s["y"])
    return {"dx": s["y"]}


def _own_combine(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_combine(s["layer"], s["route"], s["rows"], s["beside"], s["case"]["tokens"],
                          s["y"])
    return {"y": s["y"]}


def _own_combine_backward(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_combine_backward(s["layer"], s["route"], s["rows"], s["dy"],
                                   s["case"]["tokens"], s["empty"], s["d_topk_w"])
    return {"d_rows": s["empty"], "d_topk_w": s["d_topk_w"]}


def _own_clip(s):
    import int4_routed_expert_router_amd as coli
    coli.coli_moe_clip_gradients(s["gradients"], s["max_norm"], s["norm"], s["ws"])
    return {"norm": s["norm"], "grads": s["flat"]}


# -------------------------------------------------- plain forms (32 bits)
def _plain_norm(s):
    c = s["case"]
    total = s["x"] if s["residual"] is None else (s["residual"].float() + s["x"].float()).to(
        s["residual"].dtype)
    f = total.float()
    y = f * torch.rsqrt(f.square().mean(dim=1, keepdim=True) + EPS)
    if s["weight"] is not None:
        y = y * s["weight"].float()
    y = y.to(torch.bfloat16)
    q = scales = None
    if c["fmt"] == "q8_0":
        v = y.float().view(-1, 32)
        d = v.abs().amax(dim=1, keepdim=True) / 127.0
        r = v / torch.where(d > 0, d, 1.0)
        q = (torch.sign(r) * torch.floor(r.abs() + 0.5)).clamp(-127, 127).to(torch.int8)
        scales = d.to(torch.float16)
    elif c["fmt"] == "mxfp8":
        v = y.float().view(-1, 32)
        a = v.abs().amax(dim=1, keepdim=True)
        e = torch.where(a > 0, torch.frexp(a)[1] + (126 - 8), 0).clamp(0, 254)
        q = (v * torch.exp2((127 - e).float())).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        q, scales = q.view(torch.uint8).view(y.shape), e.to(torch.uint8).view(y.shape[0], -1)
    return _out_norm(c, y if c["y"] else None, q, scales,
                     None if s["residual"] is None else total)


def _plain_norm_backward(s):
    f, dy = s["total"].float(), s["dy"].float()
    rstd = torch.rsqrt(f.square().mean(dim=1, keepdim=True) + EPS)
    hat = f * rstd
    dn = dy if s["weight"] is None else dy * s["weight"].float()
    d = rstd * (dn - hat * (dn * hat).mean(dim=1, keepdim=True))
    if s["d_total"] is not None:
        d = d + s["d_total"].float()
    return {"dx": d.to(torch.bfloat16),
            "d_residual": d if s["case"]["residual"] == "f32" else None,
            "d_weight": None if s["weight"] is None else (dy * hat).sum(dim=0)}


def _plain_dispatch(s):
    pair = s["pair_of_row"]
    rows = s["x"][pair.clamp(min=0) // s["case"]["top_k"]]
    return {"rows": torch.where((pair >= 0)[:, None], rows, s["empty"])}


def _of_pairs(s):
    """The rows of every token's pairs [T, k, H] in 32 bits; zeros where a pair has none."""
    c = s["case"]
    pos = s["pair_pos"].to(torch.int64)
    r = torch.where((pos >= 0)[:, None], s["rows"][pos.clamp(min=0)], 0.0)
    return r.float().view(c["tokens"], c["top_k"], c["hidden"])


def _plain_dispatch_backward(s):
    d = _of_pairs(s).sum(dim=1)
    d = d if s["beside"] is None else d + s["beside"].float()
    return {"dx": d.to(DTYPES[s["case"]["out"]])}


def _plain_combine(s):
    c = s["case"]
    y = (_of_pairs(s) * s["weights"].view(c["tokens"], c["top_k"], 1)).sum(dim=1)
    y = y if s["beside"] is None else y + s["beside"].float()
    return {"y": y.to(DTYPES[c["out"]])}


def _plain_combine_backward(s):
    c, pair = s["case"], s["pair_of_row"]
    d_w = (_of_pairs(s) * s["dy"].float()[:, None, :]).sum(dim=2).reshape(-1)
    at = pair.clamp(min=0)
    d = s["dy"].float()[at // c["top_k"]] * s["weights"][at][:, None]
    d = torch.where((pair >= 0)[:, None], d.to(DTYPES[c["rows"]]), s["empty"])
    return {"d_rows": d, "d_topk_w": d_w}


def _plain_clip(s):
    norm = torch.stack([t.double().square().sum() for t in s["grads"]]).sum().sqrt().float()
    factor = torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    flat = torch.cat([torch.nn.functional.pad((t.float() * factor).reshape(-1), (0, -t.numel() % 64))
                      for t in s["grads"]])
    return {"norm": torch.stack((norm, factor)), "grads": flat}


_RUN_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "dispatch": _own_dispatch,
            "dispatch_backward": _own_dispatch_backward, "combine": _own_combine,
            "combine_backward": _own_combine_backward, "clip": _own_clip}
_RUN_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward,
              "dispatch": _plain_dispatch, "dispatch_backward": _plain_dispatch_backward,
              "combine": _plain_combine, "combine_backward": _plain_combine_backward,
              "clip": _plain_clip}


# ------------------------------------------------------------------ floors
def work(case):
    size = {"none": 0, "bf16": 2, "f32": 4}
    if case["op"] == "clip":
        h, i, n, r, e = (case[k] for k in ("hidden", "inter", "adapters", "rank", "experts"))
        wide = case["layers"] * (3 * n * r * (h + i) + 2 * h + 1)
        half = case["layers"] * e * h
        return {"bytes": 8 * wide + 6 * half, "flops": 3 * (wide + half)}
    h, t = case["hidden"], case["tokens"]
    if case["op"] == "norm":
        a = 2 + 2 * size[case["residual"]] + (2 if case["y"] else 0)
        a += {"none": 0, "q8_0": 1 + 2 / 32, "mxfp8": 1 + 1 / 32}[case["fmt"]]
        return {"bytes": int(t * h * a + h * size[case["weight"]]), "flops": 8 * t * h}
    if case["op"] == "norm_backward":
        stream = max(2, size[case["residual"]])
        a = stream + 2 + (stream if case["through"] else 0) + 2
        a += 4 if case["residual"] == "f32" else 0
        return {"bytes": int(t * h * a + h * (size[case["weight"]] + 4)), "flops": 12 * t * h}
    k, rows, out = case["top_k"], size[case["rows"]], size[case["out"]]
    p = t * k
    if case["op"] == "dispatch":
        return {"bytes": int(h * (t + p) * rows + 4 * p), "flops": p * h}
    if case["op"] == "combine_backward":
        return {"bytes": int(h * (2 * p * rows + t * out) + 12 * p), "flops": 3 * p * h}
    beside = rows if case["beside"] else 0
    return {"bytes": int(h * (p * rows + t * (out + beside)) + 8 * p), "flops": 2 * p * h}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "norm_backward":
        return _exact_norm_backward(s)
    if case["op"] == "clip":
        return _exact_clip(s)
    return _exact_rows(s)


def _exact_norm(s):
    """E4M3 codes' places take what is rounded to them, before the rounding; Q8_0's, whose
    output is in 16 bits, what the codes stand for."""
    c = s["case"]
    v, total = s["x"].double(), None
    if s["residual"] is not None:
        total = v + s["residual"].double()
        # the norm is that of the stored sum
        v = total if c["residual"] == "f32" else total.float().to(torch.bfloat16).double()
    y = v / torch.sqrt(torch.sum(v * v, dim=1, keepdim=True) / c["hidden"] + EPS)
    if s["weight"] is not None:
        y *= s["weight"].double()
    r = {"y": y} if c["y"] else {}
    if c["fmt"] == "q8_0":
        v = y.float().to(torch.bfloat16).double().view(-1, 32)
        d = v.abs().max(dim=1, keepdim=True).values / 127
        code = torch.trunc(v / d.clamp(min=1e-300) + torch.where(v < 0, -0.5, 0.5))
        r["q"] = code * d.to(torch.float16).double()
    elif c["fmt"] == "mxfp8":
        block = y.view(-1, 32)
        top = block.float().to(torch.bfloat16).double().abs().max(dim=1, keepdim=True).values
        two = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-30))) - 8)
        r["q"], r["scales"] = (block / two).view(y.shape), two.view(c["tokens"], -1)
    if total is not None:
        r["total"] = total
    return r


def _exact_norm_backward(s):
    """Through autograd of the norm as it is defined, some rows at a time."""
    c = s["case"]
    t, h = c["tokens"], c["hidden"]
    d = torch.empty(t, h, dtype=torch.float64, device="cuda")
    w = torch.ones(h, dtype=torch.float64, device="cuda") if s["weight"] is None else s["weight"].double()
    dw = torch.zeros_like(w)
    for at in torch.arange(t, device="cuda").split(2048):
        v = s["total"][at].double().requires_grad_(True)
        u = w.clone().requires_grad_(True)
        y = u * v / torch.sqrt(torch.sum(v * v, dim=1, keepdim=True) / h + EPS)
        a, b = torch.autograd.grad((y * s["dy"][at].double()).sum(), (v, u))
        d[at] = a if s["d_total"] is None else a + s["d_total"][at].double()
        dw += b
    return {"dx": d, "d_residual": d if c["residual"] == "f32" else None,
            "d_weight": None if s["weight"] is None else dw}


def _exact_rows(s):
    c = s["case"]
    t, h, k = c["tokens"], c["hidden"], c["top_k"]
    pos = s["pair_pos"].view(t, k).to(torch.int64)
    has = pos >= 0
    if c["op"] == "dispatch":
        rows = s["empty"].double()
        for j in range(k):
            rows[pos[has[:, j], j]] = s["x"][has[:, j]].double()
        return {"rows": rows}
    w = s["weights"].view(t, k).double()
    if c["op"] == "combine_backward":
        dy, rows = s["dy"].double(), s["empty"].double()
        d_w = torch.zeros(t, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            at, to = has[:, j], pos[has[:, j], j]
            rows[to] = dy[at] * w[at, j, None]
            d_w[at, j] = torch.sum(dy[at] * s["rows"][to].double(), dim=1)
        return {"d_rows": rows, "d_topk_w": d_w.view(-1)}
    y = torch.zeros(t, h, dtype=torch.float64, device="cuda")
    if s["beside"] is not None:
        y += s["beside"].double()
    for j in range(k):
        at = has[:, j]
        part = s["rows"][pos[at, j]].double()
        y[at] += part * w[at, j, None] if c["op"] == "combine" else part
    return {"y" if c["op"] == "combine" else "dx": y}


def _exact_clip(s):
    norm = math.sqrt(sum(float(torch.dot(t.double().view(-1), t.double().view(-1)))
                         for t in s["grads"]))
    factor = min(1.0, s["max_norm"] / norm)
    flat = torch.zeros(s["flat"].shape, dtype=torch.float64, device="cuda")
    for a, t in zip(s["at"], s["grads"]):
        flat[a:a + t.numel()] = factor * t.double().view(-1)
    return {"norm": torch.tensor([norm, factor], dtype=torch.float64), "grads": flat}
