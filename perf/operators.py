"""Cases, plain forms and calls of the layer library's training and adapter operators.

Operators: a projection of one expert matrix with the low-rank adapters of many
requests beside it, its backward pass, the router's balance loss with per-expert
counts, and the gradient of the route.  `run` computes each either with elementary
torch operations in 32 bits (own = False) or through the library (own = True).
"""
import math

import numpy as np
import torch

own = False

# (hidden, inter) of the layer shapes the library is tested and benchmarked on
SHAPES = ((256, 128), (2048, 512), (2048, 1024), (6144, 2048))
FORMATS = ("int4", "int8", "mxfp4")


# ------------------------------------------------------------------ cases
def _project(name, fmt, shape, matrix, tokens, requests, adapters, rank, out="bf16", tail=0,
             op="project"):
    return dict(name=name, op=op, fmt=fmt, hidden=shape[0], inter=shape[1], matrix=matrix,
                tokens=tokens, requests=requests, adapters=adapters, rank=rank, out=out, tail=tail)


def _router(name, op, experts, top_k, tokens, sequences, sigmoid, renorm, masked, tail=0,
            balance=True, weights=True):
    return dict(name=name, op=op, experts=experts, top_k=top_k, tokens=tokens,
                sequences=sequences, sigmoid=sigmoid, renorm=renorm, masked=masked, tail=tail,
                balance=balance, weights=weights)


def listed():
    return [
        # one user decoding one token through the shared expert's gate
        _project("project_1_token", "int4", SHAPES[3], 0, 1, 1, 4, 16),
        # a decode batch: sixteen users, eight adapters, one token each; int8 codes, fp32 result
        _project("project_16_users", "int8", SHAPES[1], 1, 16, 16, 8, 32, out="f32"),
        # a full decode batch of MXFP4 weights with as many adapters as half the users
        _project("project_64_users", "mxfp4", SHAPES[3], 2, 64, 64, 32, 64),
        # a step that mixes short prompts of several users, odd lengths, padding rows behind
        _project("project_mixed_517", "int4", SHAPES[2], 2, 517, 37, 16, 24, out="f32", tail=5),
        # long prompts of a few users
        _project("project_prompts_8192", "int4", SHAPES[3], 0, 8192, 5, 4, 64),
        # a training step on a few short sequences
        _project("project_backward_65", "int4", SHAPES[2], 0, 65, 3, 2, 8,
                 op="project_backward"),
        # a training step of two adapters on full sequences
        _project("project_backward_8192", "int4", SHAPES[3], 2, 8192, 4, 2, 64,
                 op="project_backward"),
        # the smallest layer's four tokens
        _router("balance_4", "balance", 8, 2, 4, 1, False, False, False),
        # a ragged micro-batch with padded tokens, sigmoid routing
        _router("balance_ragged_2051", "balance", 256, 8, 2051, 7, True, True, True, tail=3),
        # a full batch, one sequence
        _router("balance_65536", "balance", 256, 8, 65536, 1, False, False, False),
        # the router's gradient on a small micro-batch of a softmax layer
        _router("route_backward_513", "route_backward", 64, 8, 513, 3, False, False, True),
        # and on a full batch of a sigmoid layer
        _router("route_backward_65536", "route_backward", 256, 8, 65536, 16, True, True, False),
    ]


def draw(rng):
    log = lambda lo, hi: int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))  # noqa: E731
    op = rng.choice(("project", "project", "project_backward", "balance", "route_backward"))
    if op in ("project", "project_backward"):
        tokens = log(1, 8000)
        requests = min(tokens, log(1, 64)) if tokens > 64 or rng.random() < 0.4 else tokens
        c = _project("", rng.choice(FORMATS), rng.choice(SHAPES), rng.randrange(3), tokens,
                     requests, log(1, 4 if tokens > 2048 else 32), rng.randrange(1, 65),
                     out=rng.choice(("bf16", "f32")) if op == "project" else "bf16",
                     tail=rng.choice((0, 0, 1, 7)) if tokens > requests + 8 else 0, op=op)
    else:
        tokens, (experts, top_k) = log(1, 60000), rng.choice(((8, 2), (64, 8), (256, 8), (160, 6)))
        c = _router("", op, experts, top_k, tokens, min(tokens, log(1, 40)), rng.random() < 0.5,
                    rng.random() < 0.5, rng.random() < 0.5,
                    tail=rng.choice((0, 0, 3)) if tokens > 64 else 0,
                    balance=op == "balance" or rng.random() < 0.7)
        c["weights"] = op == "balance" or not c["balance"] or rng.random() < 0.7
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def _dims(case):
    """Rows and columns (N, K) of the case's matrix."""
    h, i = case["hidden"], case["inter"]
    return (h, i) if case["matrix"] == 2 else (i, h)


def _cuts(rng, total, parts):
    """Offsets that part `total` rows at random, the first at zero; some parts may be empty."""
    if parts == total:
        return np.arange(parts + 1, dtype=np.int32)
    inner = np.sort(rng.integers(0, total + 1, parts - 1))
    return np.concatenate(([0], inner, [total])).astype(np.int32)


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _prepare_project(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    rng = np.random.default_rng(seed + 1)
    h, i, t, r, na = (case[n] for n in ("hidden", "inter", "tokens", "rank", "adapters"))
    n, k = _dims(case)
    # the container of one routed and the shared expert: gate, up, down each
    bits, group = (8 if case["fmt"] == "int8" else 4), (32 if case["fmt"] == "mxfp4" else 64)
    codes = torch.randint(0, 256, (2 * 3 * h * i * bits // 8,), generator=g, device="cuda",
                          dtype=torch.uint8)
    ns = 2 * 3 * h * i // group
    if case["fmt"] == "mxfp4":
        scales = torch.randint(118, 123, (ns,), generator=g, device="cuda", dtype=torch.uint8)
    else:
        scales = (_normal(g, ns).abs() * (0.02 / 16 if bits == 8 else 0.02)).to(torch.float16)
    stride = (r + 7) // 8 * 8  # adapters of several ranks share one table of this width
    rank = rng.integers(1, r + 1, na)
    rank[::2] = r
    offsets = _cuts(rng, t - case["tail"], case["requests"])
    # every third request without an adapter where there are several
    adapter = rng.permutation(case["requests"]) % na
    if case["requests"] > 2:
        adapter[::3] = -1
    s = dict(
        case=case, codes=codes, scales=scales,
        x=_normal(g, t, k).to(torch.bfloat16),
        a=_normal(g, na, stride, k, std=k ** -0.5).to(torch.bfloat16),
        b=_normal(g, na, n, stride, std=0.1).to(torch.bfloat16),
        rank=torch.from_numpy(rank.astype(np.int32)).cuda(),
        scale=torch.from_numpy(rng.uniform(0.5, 4.0, na).astype(np.float32)).cuda(),
        offsets=torch.from_numpy(offsets).cuda(),
        adapter=torch.from_numpy(adapter.astype(np.int32)).cuda())
    if case["op"] == "project_backward":
        s["dy"] = _normal(g, t, n, std=1e-2).to(torch.bfloat16)
    if own:
        _handles_project(s)
    return s


def _handles_project(s):
    import int4_routed_expert_router_amd as coli
    case = s["case"]
    n, k = _dims(case)
    t, backward = case["tokens"], case["op"] == "project_backward"
    s["layer"] = coli.Layer(case["hidden"], case["inter"], 1, 1, 1, 0, s["codes"], s["scales"],
                            int8=case["fmt"] == "int8", mxfp4=case["fmt"] == "mxfp4")
    s["adapters"] = coli.Adapters(s["a"], s["b"], s["rank"], s["scale"])
    s["requests"] = coli.Requests(s["offsets"], s["adapter"])
    s["ws"] = coli.project_workspace(s["layer"], case["matrix"], s["adapters"], t, backward)
    if backward:
        s["dx"] = torch.empty(t, k, dtype=torch.bfloat16, device="cuda")
        s["da"] = torch.empty(s["a"].shape, dtype=torch.float32, device="cuda")
        s["db"] = torch.empty(s["b"].shape, dtype=torch.float32, device="cuda")
    else:
        f32 = case["out"] == "f32"
        s["y"] = torch.empty(t, n, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
        s["y_dtype"] = coli.COLI_OUT_F32 if f32 else coli.COLI_OUT_BF16


def _prepare_router(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    rng = np.random.default_rng(seed + 2)
    e, k, t, ns = (case[n] for n in ("experts", "top_k", "tokens", "sequences"))
    # a few hot experts, as a router in training has them
    logits = _normal(g, t, e) * 1.5 + _normal(g, e) * 0.7
    s = dict(case=case, logits=logits,
             idx=logits.topk(k, dim=1).indices.to(torch.int32).reshape(-1),
             offsets=torch.from_numpy(_cuts(rng, t - case["tail"], ns)).cuda(), valid=None)
    if case["masked"]:
        s["valid"] = (torch.rand(t, generator=g, device="cuda") < 0.85).to(torch.uint8)
    if case["op"] == "route_backward":
        s["d_w"] = _normal(g, t * k, std=1e-2) if case["weights"] else None
        s["d_loss"] = torch.rand(2, generator=g, device="cuda") * 0.02 + 0.01
        # what the forward pass left: choices and valid tokens of each sequence
        seq = _row_of(s["offsets"], t)
        live = seq >= 0
        if case["masked"]:
            live &= s["valid"] != 0
        sel = seq[live].to(torch.int64)
        s["tokens"] = torch.bincount(sel, minlength=ns).to(torch.int32)
        flat = (sel[:, None] * e + s["idx"].view(t, k)[live].to(torch.int64)).reshape(-1)
        s["counts"] = torch.bincount(flat, minlength=ns * e).to(torch.int32).view(ns, e)
        s["totals"] = torch.stack((s["tokens"].sum(), (s["tokens"] > 0).sum())).to(torch.int32)
    if own:
        _handles_router(s)
    return s


def _handles_router(s):
    import int4_routed_expert_router_amd as coli
    case = s["case"]
    t = case["tokens"]
    flags = coli.COLI_ROUTE_SIGMOID if case["sigmoid"] else coli.COLI_ROUTE_SOFTMAX
    if case["renorm"]:
        flags |= coli.COLI_ROUTE_RENORM
    s["layer"] = coli.Layer(64, 64, case["experts"], 0, case["top_k"], flags, None, None)
    s["balance"] = coli.Balance(s["layer"], case["sequences"], s["offsets"], s["valid"])
    if case["op"] == "balance":
        s["ws"] = coli.balance_workspace(s["layer"], t, case["sequences"])
    else:
        for n in ("counts", "tokens", "totals"):
            getattr(s["balance"], n).copy_(s[n])
        s["d_logits"] = torch.empty_like(s["logits"])


def prepare(case, seed):
    if case["op"] in ("project", "project_backward"):
        return _prepare_project(case, seed)
    return _prepare_router(case, seed)


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _RUN_OWN[op](s)
    return _RUN_PLAIN[op](s)


def _own_project(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    coli.coli_moe_project(s["layer"], 1, c["matrix"], s["adapters"], s["requests"], s["x"],
                          c["tokens"], s["y"], s["y_dtype"], s["ws"])
    return {"y": s["y"]}


def _own_project_backward(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    coli.coli_moe_project_backward(s["layer"], 1, c["matrix"], s["adapters"], s["requests"],
                                   s["x"], s["dy"], c["tokens"], s["dx"], s["da"], s["db"],
                                   s["ws"])
    return {"dx": s["dx"], "da": s["da"], "db": s["db"]}


def _own_balance(s):
    import int4_routed_expert_router_amd as coli
    b = s["balance"]
    coli.coli_moe_balance_loss(s["layer"], s["logits"], s["idx"], s["case"]["tokens"], b, s["ws"])
    return {"loss": b.loss, "counts": b.counts, "mean_prob": b.mean_prob, "tokens": b.tokens}


def _own_route_backward(s):
    import int4_routed_expert_router_amd as coli
    c = s["case"]
    with_loss = c["balance"]
    coli.coli_moe_route_backward(s["layer"], s["logits"], s["idx"], c["tokens"], s["d_w"],
                                 s["balance"] if with_loss else None,
                                 s["d_loss"] if with_loss else None, s["d_logits"])
    return {"d_logits": s["d_logits"]}


# -------------------------------------------------- plain forms (32 bits)
def _row_of(offsets, t):
    """The part of each row, -1 for rows before the first and behind the last."""
    at = torch.arange(t, device="cuda", dtype=torch.int32)
    part = torch.searchsorted(offsets, at, right=True) - 1
    return torch.where((part >= 0) & (part < offsets.numel() - 1), part, -1)


def _weight(s):
    """The shared expert's matrix [N, K] as the values its codes and scales stand for."""
    c = s["case"]
    n, k = _dims(c)
    size, at = c["hidden"] * c["inter"], (3 + c["matrix"]) * c["hidden"] * c["inter"]
    if c["fmt"] == "int8":
        q = s["codes"][at:at + size].view(torch.int8).float()
    else:
        byte = s["codes"][at // 2:(at + size) // 2]
        nib = torch.stack((byte & 15, byte >> 4), dim=-1).reshape(-1).to(torch.int64)
        if c["fmt"] == "int4":
            q = (nib - 16 * (nib > 7)).float()
        else:
            value = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda", dtype=torch.float32)
            q = value[nib & 7] * (1 - 2 * (nib >> 3)).float()
    group = 32 if c["fmt"] == "mxfp4" else 64
    sc = s["scales"][at // group:(at + size) // group]
    sc = torch.exp2(sc.float() - 127) if c["fmt"] == "mxfp4" else sc.float()
    return (q.view(-1, group) * sc[:, None]).view(n, k)


def _tables(s):
    """All adapters side by side: A [n*R, K], B [N, n*R], and the factor of each (row, column):
    the adapter's scale in the row's own adapter's columns up to its rank, else zero."""
    a, b = s["a"].float(), s["b"].float()
    na, width, k = a.shape
    keep = torch.arange(width, device="cuda")[None, :] < s["rank"][:, None]
    a = torch.where(keep[:, :, None], a, 0.0).reshape(na * width, k)
    b = torch.where(keep[:, None, :], b, 0.0).permute(1, 0, 2).reshape(-1, na * width)
    part = _row_of(s["offsets"], s["case"]["tokens"])
    mine = torch.where(part >= 0, s["adapter"].to(torch.int64)[part.clamp(min=0)], -1)
    hot = (mine[:, None] == torch.arange(na, device="cuda")[None, :]).float() * s["scale"]
    return a, b, hot.repeat_interleave(width, dim=1)


def _plain_project(s):
    a, b, hot = _tables(s)
    x = s["x"].float()
    y = x @ _weight(s).t() + ((x @ a.t()) * hot) @ b.t()
    return {"y": y if s["case"]["out"] == "f32" else y.to(torch.bfloat16)}


def _plain_project_backward(s):
    a, b, hot = _tables(s)
    x, dy = s["x"].float(), s["dy"].float()
    v = (dy @ b) * hot
    u = (x @ a.t()) * hot
    na, width, k = s["a"].shape
    return {"dx": (dy @ _weight(s) + v @ a).to(torch.bfloat16),
            "da": (v.t() @ x).view(na, width, k),
            "db": (dy.t() @ u).view(-1, na, width).permute(1, 0, 2).contiguous()}


def _live(s):
    """Each row's sequence, and whether the row counts."""
    seq = _row_of(s["offsets"], s["case"]["tokens"])
    live = seq >= 0
    if s["valid"] is not None:
        live = live & (s["valid"] != 0)
    return seq, live


def _probs(s):
    l = s["logits"]
    score = torch.nn.functional.logsigmoid(l) if s["case"]["sigmoid"] else l
    e = torch.exp(score - score.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _lse(l):
    m = l.amax(dim=1, keepdim=True)
    return (m + torch.log(torch.exp(l - m).sum(dim=1, keepdim=True)))[:, 0]


def _plain_balance(s):
    c = s["case"]
    t, e, k, ns = c["tokens"], c["experts"], c["top_k"], c["sequences"]
    seq, live = _live(s)
    # sums over the sequences: blocks of 256 rows times the marks of each sequence's counted
    # rows, then over the blocks, in 64 bits
    chosen = torch.zeros(t, e, device="cuda", dtype=torch.float64)
    chosen = chosen.scatter(1, s["idx"].view(t, k).to(torch.int64), 1.0)
    rows = torch.cat((torch.ones_like(chosen[:, :1]), chosen, _probs(s).double()), dim=1)
    member = ((seq[:, None] == torch.arange(ns, device="cuda")) & live[:, None]).double()
    pad = (0, 0, 0, -t % 256)
    rows = torch.nn.functional.pad(rows, pad).view(-1, 256, 2 * e + 1)
    member = torch.nn.functional.pad(member, pad).view(-1, 256, ns)
    sums = torch.bmm(member.transpose(1, 2).contiguous(), rows).sum(dim=0)
    tokens, counts = sums[:, 0].to(torch.int64), sums[:, 1:e + 1].to(torch.int64)
    sums = sums[:, e + 1:]
    mean = (sums / tokens.clamp(min=1)[:, None]).float()
    f = counts.float() * (e / k) / tokens.clamp(min=1)[:, None].float()
    balance = (f * mean).sum() / (tokens > 0).sum().clamp(min=1)
    z = torch.where(live, _lse(s["logits"]).square(), 0.0).double().sum() / tokens.sum().clamp(min=1)
    return {"loss": torch.stack((balance, z.float())), "counts": counts.to(torch.int32),
            "mean_prob": mean, "tokens": tokens.to(torch.int32)}


def _plain_route_backward(s):
    c = s["case"]
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    l, idx = s["logits"], s["idx"].view(t, k).to(torch.int64)
    seq, live = _live(s)
    d = torch.zeros_like(l)
    if c["balance"]:
        p = _probs(s)
        n = s["tokens"].clamp(min=1).float()
        f = s["counts"].float() * (e / k) / n[:, None]
        f = (f * (s["d_loss"][0] / s["totals"][1].clamp(min=1)) / n[:, None])[seq.clamp(min=0)]
        inner = p * (f - (f * p).sum(dim=1, keepdim=True))
        d = d + (inner * torch.sigmoid(-l) if c["sigmoid"] else inner)
        lse = _lse(l)
        d = d + torch.exp(l - lse[:, None]) * (
            2 * s["d_loss"][1] / s["totals"][0].clamp(min=1) * lse)[:, None]
        d = torch.where(live[:, None], d, 0.0)
    if c["weights"]:
        g = s["d_w"].view(t, k)
        if c["balance"]:
            g = torch.where(live[:, None], g, 0.0)
        chosen = l.gather(1, idx)
        if c["renorm"]:
            score = torch.nn.functional.logsigmoid(chosen) if c["sigmoid"] else chosen
            w = torch.exp(score - score.amax(dim=1, keepdim=True))
            w = w / w.sum(dim=1, keepdim=True)
            part = w * (g - (g * w).sum(dim=1, keepdim=True))
            d = d.scatter_add(1, idx, part * torch.sigmoid(-chosen) if c["sigmoid"] else part)
        elif c["sigmoid"]:
            d = d.scatter_add(1, idx, g * torch.sigmoid(chosen) * torch.sigmoid(-chosen))
        else:
            p = _probs(s)
            gw = g * p.gather(1, idx)
            d = (d - p * gw.sum(dim=1, keepdim=True)).scatter_add(1, idx, gw)
    return {"d_logits": d}


_RUN_OWN = {"project": _own_project, "project_backward": _own_project_backward,
            "balance": _own_balance, "route_backward": _own_route_backward}
_RUN_PLAIN = {"project": _plain_project, "project_backward": _plain_project_backward,
              "balance": _plain_balance, "route_backward": _plain_route_backward}


# ------------------------------------------------------------------ floors
def work(case):
    t = case["tokens"]
    if case["op"] in ("balance", "route_backward"):
        e, k, ns = case["experts"], case["top_k"], case["sequences"]
        read = 4 * t * e + 4 * t * k + 4 * (ns + 1) + (t if case["masked"] else 0)
        if case["op"] == "balance":
            return {"bytes": read + 8 * ns * e + 4 * ns + 8, "flops": 6 * t * e}
        read += (4 * t * k if case["weights"] else 0) + (4 * ns * e if case["balance"] else 0)
        return {"bytes": read + 4 * t * e, "flops": 10 * t * e}
    n, k = _dims(case)
    requests = case["requests"]
    # adapters in use and their mean rank; a third of several requests has none
    named = requests - (requests + 2) // 3 if requests > 2 else requests
    share = named / requests
    used, rank = min(case["adapters"], named), 0.75 * case["rank"]
    weights = n * k * (1 if case["fmt"] == "int8" else 0.5) + n * k / 32
    table = 2 * used * rank * (n + k)
    rows = (t - case["tail"]) * share
    if case["op"] == "project":
        size = 4 if case["out"] == "f32" else 2
        return {"bytes": int(2 * t * k + weights + table + size * t * n),
                "flops": int(2 * t * n * k + 2 * rows * rank * (n + k))}
    grads = 4 * case["adapters"] * ((case["rank"] + 7) // 8 * 8) * (n + k)
    return {"bytes": int(2 * t * (k + n) + weights + table + 2 * t * k + grads),
            "flops": int(2 * t * n * k + 6 * rows * rank * (n + k))}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("project", "project_backward"):
        return _exact_project(s)
    return _exact_router(s)


def _spans(offsets, t):
    """The rows of each part, in the order of the parts."""
    o = [min(max(int(v), 0), t) for v in offsets.tolist()]
    return [slice(b, max(b, e)) for b, e in zip(o[:-1], o[1:])]


def _exact_weight(s):
    """The matrix in 64 bits, from a table of what each code byte holds."""
    c = s["case"]
    n, k = _dims(c)
    per = 1 if c["fmt"] == "int8" else 2  # weights of a byte
    nibble = ([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1] if c["fmt"] == "int4" else
              [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6])
    holds = [[v - 256 if v > 127 else v] if per == 1 else [nibble[v % 16], nibble[v // 16]]
             for v in range(256)]
    table = torch.tensor(holds, dtype=torch.float64, device="cuda")
    slot = s["codes"].view(2, 3, n * k // per)[1, c["matrix"]]
    sc = s["scales"].view(2, 3, n, -1)[1, c["matrix"]]
    if c["fmt"] == "mxfp4":
        sc = torch.ldexp(torch.ones(sc.shape, dtype=torch.float64, device="cuda"), sc.int() - 127)
    width = k // sc.shape[1]
    return table[slot.int()].view(n, k) * sc.double().repeat_interleave(width, dim=1)


def _exact_project(s):
    c = s["case"]
    w, x = _exact_weight(s), s["x"].double()
    spans, owner = _spans(s["offsets"], c["tokens"]), s["adapter"].tolist()
    rank, scale = s["rank"].tolist(), s["scale"].double().tolist()
    if c["op"] == "project":
        y = torch.matmul(x, w.t())
        for at, i in zip(spans, owner):
            if i >= 0:
                a, b = s["a"][i, :rank[i]].double(), s["b"][i, :, :rank[i]].double()
                y[at] += scale[i] * torch.matmul(torch.matmul(x[at], a.t()), b.t())
        return {"y": y}
    dy = s["dy"].double()
    dx = torch.matmul(dy, w)
    da = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
    db = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for at, i in zip(spans, owner):
        if i >= 0:
            a, b = s["a"][i, :rank[i]].double(), s["b"][i, :, :rank[i]].double()
            back = scale[i] * torch.matmul(dy[at], b)
            dx[at] += torch.matmul(back, a)
            da[i, :rank[i]] += torch.matmul(back.t(), x[at])
            db[i, :, :rank[i]] += scale[i] * torch.matmul(dy[at].t(), torch.matmul(x[at], a.t()))
    return {"dx": dx, "da": da, "db": db}


def _exact_router(s):
    """Through autograd of the losses and weights as they are defined."""
    c = s["case"]
    t, e, k, ns = c["tokens"], c["experts"], c["top_k"], c["sequences"]
    l = s["logits"].double().requires_grad_(True)
    idx = s["idx"].view(t, k).to(torch.int64)
    p = torch.sigmoid(l) if c["sigmoid"] else torch.softmax(l, dim=1)
    p = p / p.sum(dim=1, keepdim=True)
    counts = torch.zeros(ns, e, dtype=torch.int64, device="cuda")
    tokens = torch.zeros(ns, dtype=torch.int64, device="cuda")
    live = torch.zeros(t, dtype=torch.bool, device="cuda")
    means = []
    for q, at in enumerate(_spans(s["offsets"], t)):
        ok = torch.ones(at.stop - at.start, dtype=torch.bool, device="cuda")
        if s["valid"] is not None:
            ok = s["valid"][at] != 0
        live[at] = ok
        tokens[q] = ok.sum()
        counts[q] = torch.bincount(idx[at][ok].reshape(-1), minlength=e)
        means.append((p[at] * ok[:, None]).sum(dim=0) / tokens[q].clamp(min=1))
    mean = torch.stack(means)
    f = counts.double() * e / (k * tokens.clamp(min=1)[:, None])
    balance = (f * mean).sum() / (tokens > 0).sum().clamp(min=1)
    z = (torch.logsumexp(l, dim=1).square() * live).sum() / tokens.sum().clamp(min=1)
    if c["op"] == "balance":
        return {"loss": torch.stack((balance, z)).detach(), "counts": counts.to(torch.int32),
                "mean_prob": mean.detach(), "tokens": tokens.to(torch.int32)}
    total = 0.0
    if c["balance"]:
        total = s["d_loss"][0].double() * balance + s["d_loss"][1].double() * z
    if c["weights"]:
        score = torch.sigmoid(l) if c["sigmoid"] else torch.softmax(l, dim=1)
        w = score.gather(1, idx)
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True)
        g = s["d_w"].double().view(t, k)
        total = total + (w * (g * live[:, None] if c["balance"] else g)).sum()
    return {"d_logits": torch.autograd.grad(total, l)[0]}
