"""ctypes binding of libcoli_moe.so: argument marshalling only."""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_PKG, "libcoli_moe.so")

COLI_OK, COLI_E_INVALID, COLI_E_UNSUPPORTED, COLI_E_WORKSPACE, COLI_E_ALIGN, COLI_E_HIP = (
    0, -1, -2, -3, -4, -5)
COLI_ROUTE_SOFTMAX, COLI_ROUTE_SIGMOID, COLI_ROUTE_RENORM = 0, 1, 256
COLI_OUT_BF16, COLI_OUT_F32 = 0, 1
COLI_SRC_BF16, COLI_SRC_F32 = 0, 1
COLI_ENTRY_ROUTE, COLI_ENTRY_DECODE, COLI_ENTRY_PREFILL = 0, 1, 2
COLI_WEIGHTS_INT4, COLI_WEIGHTS_INT8, COLI_WEIGHTS_MXFP4 = 0, 1, 2
COLI_ACT_MXFP8 = 1 << 16


class ColiError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s: %s (status %d)" % (fn, coli_moe_strerror(status), status))
        self.status = status


class _LayerC(ctypes.Structure):
    _fields_ = [
        ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
        ("n_experts", ctypes.c_int32), ("n_shared", ctypes.c_int32),
        ("top_k", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("routed_scale", ctypes.c_float),
        ("q4", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("weight_format", ctypes.c_int32),
    ]


class _TraceC(ctypes.Structure):
    _fields_ = [("start", ctypes.POINTER(ctypes.c_void_p)), ("stop", ctypes.POINTER(ctypes.c_void_p)),
                ("kernel", ctypes.POINTER(ctypes.c_int32)), ("capacity", ctypes.c_int32),
                ("count", ctypes.c_int32)]


KERNEL_NAMES = ["route_fused", "route_topk", "route_group", "decode_gateup", "decode_down",
                "combine", "quantize_q8_0", "plan", "gemm_gateup", "gemm_down", "block_dots",
                "router_logits", "quantize_int4", "quantize_int8", "quantize_mxfp4", "read_probe",
                "mfma_probe", "balance", "balance_finish", "route_backward", "project_prep",
                "project_shrink", "project_gemm", "project_finish", "project_grads",
                "project_reduce", "project_stream", "project_combine"]


class _RouteC(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "topk_idx", "topk_w", "counts", "offsets", "pairs", "pair_pos", "union_ids", "n_union")]


class _AdaptersC(ctypes.Structure):
    _fields_ = [("n_adapters", ctypes.c_int32), ("max_rank", ctypes.c_int32),
                ("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("rank", ctypes.c_void_p),
                ("scale", ctypes.c_void_p)]


class _RequestsC(ctypes.Structure):
    _fields_ = [("n_requests", ctypes.c_int32), ("offsets", ctypes.c_void_p),
                ("adapter", ctypes.c_void_p)]


class _BalanceC(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32)] + [(n, ctypes.c_void_p) for n in (
        "seq_offsets", "valid", "counts", "mean_prob", "tokens", "totals", "loss")]


_lib = None


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise ImportError(
                "libcoli_moe.so is not built (expected at %s); run "
                "`python -m int4_routed_expert_router_amd.build`" % _LIB_PATH)
        lib = ctypes.CDLL(_LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        P = ctypes.POINTER
        lib.coli_moe_workspace_bytes.argtypes = [P(_LayerC), i32, i32]
        lib.coli_moe_workspace_bytes.restype = sz
        lib.coli_moe_route.argtypes = [P(_LayerC), vp, vp, i32, P(_RouteC), vp, sz, vp]
        lib.coli_moe_route_hidden.argtypes = [P(_LayerC), vp, vp, vp, i32, vp, P(_RouteC), vp,
                                              sz, vp]
        lib.coli_moe_forward_decode.argtypes = [P(_LayerC), P(_RouteC), vp, i32, vp, i32, vp, sz, vp]
        lib.coli_moe_forward_prefill.argtypes = [P(_LayerC), P(_RouteC), vp, i32, vp, i32, vp, sz, vp]
        lib.coli_moe_forward_decode_noalloc.argtypes = [P(_LayerC), P(_RouteC), vp, i32, vp, i32, vp]
        lib.coli_moe_quantize_q8_0.argtypes = [vp, i32, i64, vp, vp, vp]
        lib.coli_moe_quantize_int4_gs64.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        lib.coli_moe_quantize_int8_gs64.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        lib.coli_moe_quantize_mxfp4.argtypes = [vp, i32, i64, i64, vp, vp, vp]
        lib.coli_moe_read_probe.argtypes = [vp, i64, vp, vp]
        lib.coli_moe_mfma_probe.argtypes = [i32, i32, i32, vp, vp]
        lib.coli_moe_block_dots.argtypes = [P(_LayerC), i32, i32, vp, i32, vp, vp]
        lib.coli_moe_quantize_mxfp8.argtypes = [vp, i32, i64, vp, vp, vp]
        lib.coli_moe_mx_dots.argtypes = [P(_LayerC), i32, i32, vp, vp, i32, vp, vp]
        lib.coli_moe_project_workspace_bytes.argtypes = [P(_LayerC), i32, P(_AdaptersC), i32, i32]
        lib.coli_moe_project_workspace_bytes.restype = sz
        lib.coli_moe_project.argtypes = [P(_LayerC), i32, i32, P(_AdaptersC), P(_RequestsC), vp,
                                         i32, vp, i32, vp, sz, vp]
        lib.coli_moe_project_backward.argtypes = [P(_LayerC), i32, i32, P(_AdaptersC),
                                                  P(_RequestsC), vp, vp, i32, vp, vp, vp, vp, sz,
                                                  vp]
        lib.coli_moe_balance_workspace_bytes.argtypes = [P(_LayerC), i32, i32]
        lib.coli_moe_balance_workspace_bytes.restype = sz
        lib.coli_moe_balance_loss.argtypes = [P(_LayerC), vp, vp, i32, P(_BalanceC), vp, sz, vp]
        lib.coli_moe_route_backward.argtypes = [P(_LayerC), vp, vp, i32, vp, P(_BalanceC), vp, vp,
                                                vp]
        lib.coli_moe_strerror.argtypes = [ctypes.c_int]
        lib.coli_moe_strerror.restype = ctypes.c_char_p
        lib.coli_moe_set_trace.argtypes = [ctypes.POINTER(_TraceC)]
        lib.coli_moe_set_trace.restype = ctypes.c_int
        lib.coli_moe_version.argtypes = []
        lib.coli_moe_version.restype = ctypes.c_char_p
        for f in ("coli_moe_route", "coli_moe_route_hidden", "coli_moe_forward_decode",
                  "coli_moe_forward_decode_noalloc", "coli_moe_forward_prefill", "coli_moe_quantize_q8_0", "coli_moe_block_dots",
                  "coli_moe_quantize_int4_gs64", "coli_moe_quantize_int8_gs64",
                  "coli_moe_quantize_mxfp4", "coli_moe_read_probe",
                  "coli_moe_mfma_probe", "coli_moe_quantize_mxfp8", "coli_moe_mx_dots",
                  "coli_moe_project", "coli_moe_project_backward", "coli_moe_balance_loss",
                  "coli_moe_route_backward"):
            getattr(lib, f).restype = ctypes.c_int
        _lib = lib
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


class Layer:
    """One MoE layer: shape, routing kind and the device gs64 container.

    q4: uint8 tensor of (E+S)*3*I*H/2 bytes (int4 or MXFP4 codes) or
    (E+S)*3*I*H bytes (int8 codes, int8=True); scales: fp16 tensor of
    (E+S)*3*I*H/64 values, or for MXFP4 (mxfp4=True) a uint8 tensor of
    (E+S)*3*I*H/32 E8M0 bytes (see include/coli_moe.h for the byte layout).
    """

    def __init__(self, hidden, inter, n_experts, n_shared, top_k, flags, q4, scales,
                 routed_scale=1.0, int8=False, mxfp4=False):
        self.q4, self.scales = q4, scales  # keep the tensors alive
        fmt = COLI_WEIGHTS_MXFP4 if mxfp4 else (COLI_WEIGHTS_INT8 if int8 else COLI_WEIGHTS_INT4)
        self.c = _LayerC(hidden, inter, n_experts, n_shared, top_k, flags, routed_scale,
                         _ptr(q4), _ptr(scales), fmt)

    @classmethod
    def from_spec(cls, spec, q4, scales):
        return cls(spec.hidden, spec.inter, spec.n_experts, spec.n_shared, spec.top_k,
                   spec.flags, q4, scales, spec.routed_scale, getattr(spec, "int8", False),
                   getattr(spec, "mxfp4", False))

    hidden = property(lambda s: s.c.hidden)
    inter = property(lambda s: s.c.inter)
    n_experts = property(lambda s: s.c.n_experts)
    n_shared = property(lambda s: s.c.n_shared)
    top_k = property(lambda s: s.c.top_k)


class Route:
    """Device buffers written by coli_moe_route for up to `max_tokens` tokens."""

    def __init__(self, layer: Layer, max_tokens: int, device="cuda"):
        P = max_tokens * layer.top_k
        E = layer.n_experts
        i32 = dict(dtype=torch.int32, device=device)
        self.topk_idx = torch.empty(P, **i32)
        self.topk_w = torch.empty(P, dtype=torch.float32, device=device)
        self.counts = torch.empty(E, **i32)
        self.offsets = torch.empty(E + 1, **i32)
        self.pairs = torch.empty(P, **i32)
        self.pair_pos = torch.empty(P, **i32)
        self.union_ids = torch.empty(E, **i32)
        self.n_union = torch.empty(1, **i32)
        self.c = _RouteC(*[_ptr(getattr(self, n)) for n, _ in _RouteC._fields_])


def _need(t, name, dtype, numel, dev):
    """A dense tensor of this type, on GPU `dev` (-1: the CPU), of at least so many elements, or None."""
    if t is None or (t.dtype is dtype and t.get_device() == dev and t.numel() >= numel
                     and t.is_contiguous()):
        return
    raise ValueError("%s: expected a contiguous %s tensor of at least %d elements on %s, got "
                     "%s %s on %s%s" % (name, dtype, numel, "cuda:%d" % dev if dev >= 0 else "cpu",
                                        tuple(t.shape), t.dtype, t.device,
                                        "" if t.is_contiguous() else " (strided)"))


class Adapters:
    """Low-rank adapters of one N x K matrix: a [n, R, K] and b [n, N, R] bf16
    on the device, R a multiple of 8 up to 128; rank [n] int32 and scale [n]
    fp32 (both optional) on the device."""

    def __init__(self, a, b, rank=None, scale=None):
        if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[1] != b.shape[2]:
            raise ValueError("adapters: expected a [n, R, K] and b [n, N, R], got %s and %s"
                             % (tuple(a.shape), tuple(b.shape)))
        n, r, k = a.shape
        dev = a.get_device()
        _need(a, "a", torch.bfloat16, a.numel(), dev)
        _need(b, "b", torch.bfloat16, b.numel(), dev)
        _need(rank, "rank", torch.int32, n, dev)
        _need(scale, "scale", torch.float32, n, dev)
        self.a, self.b, self.rank, self.scale = a, b, rank, scale  # keep the tensors alive
        self.n, self.r, self.k, self.rows = n, r, k, b.shape[1]
        self.c = _AdaptersC(n, r, _ptr(a), _ptr(b), _ptr(rank), _ptr(scale))


class Requests:
    """The rows and the adapter of every request of a batch: offsets [n + 1]
    and adapter [n], int32 on the device (see include/coli_moe.h)."""

    def __init__(self, offsets, adapter):
        _need(adapter, "adapter", torch.int32, 1, adapter.get_device())
        _need(offsets, "offsets", torch.int32, adapter.numel() + 1, adapter.get_device())
        self.offsets, self.adapter = offsets, adapter
        self.c = _RequestsC(adapter.numel(), _ptr(offsets), _ptr(adapter))


class Balance:
    """Sequences and mask of a routed batch, and the device buffers that
    coli_moe_balance_loss writes: loss [2] (balance, z), counts and mean_prob
    [n_seq, E], tokens [n_seq], totals [2]."""

    def __init__(self, layer: Layer, n_seq: int = 1, seq_offsets=None, valid=None, device="cuda"):
        device = torch.device(device) if seq_offsets is None else seq_offsets.device
        E = layer.n_experts
        self.seq_offsets, self.valid = seq_offsets, valid
        self.counts = torch.empty(n_seq, E, dtype=torch.int32, device=device)
        self.mean_prob = torch.empty(n_seq, E, dtype=torch.float32, device=device)
        self.tokens = torch.empty(n_seq, dtype=torch.int32, device=device)
        self.totals = torch.empty(2, dtype=torch.int32, device=device)
        self.loss = torch.empty(2, dtype=torch.float32, device=device)
        _need(seq_offsets, "seq_offsets", torch.int32, n_seq + 1, self.loss.get_device())
        _need(valid, "valid", torch.uint8, 1, self.loss.get_device())
        self.c = _BalanceC(n_seq, *[_ptr(getattr(self, n)) for n, _ in _BalanceC._fields_[1:]])


def coli_moe_strerror(status: int) -> str:
    return _load().coli_moe_strerror(status).decode()


def coli_moe_version() -> str:
    return _load().coli_moe_version().decode()


def coli_moe_workspace_bytes(layer: Layer, T: int, entry: int) -> int:
    return int(_load().coli_moe_workspace_bytes(ctypes.byref(layer.c), T, entry))


def workspace(layer: Layer, T: int, entry: int, device="cuda") -> torch.Tensor:
    """A device buffer large enough for `entry` at T tokens (256-byte aligned)."""
    n = coli_moe_workspace_bytes(layer, T, entry)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _check(fn, rc):
    if rc != COLI_OK:
        raise ColiError(fn, rc)


def coli_moe_route(layer: Layer, logits, sel_bias, T: int, route: Route, ws=None, stream=None):
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check("coli_moe_route", _load().coli_moe_route(
        ctypes.byref(layer.c), _ptr(logits), _ptr(sel_bias), T, ctypes.byref(route.c),
        _ptr(ws), nb, _stream(stream)))


def coli_moe_route_hidden(layer: Layer, w_router, x, sel_bias, T: int, logits, route: Route,
                          ws=None, stream=None):
    nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check("coli_moe_route_hidden", _load().coli_moe_route_hidden(
        ctypes.byref(layer.c), _ptr(w_router), _ptr(x), _ptr(sel_bias), T, _ptr(logits),
        ctypes.byref(route.c), _ptr(ws), nb, _stream(stream)))


def coli_moe_forward_decode(layer: Layer, route: Route, x, T: int, y, y_dtype: int, ws,
                            stream=None):
    _check("coli_moe_forward_decode", _load().coli_moe_forward_decode(
        ctypes.byref(layer.c), ctypes.byref(route.c), _ptr(x), T, _ptr(y), y_dtype,
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_forward_decode_noalloc(layer: Layer, route: Route, x, T: int, y, y_dtype: int,
                                    stream=None):
    _check("coli_moe_forward_decode_noalloc", _load().coli_moe_forward_decode_noalloc(
        ctypes.byref(layer.c), ctypes.byref(route.c), _ptr(x), T, _ptr(y), y_dtype,
        _stream(stream)))


def coli_moe_forward_prefill(layer: Layer, route: Route, x, T: int, y, y_dtype: int, ws,
                             stream=None):
    _check("coli_moe_forward_prefill", _load().coli_moe_forward_prefill(
        ctypes.byref(layer.c), ctypes.byref(route.c), _ptr(x), T, _ptr(y), y_dtype,
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def coli_moe_quantize_q8_0(src, src_dtype: int, n: int, q, d, stream=None):
    _check("coli_moe_quantize_q8_0", _load().coli_moe_quantize_q8_0(
        _ptr(src), src_dtype, n, _ptr(q), _ptr(d), _stream(stream)))


def coli_moe_quantize_int4_gs64(src, src_dtype: int, rows: int, K: int, q4, scales,
                                stream=None):
    _check("coli_moe_quantize_int4_gs64", _load().coli_moe_quantize_int4_gs64(
        _ptr(src), src_dtype, rows, K, _ptr(q4), _ptr(scales), _stream(stream)))


def coli_moe_quantize_int8_gs64(src, src_dtype: int, rows: int, K: int, q, scales,
                                stream=None):
    _check("coli_moe_quantize_int8_gs64", _load().coli_moe_quantize_int8_gs64(
        _ptr(src), src_dtype, rows, K, _ptr(q), _ptr(scales), _stream(stream)))


def coli_moe_quantize_mxfp4(src, src_dtype: int, rows: int, K: int, q4, e8m0, stream=None):
    _check("coli_moe_quantize_mxfp4", _load().coli_moe_quantize_mxfp4(
        _ptr(src), src_dtype, rows, K, _ptr(q4), _ptr(e8m0), _stream(stream)))


def coli_moe_read_probe(src, nbytes: int, sink, stream=None):
    _check("coli_moe_read_probe", _load().coli_moe_read_probe(
        _ptr(src), nbytes, _ptr(sink), _stream(stream)))


COLI_MFMA_I8_K32, COLI_MFMA_I8_K64, COLI_MFMA_BF16_K32 = 0, 1, 2
MFMA_PROBE_OPS = {COLI_MFMA_I8_K32: 2 * 16 * 16 * 32, COLI_MFMA_I8_K64: 2 * 16 * 16 * 64,
                  COLI_MFMA_BF16_K32: 2 * 16 * 16 * 32}


def coli_moe_mfma_probe(kind: int, iters: int, workgroups: int, sink, stream=None):
    """Returns the operations the launch performs."""
    _check("coli_moe_mfma_probe", _load().coli_moe_mfma_probe(
        kind, iters, workgroups, _ptr(sink), _stream(stream)))
    return workgroups * 4 * iters * 4 * MFMA_PROBE_OPS[kind]


def coli_moe_block_dots(layer: Layer, expert: int, matrix: int, q_act, T: int, dots,
                        stream=None):
    _check("coli_moe_block_dots", _load().coli_moe_block_dots(
        ctypes.byref(layer.c), expert, matrix, _ptr(q_act), T, _ptr(dots), _stream(stream)))


def coli_moe_quantize_mxfp8(src, src_dtype: int, n: int, q, e8m0, stream=None):
    _check("coli_moe_quantize_mxfp8", _load().coli_moe_quantize_mxfp8(
        _ptr(src), src_dtype, n, _ptr(q), _ptr(e8m0), _stream(stream)))


def coli_moe_mx_dots(layer: Layer, expert: int, matrix: int, q_act, e_act, T: int, out,
                     stream=None):
    _check("coli_moe_mx_dots", _load().coli_moe_mx_dots(
        ctypes.byref(layer.c), expert, matrix, _ptr(q_act), _ptr(e_act), T, _ptr(out),
        _stream(stream)))


def _shape_nk(layer: Layer, matrix: int):
    return (layer.hidden, layer.inter) if matrix == 2 else (layer.inter, layer.hidden)


def _run(name, on, stream, *args):
    """Calls the library on the device of tensor `on`: by default on that
    device's current stream, which is made current for the call if it is not."""
    fn = getattr(_load(), name)
    dev = on.get_device()
    if dev < 0:
        raise ValueError("%s: tensors have to be on the GPU, got %s" % (name, on.device))
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    if dev == torch._C._cuda_getDevice():
        rc = fn(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, s)
    if rc != COLI_OK:
        raise ColiError(name, rc)


def _ws(ws, on):
    """Pointer and bytes of a workspace."""
    _need(ws, "ws", ws.dtype, 0, on.get_device())
    return ws.data_ptr(), ws.numel() * ws.element_size()


def coli_moe_project_workspace_bytes(layer: Layer, matrix: int, adapters, T: int,
                                     backward: bool = False) -> int:
    return int(_load().coli_moe_project_workspace_bytes(
        ctypes.byref(layer.c), matrix, None if adapters is None else ctypes.byref(adapters.c), T,
        int(backward)))


def project_workspace(layer: Layer, matrix: int, adapters, T: int, backward: bool = False,
                      device="cuda") -> torch.Tensor:
    """A device buffer large enough for coli_moe_project[_backward] at T rows."""
    n = coli_moe_project_workspace_bytes(layer, matrix, adapters, T, backward)
    return torch.empty(max(n, 256), dtype=torch.uint8,
                       device=device if adapters is None else adapters.a.device)


def _project_args(layer, matrix, adapters, requests, x, T):
    n, k = _shape_nk(layer, matrix)
    dev = x.get_device()
    _need(x, "x", torch.bfloat16, T * k, dev)
    for w in (layer.q4, layer.scales):
        if isinstance(w, torch.Tensor) and w.get_device() != dev:
            raise ValueError("the layer's weights on %s, x on %s" % (w.device, x.device))
    if adapters is None or requests is None:
        ad = None if adapters is None else ctypes.byref(adapters.c)
        return n, k, dev, ad, None if requests is None else ctypes.byref(requests.c)
    if adapters.k != k or adapters.rows != n:
        raise ValueError("adapters of a %d x %d matrix given for a %d x %d one"
                         % (adapters.rows, adapters.k, n, k))
    if adapters.a.get_device() != dev or requests.adapter.get_device() != dev:
        raise ValueError("adapters on %s, requests on %s, x on %s"
                         % (adapters.a.device, requests.adapter.device, x.device))
    return n, k, dev, ctypes.byref(adapters.c), ctypes.byref(requests.c)


def coli_moe_project(layer: Layer, expert: int, matrix: int, adapters, requests, x, T: int, y,
                     y_dtype: int, ws, stream=None):
    """y = x W^T + the requests' adapters (adapters and requests may both be None)."""
    n, _, dev, ad, rq = _project_args(layer, matrix, adapters, requests, x, T)
    _need(y, "y", torch.float32 if y_dtype == COLI_OUT_F32 else torch.bfloat16, T * n, dev)
    _run("coli_moe_project", x, stream, ctypes.byref(layer.c), expert, matrix, ad, rq,
         x.data_ptr(), T, y.data_ptr(), y_dtype, *_ws(ws, x))


def coli_moe_project_backward(layer: Layer, expert: int, matrix: int, adapters, requests, x, dy,
                              T: int, dx, d_a, d_b, ws, stream=None):
    """dx (bf16), d_a and d_b (fp32) of coli_moe_project; dx, or d_a and d_b, may be None."""
    n, k, dev, ad, rq = _project_args(layer, matrix, adapters, requests, x, T)
    _need(dy, "dy", torch.bfloat16, T * n, dev)
    _need(dx, "dx", torch.bfloat16, T * k, dev)
    if adapters is not None:
        _need(d_a, "d_a", torch.float32, adapters.a.numel(), dev)
        _need(d_b, "d_b", torch.float32, adapters.b.numel(), dev)
    _run("coli_moe_project_backward", x, stream, ctypes.byref(layer.c), expert, matrix, ad, rq,
         x.data_ptr(), dy.data_ptr(), T, _ptr(dx), _ptr(d_a), _ptr(d_b), *_ws(ws, x))


def coli_moe_balance_workspace_bytes(layer: Layer, T: int, n_seq: int = 1) -> int:
    return int(_load().coli_moe_balance_workspace_bytes(ctypes.byref(layer.c), T, n_seq))


def balance_workspace(layer: Layer, T: int, n_seq: int = 1, device="cuda") -> torch.Tensor:
    """A device buffer large enough for coli_moe_balance_loss at T tokens."""
    return torch.empty(max(coli_moe_balance_workspace_bytes(layer, T, n_seq), 256),
                       dtype=torch.uint8, device=device)


def _balance_args(layer, logits, topk_idx, T, balance):
    dev, E = logits.get_device(), layer.n_experts
    _need(logits, "logits", torch.float32, T * E, dev)
    _need(topk_idx, "topk_idx", torch.int32, T * layer.top_k, dev)
    if balance is not None:
        _need(balance.valid, "valid", torch.uint8, T, dev)
        _need(balance.counts, "balance", torch.int32, balance.c.n_seq * E, dev)
    return dev


def coli_moe_balance_loss(layer: Layer, logits, topk_idx, T: int, balance: Balance, ws,
                          stream=None):
    _balance_args(layer, logits, topk_idx, T, balance)
    _run("coli_moe_balance_loss", logits, stream, ctypes.byref(layer.c), logits.data_ptr(),
         topk_idx.data_ptr(), T, ctypes.byref(balance.c), *_ws(ws, logits))


def coli_moe_route_backward(layer: Layer, logits, topk_idx, T: int, d_topk_w, balance, d_loss,
                            d_logits, stream=None):
    """d_logits of the routing weights (d_topk_w) and of the balance and z-losses
    (balance, d_loss); either part may be None."""
    dev = _balance_args(layer, logits, topk_idx, T, balance)
    _need(d_topk_w, "d_topk_w", torch.float32, T * layer.top_k, dev)
    _need(d_loss, "d_loss", torch.float32, 2, dev)
    _need(d_logits, "d_logits", torch.float32, T * layer.n_experts, dev)
    _run("coli_moe_route_backward", logits, stream, ctypes.byref(layer.c), logits.data_ptr(),
         topk_idx.data_ptr(), T, _ptr(d_topk_w),
         None if balance is None else ctypes.byref(balance.c), _ptr(d_loss), d_logits.data_ptr())


def _hip_runtime():
    """The HIP runtime already loaded in this process (torch's or the system's)."""
    path = None
    with open("/proc/self/maps") as f:
        for line in f:
            if "libamdhip64.so" in line:
                path = line.split()[-1]
                break
    return ctypes.CDLL(path or "libamdhip64.so")


class KernelTimer:
    """Times every kernel the library launches while active: each dispatch
    stamps its own start and stop event (hipExtLaunchKernel)."""

    def __init__(self, capacity: int = 4096):
        _load()
        self.hip = _hip_runtime()
        self.hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p,
                                                 ctypes.c_void_p]
        self.hip.hipEventSynchronize.argtypes = [ctypes.c_void_p]
        self.hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self.start = (ctypes.c_void_p * capacity)()
        self.stop = (ctypes.c_void_p * capacity)()
        self.kernel = (ctypes.c_int32 * capacity)()
        for arr in (self.start, self.stop):
            for i in range(capacity):
                ev = ctypes.c_void_p()
                if self.hip.hipEventCreate(ctypes.byref(ev)) != 0:
                    raise RuntimeError("hipEventCreate failed")
                arr[i] = ev
        self.c = _TraceC(ctypes.cast(self.start, ctypes.POINTER(ctypes.c_void_p)),
                         ctypes.cast(self.stop, ctypes.POINTER(ctypes.c_void_p)),
                         ctypes.cast(self.kernel, ctypes.POINTER(ctypes.c_int32)), capacity, 0)

    def __enter__(self):
        self.c.count = 0
        _check("coli_moe_set_trace", _load().coli_moe_set_trace(ctypes.byref(self.c)))
        return self

    def __exit__(self, *exc):
        _load().coli_moe_set_trace(None)
        return False

    def results(self):
        """[(kernel name, milliseconds)] of every timed kernel, in launch order."""
        out = []
        for i in range(self.c.count):
            self.hip.hipEventSynchronize(self.stop[i])
            ms = ctypes.c_float()
            if self.hip.hipEventElapsedTime(ctypes.byref(ms), self.start[i], self.stop[i]) != 0:
                raise RuntimeError("hipEventElapsedTime failed")
            out.append((KERNEL_NAMES[self.kernel[i]], ms.value))
        return out

    def close(self):
        for arr in (self.start, self.stop):
            for ev in arr:
                if ev:
                    self.hip.hipEventDestroy(ev)


def raw_library():
    """The loaded ctypes library (tests use it to check exported symbols)."""
    return _load()
