"""Python binding of ``libqgg.so``, the gfx950 quantized MoE grouped-GEMM library.

Argument marshalling only: every step of the path runs in the library's HIP
kernels, which this module reaches through ctypes with raw device pointers and
the current HIP stream.  PyTorch supplies device memory and streams.  If the
library is not built, every call raises; there is no fallback.

Names follow the C-ABI in ``include/qgg.h``: ``moe_route``, ``expert_permute``,
``dequant_grouped_gemm``, ``lora_grouped_gemm``, ``moe_ffn_fwd``, ``moe_dx_bwd``,
``moe_router_bwd``; scored routing (``moe_route_scored``, ``moe_route_scored_bwd``) and 8-bit
floating point (``fp8_quantize``, ``fp8_dequantize``, ``fp8_grouped_gemm``, ``swiglu_fp8``,
``swiglu_fp8_bwd``, ``moe_combine``).
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

from . import accounting  # noqa: F401  (host-side byte/FLOP accounting)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqgg.so")

FMT_MXFP4 = 1
FMT_INT4 = 2
LAYOUT_ROWS = 0
LAYOUT_MFMA = 1
CHUNKED = 0
FUSED = 1
A_SORTED = 0
A_TOKENS = 1
TRANSPOSE_W = 2
DEQUANT_ONLY = 4
CALL_PERMUTE = 1
CALL_GEMM = 2
CALL_FFN_FWD = 3
CALL_DX_BWD = 4
CALL_LORA_BWD = 5
CALL_FFN_LORA_BWD = 6

STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported", 3: "workspace too small", 4: "HIP error"}

# Every symbol include/qgg.h declares.
EXPORTS = ("moe_route", "expert_permute", "dequant_grouped_gemm", "lora_grouped_gemm",
           "lora_grouped_gemm_bwd", "moe_ffn_fwd", "moe_ffn_fwd_noalloc", "moe_ffn_fwd_lora",
           "moe_dx_bwd", "moe_ffn_bwd_lora",
           "moe_router_bwd", "moe_route_scored", "moe_route_scored_bwd", "qgg_fp8_quantize",
           "qgg_fp8_dequantize", "fp8_grouped_gemm", "moe_swiglu_fp8", "moe_swiglu_fp8_bwd",
           "moe_combine", "qgg_repack_weights", "qgg_check_weights", "qgg_workspace_bytes",
           "qgg_set_timing_events", "qgg_timing_count", "qgg_timing_kind", "qgg_status_string",
           "qgg_version")

_lib = None


class QggError(RuntimeError):
    pass


class _QWeight(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("E", ctypes.c_int32), ("N", ctypes.c_int32),
                ("K", ctypes.c_int32), ("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("layout", ctypes.c_int32)]


class _Lora(ctypes.Structure):
    _fields_ = [("rank", ctypes.c_int32), ("alpha", ctypes.c_float), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p)]


class _RouteOpts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class _Fp8Weight(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("scale_type", ctypes.c_int32), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]


class _Perm(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in
                ("counts", "offsets", "perm", "inv_perm", "active", "n_active")]


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise QggError(f"{LIB_PATH} is missing: build it with "
                           "`python -m quantized_grouped_gemm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_route.argtypes = [P, i32, i32, i32, P, P, P, P]
        L.expert_permute.argtypes = [P, i32, i32, i32, ctypes.POINTER(_Perm), P, i32, P, P, P, sz, P]
        L.dequant_grouped_gemm.argtypes = [ctypes.POINTER(_QWeight), P, i32, ctypes.POINTER(_Perm),
                                           i32, i32, i32, i32, P, sz, P, P]
        L.lora_grouped_gemm.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_Lora), P, i32,
                                        ctypes.POINTER(_Perm), i32, i32, i32, i32, P, sz, P, P, P]
        L.lora_grouped_gemm_bwd.argtypes = [ctypes.POINTER(_Lora), i32, i32, i32, P, i32, P, P,
                                            ctypes.POINTER(_Perm), i32, i32, P, sz, P, P, P, P]
        L.moe_ffn_fwd.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight), P, P, i32,
                                  i32, i32, i32, i32, i32, i32, P, P, ctypes.POINTER(_Perm), P, P,
                                  P, sz, P, P]
        L.moe_ffn_fwd_noalloc.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight), P,
                                          P, i32, i32, i32, i32, i32, i32, i32, P, P,
                                          ctypes.POINTER(_Perm), P, P, P, P]
        L.moe_ffn_fwd_lora.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight),
                                       ctypes.POINTER(_Lora), ctypes.POINTER(_Lora), P, P, i32,
                                       i32, i32, i32, i32, i32, i32, P, P, ctypes.POINTER(_Perm),
                                       P, P, P, P, P, sz, P, P]
        L.moe_dx_bwd.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight), P, P,
                                 ctypes.POINTER(_Perm), P, i32, i32, i32, i32, i32, i32, i32, P,
                                 sz, P, P]
        L.moe_ffn_bwd_lora.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight),
                                       ctypes.POINTER(_Lora), ctypes.POINTER(_Lora), P, P, P,
                                       ctypes.POINTER(_Perm), P, P, P, i32, i32, i32, i32, i32,
                                       i32, i32, P, sz, P, P, P, P, P, P]
        L.moe_router_bwd.argtypes = [ctypes.POINTER(_QWeight), ctypes.POINTER(_QWeight), P, P, P,
                                     ctypes.POINTER(_Perm), P, i32, i32, i32, i32, i32, i32, i32,
                                     P, sz, P, P, P, P]
        L.qgg_repack_weights.argtypes = [ctypes.POINTER(_QWeight), P, P, P]
        L.qgg_repack_weights.restype = ctypes.c_int
        L.qgg_check_weights.argtypes = [ctypes.POINTER(_QWeight), P, P]
        L.qgg_check_weights.restype = ctypes.c_int
        L.qgg_workspace_bytes.argtypes = [i32, i32, i32, i32, i32, i32, i32, i32,
                                          ctypes.POINTER(ctypes.c_size_t)]
        L.qgg_workspace_bytes.restype = ctypes.c_size_t
        L.qgg_set_timing_events.argtypes = [P, i32]
        L.qgg_set_timing_events.restype = ctypes.c_int
        L.qgg_timing_count.restype = ctypes.c_int
        L.qgg_timing_kind.argtypes = [i32]
        L.qgg_timing_kind.restype = ctypes.c_int
        L.qgg_status_string.argtypes = [i32]
        L.qgg_status_string.restype = ctypes.c_char_p
        L.qgg_version.restype = ctypes.c_char_p
        i64 = ctypes.c_int64
        L.moe_route_scored.argtypes = [P, i32, P, i32, i32, i32, ctypes.POINTER(_RouteOpts), P, P,
                                       P, P]
        L.moe_route_scored_bwd.argtypes = [P, i32, P, P, i32, i32, i32,
                                           ctypes.POINTER(_RouteOpts), P, P]
        L.qgg_fp8_quantize.argtypes = [P, i64, i32, P, P, P]
        L.qgg_fp8_dequantize.argtypes = [P, P, i64, i32, P, P]
        L.fp8_grouped_gemm.argtypes = [ctypes.POINTER(_Fp8Weight), P, P, i32,
                                       ctypes.POINTER(_Perm), i32, i32, P, P]
        L.moe_swiglu_fp8.argtypes = [P, P, i64, i32, P, P, P, P, P, P]
        L.moe_swiglu_fp8_bwd.argtypes = [P, P, P, P, ctypes.POINTER(_Perm), i32, i32, i32, P, P, P,
                                         P, P]
        L.moe_combine.argtypes = [P, i32, ctypes.POINTER(_Perm), P, i32, i32, P, P]
        for f in ("moe_route_scored", "moe_route_scored_bwd", "qgg_fp8_quantize",
                  "qgg_fp8_dequantize", "fp8_grouped_gemm", "moe_swiglu_fp8", "moe_swiglu_fp8_bwd",
                  "moe_combine"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("moe_route", "expert_permute", "dequant_grouped_gemm", "lora_grouped_gemm",
                  "lora_grouped_gemm_bwd", "moe_ffn_fwd", "moe_ffn_fwd_noalloc",
                  "moe_ffn_fwd_lora", "moe_dx_bwd", "moe_ffn_bwd_lora", "moe_router_bwd"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def _check(rc: int, what: str):
    if rc != 0:
        raise QggError(f"{what}: {lib().qgg_status_string(rc).decode()} ({rc})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


@dataclass
class QWeight:
    """Frozen 4-bit expert weights on the device: packed bytes and scales
    (uint8 E8M0 for MXFP4, BF16 bits for INT4) of E experts of [N][K], in
    LAYOUT_ROWS ([E][N][K/2], [E][N][K/32]) or LAYOUT_MFMA order (same sizes,
    see include/qgg.h).  Shapes are given by E, N, K."""
    fmt: int
    packed: "object"
    scales: "object"
    layout: int = LAYOUT_ROWS
    shape: tuple = None

    def __post_init__(self):
        if self.shape is None:
            self.shape = (self.packed.shape[0], self.packed.shape[1], self.packed.shape[2] * 2)

    @property
    def E(self):
        return self.shape[0]

    @property
    def N(self):
        return self.shape[1]

    @property
    def K(self):
        return self.shape[2]

    def c(self):
        return _QWeight(self.fmt, self.E, self.N, self.K, self.packed.data_ptr(),
                        self.scales.data_ptr(), self.layout)


def repack(w: "QWeight") -> "QWeight":
    """The MFMA-tiled copy of row-layout weights (qgg_repack_weights)."""
    import torch
    assert w.layout == LAYOUT_ROWS
    p = torch.empty_like(w.packed)
    s = torch.empty_like(w.scales)
    wc = w.c()
    _check(lib().qgg_repack_weights(ctypes.byref(wc), _ptr(p), _ptr(s), _stream()),
           "qgg_repack_weights")
    return QWeight(w.fmt, p, s, LAYOUT_MFMA, w.shape)


def check_weights(w: "QWeight", err_flag=None):
    """qgg_check_weights: bit 4 of the returned device int32 flag is set when a
    scale of ``w`` lies outside the fused decoder's exact domain (``err_flag``,
    if given, is that device tensor, zeroed by the caller)."""
    import torch
    if err_flag is None:
        err_flag = torch.zeros(1, dtype=torch.int32, device=w.packed.device)
    wc = w.c()
    _check(lib().qgg_check_weights(ctypes.byref(wc), _ptr(err_flag), _stream()),
           "qgg_check_weights")
    return err_flag


_timing_keep = None


def set_timing_events(events, capacity: int):
    """qgg_set_timing_events with a list of 2*capacity recorded-once
    torch.cuda.Event(enable_timing=True) objects (None stops)."""
    global _timing_keep
    if events is None:
        _timing_keep = None
        _check(lib().qgg_set_timing_events(None, 0), "qgg_set_timing_events")
        return
    arr = (ctypes.c_void_p * len(events))(*[e.cuda_event for e in events])
    _timing_keep = arr
    _check(lib().qgg_set_timing_events(ctypes.cast(arr, ctypes.c_void_p), capacity),
           "qgg_set_timing_events")


def timing_count() -> int:
    return int(lib().qgg_timing_count())


def timing_kinds(n: int):
    return [int(lib().qgg_timing_kind(i)) for i in range(n)]


@dataclass
class Perm:
    """Routing permutation (device int32 tensors), see ``qgg_perm``."""
    counts: "object"
    offsets: "object"
    perm: "object"
    inv_perm: "object"
    active: "object"
    n_active: "object"

    @staticmethod
    def empty(P: int, E: int, device):
        import torch
        z = lambda n: torch.empty(max(n, 1), dtype=torch.int32, device=device)  # noqa: E731
        return Perm(z(E), z(E + 1), z(P), z(P), z(E), z(1))

    def c(self):
        return _Perm(*(t.data_ptr() for t in (self.counts, self.offsets, self.perm,
                                               self.inv_perm, self.active, self.n_active)))


def workspace_bytes(call: int, T: int, d: int, E: int, k: int, n_or_inter: int, variant: int,
                    chunk: int):
    """(total workspace bytes, dequant scratch bytes) for a call."""
    s = ctypes.c_size_t(0)
    total = lib().qgg_workspace_bytes(call, T, d, E, k, n_or_inter, variant, chunk,
                                      ctypes.byref(s))
    return int(total), int(s.value)


class Workspace:
    """A reusable device byte buffer that grows on demand.

    Calls run in stream order on the current stream, so one workspace serves any
    number of calls issued on that stream; calls that may run concurrently on
    different streams each need their own (the module default is shared)."""

    def __init__(self):
        self.buf = None

    def get(self, nbytes: int, device):
        import torch
        if self.buf is None or self.buf.numel() < nbytes or self.buf.device != device:
            self.buf = None
            self.buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        return self.buf


_default_ws = Workspace()


def moe_route(logits, k: int, err_flag=None):
    """(topk_ids int32 [T,k], topk_gates fp32 [T,k]) for fp32 logits [T,E]."""
    import torch
    T, E = logits.shape
    ids = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    gates = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(gates), _ptr(err_flag),
                           _stream()), "moe_route")
    return ids, gates


def expert_permute(topk_ids, E: int, x=None, err_flag=None, ws: Workspace | None = None):
    """Perm for int32 ids [T,k]; with x [T,d] BF16 also returns x_perm [P,d]."""
    import torch
    T, k = topk_ids.shape
    dev = topk_ids.device
    p = Perm.empty(T * k, E, dev)
    x_perm = None
    d = 0
    if x is not None:
        d = x.shape[1]
        x_perm = torch.empty((T * k, d), dtype=x.dtype, device=dev)
    nb, _ = workspace_bytes(CALL_PERMUTE, T, 128, E, k, 64, FUSED, 0)
    buf = (ws or _default_ws).get(nb, dev)
    pc = p.c()
    _check(lib().expert_permute(_ptr(topk_ids), T, k, E, ctypes.byref(pc), _ptr(x), d,
                                _ptr(x_perm), _ptr(err_flag), _ptr(buf), buf.numel(), _stream()),
           "expert_permute")
    return p, x_perm


def dequant_grouped_gemm(w: QWeight, a, perm: Perm, T: int, k: int, variant: int = FUSED,
                         chunk: int = 0, flags: int = A_TOKENS, ws: Workspace | None = None,
                         out=None):
    """y [P, N] (or [P, K] with TRANSPOSE_W) in sorted order, BF16."""
    import torch
    dev = w.packed.device
    P = T * k
    trans = bool(flags & TRANSPOSE_W)
    ncols = w.K if trans else w.N
    if flags & DEQUANT_ONLY:
        y = None
    else:
        y = out if out is not None else torch.empty((P, ncols), dtype=torch.bfloat16, device=dev)
    nb, _ = workspace_bytes(CALL_GEMM, T, w.K, w.E, k, w.N, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    wc, pc = w.c(), perm.c()
    _check(lib().dequant_grouped_gemm(ctypes.byref(wc), _ptr(a), flags, ctypes.byref(pc), T, k,
                                      variant, chunk, _ptr(buf), buf.numel(), _ptr(y), _stream()),
           "dequant_grouped_gemm")
    return y if y is not None else buf


def lora_grouped_gemm(w: QWeight, A, B, alpha: float, a, perm: Perm, T: int, k: int,
                      variant: int = FUSED, chunk: int = 0, flags: int = A_TOKENS,
                      ws: Workspace | None = None):
    """(y [P, N], u [P, rank]) BF16 in sorted order: the projection with a LoRA adapter,
    A [E, rank, K] and B [E, N, rank] BF16 device tensors."""
    import torch
    dev = w.packed.device
    P = T * k
    rank = A.shape[1]
    y = torch.empty((P, w.N), dtype=torch.bfloat16, device=dev)
    u = torch.empty((P, rank), dtype=torch.bfloat16, device=dev)
    nb, _ = workspace_bytes(CALL_GEMM, T, w.K, w.E, k, w.N, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    wc, pc = w.c(), perm.c()
    lc = _Lora(rank, float(alpha), A.data_ptr(), B.data_ptr())
    _check(lib().lora_grouped_gemm(ctypes.byref(wc), ctypes.byref(lc), _ptr(a), flags,
                                   ctypes.byref(pc), T, k, variant, chunk, _ptr(buf), buf.numel(),
                                   _ptr(u), _ptr(y), _stream()), "lora_grouped_gemm")
    return y, u


def lora_grouped_gemm_bwd(A, B, alpha: float, a, dy, u, perm: Perm, T: int, k: int,
                          flags: int = A_TOKENS, want=("dx", "dA", "dB"),
                          ws: Workspace | None = None):
    """{"dx": [P, K] BF16, "dA": [E, rank, K] fp32, "dB": [E, N, rank] fp32} (those in
    `want`): the adapter's backward for the upstream gradient dy [P, N] (sorted)."""
    import torch
    E, rank, K = A.shape
    N = B.shape[1]
    dev = dy.device
    P = T * k
    dx = torch.empty((P, K), dtype=torch.bfloat16, device=dev) if "dx" in want else None
    dA = torch.empty((E, rank, K), dtype=torch.float32, device=dev) if "dA" in want else None
    dB = torch.empty((E, N, rank), dtype=torch.float32, device=dev) if "dB" in want else None
    nb, _ = workspace_bytes(CALL_LORA_BWD, T, N, E, k, rank, FUSED, 0)
    buf = (ws or _default_ws).get(nb, dev)
    pc = perm.c()
    lc = _Lora(rank, float(alpha), A.data_ptr(), B.data_ptr())
    _check(lib().lora_grouped_gemm_bwd(ctypes.byref(lc), E, N, K, _ptr(a), flags, _ptr(dy),
                                       _ptr(u), ctypes.byref(pc), T, k, _ptr(buf), buf.numel(),
                                       _ptr(dx), _ptr(dA), _ptr(dB), _stream()),
           "lora_grouped_gemm_bwd")
    return {"dx": dx, "dA": dA, "dB": dB}


def moe_ffn_fwd(w_gate_up: QWeight, w_down: QWeight, x, logits, k: int, variant: int = FUSED,
                chunk: int = 0, save_h: bool = False, err_flag=None, ws: Workspace | None = None):
    """dict(y [T,d], topk_ids, topk_gates, perm, h [P,2I] or None)."""
    import torch
    T, d = x.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = x.device
    P = T * k
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    p = Perm.empty(P, E, dev)
    h = torch.empty((P, 2 * inter), dtype=torch.bfloat16, device=dev) if save_h else None
    y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    nb, _ = workspace_bytes(CALL_FFN_FWD, T, d, E, k, inter, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), p.c()
    _check(lib().moe_ffn_fwd(ctypes.byref(g), ctypes.byref(dn), _ptr(x), _ptr(logits), T, d, E, k,
                             inter, variant, chunk, _ptr(ids), _ptr(gates), ctypes.byref(pc),
                             _ptr(h), _ptr(err_flag), _ptr(buf), buf.numel(), _ptr(y), _stream()),
           "moe_ffn_fwd")
    return dict(y=y, topk_ids=ids, topk_gates=gates, perm=p, h=h)


STATIC_SCRATCH_BYTES = 32 << 20


def moe_ffn_fwd_noalloc(w_gate_up: QWeight, w_down: QWeight, x, logits, k: int,
                        variant: int = FUSED, chunk: int = 0, save_h: bool = False,
                        err_flag=None):
    """moe_ffn_fwd on the library's static scratch (no workspace); same result dict."""
    import torch
    T, d = x.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = x.device
    P = T * k
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    p = Perm.empty(P, E, dev)
    h = torch.empty((P, 2 * inter), dtype=torch.bfloat16, device=dev) if save_h else None
    y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), p.c()
    _check(lib().moe_ffn_fwd_noalloc(ctypes.byref(g), ctypes.byref(dn), _ptr(x), _ptr(logits), T,
                                     d, E, k, inter, variant, chunk, _ptr(ids), _ptr(gates),
                                     ctypes.byref(pc), _ptr(h), _ptr(err_flag), _ptr(y),
                                     _stream()), "moe_ffn_fwd_noalloc")
    return dict(y=y, topk_ids=ids, topk_gates=gates, perm=p, h=h)


def moe_ffn_fwd_lora(w_gate_up: QWeight, w_down: QWeight, lora_gate_up, lora_down, x, logits,
                     k: int, variant: int = FUSED, chunk: int = 0, save_h: bool = False,
                     err_flag=None, ws: Workspace | None = None):
    """moe_ffn_fwd with BF16 LoRA adapters: lora_gate_up / lora_down are (A, B, alpha)
    tuples of device tensors (A [E, r, K], B [E, N, r]) or None.  Adds u_gate_up /
    u_down [P, r] (sorted order) to the result."""
    import torch
    T, d = x.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = x.device
    P = T * k
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    p = Perm.empty(P, E, dev)
    h = torch.empty((P, 2 * inter), dtype=torch.bfloat16, device=dev) if save_h else None
    y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)

    def adapter(l):
        if l is None:
            return None, None
        A, B, alpha = l
        u = torch.empty((P, A.shape[1]), dtype=torch.bfloat16, device=dev)
        return _Lora(A.shape[1], float(alpha), A.data_ptr(), B.data_ptr()), u

    lgu, ugu = adapter(lora_gate_up)
    ldn, udn = adapter(lora_down)
    nb, _ = workspace_bytes(CALL_FFN_FWD, T, d, E, k, inter, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), p.c()
    _check(lib().moe_ffn_fwd_lora(ctypes.byref(g), ctypes.byref(dn),
                                  ctypes.byref(lgu) if lgu else None,
                                  ctypes.byref(ldn) if ldn else None, _ptr(x), _ptr(logits), T, d,
                                  E, k, inter, variant, chunk, _ptr(ids), _ptr(gates),
                                  ctypes.byref(pc), _ptr(h), _ptr(ugu), _ptr(udn),
                                  _ptr(err_flag), _ptr(buf), buf.numel(), _ptr(y), _stream()),
           "moe_ffn_fwd_lora")
    return dict(y=y, topk_ids=ids, topk_gates=gates, perm=p, h=h, u_gate_up=ugu, u_down=udn)


def moe_dx_bwd(w_gate_up: QWeight, w_down: QWeight, dy, topk_gates, perm: Perm, h_saved, k: int,
               variant: int = FUSED, chunk: int = 0, ws: Workspace | None = None):
    """dx [T,d] BF16: the input gradient through the frozen base."""
    import torch
    T, d = dy.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = dy.device
    dx = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    nb, _ = workspace_bytes(CALL_DX_BWD, T, d, E, k, inter, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), perm.c()
    _check(lib().moe_dx_bwd(ctypes.byref(g), ctypes.byref(dn), _ptr(dy), _ptr(topk_gates),
                            ctypes.byref(pc), _ptr(h_saved), T, d, E, k, inter, variant, chunk,
                            _ptr(buf), buf.numel(), _ptr(dx), _stream()), "moe_dx_bwd")
    return dx


def moe_ffn_bwd_lora(w_gate_up: QWeight, w_down: QWeight, lora_gate_up, lora_down, x, dy,
                     topk_gates, perm: Perm, h_saved, u_gate_up, u_down, k: int,
                     variant: int = FUSED, chunk: int = 0,
                     want=("dx", "dA_gate_up", "dB_gate_up", "dA_down", "dB_down"),
                     ws: Workspace | None = None):
    """Backward of moe_ffn_fwd_lora: {"dx": [T, d] BF16, "dA_gate_up": [E, r, d],
    "dB_gate_up": [E, 2I, r], "dA_down": [E, r, I], "dB_down": [E, d, r]} (fp32;
    those in `want` whose adapter is given, else None).  lora_gate_up /
    lora_down are (A, B, alpha) tuples as for moe_ffn_fwd_lora, or None."""
    import torch
    T, d = dy.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = dy.device

    def grad(name, l, shape_of):
        if l is None or name not in want:
            return None
        return torch.empty(shape_of(l), dtype=torch.float32, device=dev)

    dx = torch.empty((T, d), dtype=torch.bfloat16, device=dev) if "dx" in want else None
    dAg = grad("dA_gate_up", lora_gate_up, lambda l: tuple(l[0].shape))
    dBg = grad("dB_gate_up", lora_gate_up, lambda l: tuple(l[1].shape))
    dAd = grad("dA_down", lora_down, lambda l: tuple(l[0].shape))
    dBd = grad("dB_down", lora_down, lambda l: tuple(l[1].shape))

    def adapter(l):
        if l is None:
            return None
        A, B, alpha = l
        return _Lora(A.shape[1], float(alpha), A.data_ptr(), B.data_ptr())

    lg, ld = adapter(lora_gate_up), adapter(lora_down)
    nb, _ = workspace_bytes(CALL_FFN_LORA_BWD, T, d, E, k, inter, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), perm.c()
    _check(lib().moe_ffn_bwd_lora(ctypes.byref(g), ctypes.byref(dn),
                                  ctypes.byref(lg) if lg else None,
                                  ctypes.byref(ld) if ld else None, _ptr(x), _ptr(dy),
                                  _ptr(topk_gates), ctypes.byref(pc), _ptr(h_saved),
                                  _ptr(u_gate_up), _ptr(u_down), T, d, E, k, inter, variant,
                                  chunk, _ptr(buf), buf.numel(), _ptr(dx), _ptr(dAg), _ptr(dBg),
                                  _ptr(dAd), _ptr(dBd), _stream()), "moe_ffn_bwd_lora")
    return {"dx": dx, "dA_gate_up": dAg, "dB_gate_up": dBg, "dA_down": dAd, "dB_down": dBd}


def moe_router_bwd(w_gate_up: QWeight, w_down: QWeight, dy, topk_ids, topk_gates, perm: Perm,
                   h_saved, k: int, variant: int = FUSED, chunk: int = 0, want_dx: bool = True,
                   ws: Workspace | None = None):
    """{"dx": [T,d] BF16 or None, "dgates": [T,k] fp32, "dlogits": [T,E] fp32}: the
    router gradient through the frozen base (and the input gradient if want_dx)."""
    import torch
    T, d = dy.shape
    E = w_gate_up.E
    inter = w_gate_up.N // 2
    dev = dy.device
    dx = torch.empty((T, d), dtype=torch.bfloat16, device=dev) if want_dx else None
    dg = torch.empty((T, k), dtype=torch.float32, device=dev)
    dl = torch.empty((T, E), dtype=torch.float32, device=dev)
    nb, _ = workspace_bytes(CALL_DX_BWD, T, d, E, k, inter, variant, chunk)
    buf = (ws or _default_ws).get(nb, dev)
    g, dn, pc = w_gate_up.c(), w_down.c(), perm.c()
    _check(lib().moe_router_bwd(ctypes.byref(g), ctypes.byref(dn), _ptr(dy), _ptr(topk_ids),
                                _ptr(topk_gates), ctypes.byref(pc), _ptr(h_saved), T, d, E, k,
                                inter, variant, chunk, _ptr(buf), buf.numel(), _ptr(dx), _ptr(dg),
                                _ptr(dl), _stream()), "moe_router_bwd")
    return {"dx": dx, "dgates": dg, "dlogits": dl}


# ---- scored routing and 8-bit floating point -------------------------------

SCORES = {"softmax": 0, "sigmoid": 1}
SCALE_BLOCK = 128          # columns of a row, or rows and columns of a weight, per scale


def _need(name: str, t, dtypes, shape=None, device=None):
    """Raise unless t is a contiguous CUDA tensor of one of the dtypes, of the shape (-1: any)
    and on the device."""
    import torch
    if not isinstance(t, torch.Tensor):
        raise QggError(f"{name}: a tensor is needed, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise QggError(f"{name}: dtype {t.dtype}, want {' or '.join(map(str, dtypes))}")
    if shape is not None and (t.dim() != len(shape) or
                              any(w not in (-1, n) for n, w in zip(t.shape, shape))):
        raise QggError(f"{name}: shape {tuple(t.shape)}, want {tuple(shape)}")
    if not t.is_cuda:
        raise QggError(f"{name}: on {t.device}, want a GPU")
    if device is not None and t.device != device:
        raise QggError(f"{name}: on {t.device}, the call's other tensors are on {device}")
    if not t.is_contiguous():
        raise QggError(f"{name}: not contiguous")


class _On:
    """Makes a tensor's device current for a call (launches go to the current device) and gives
    that device's current stream.  The stream handle is read without a Stream object around it,
    whose making costs as much as a launch."""

    def __init__(self, device):
        import torch
        self.index = device.index
        self.guard = None
        if self.index != torch._C._cuda_getDevice():
            self.guard = torch.cuda.device(device)
        self.raw_stream = torch._C._cuda_getCurrentRawStream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        return self.raw_stream(self.index)

    def __exit__(self, *a):
        if self.guard is not None:
            self.guard.__exit__(*a)


def _at(t):
    return None if t is None else t.data_ptr()


def _need_perm(perm: Perm, P: int, device, E: int | None = None):
    import torch
    i32 = (torch.int32,)
    if E is None:
        E = perm.counts.numel()
    for name, n in (("counts", E), ("offsets", E + 1), ("active", E), ("n_active", 1),
                    ("perm", P), ("inv_perm", P)):
        t = getattr(perm, name)
        _need(f"perm.{name}", t, i32, None, device)
        if t.numel() != max(n, 1):
            raise QggError(f"perm.{name}: {t.numel()} entries, want {max(n, 1)}")


def _code_types():
    import torch
    return (torch.float8_e4m3fn, torch.uint8), (torch.float8_e8m0fnu, torch.uint8)


def _route_opts(score, n_group, topk_group, group_top, renorm, scale):
    if score not in SCORES:
        raise QggError(f"score {score!r}, want one of {sorted(SCORES)}")
    return _RouteOpts(SCORES[score], n_group, topk_group, group_top, int(bool(renorm)),
                      float(scale))


def moe_route_scored(logits, k: int, score: str = "sigmoid", bias=None, n_group: int = 1,
                     topk_group: int = 1, group_top: int = 2, renorm: bool = True,
                     scale: float = 1.0, err_flag=None):
    """(topk_ids int32 [T,k], topk_gates fp32 [T,k]) for fp32 or BF16 logits [T,E]: softmax or
    sigmoid scores, `bias` [E] fp32 added for the choice only, the `topk_group` best of
    `n_group` groups by the sum of their `group_top` best, gates renormalised and scaled."""
    import torch
    _need("logits", logits, (torch.float32, torch.bfloat16), (-1, -1))
    T, E = logits.shape
    dev = logits.device
    if bias is not None:
        _need("bias", bias, (torch.float32,), (E,), dev)
    if err_flag is not None:
        _need("err_flag", err_flag, (torch.int32,), (1,), dev)
    if n_group == 1:
        group_top = 1
    o = _route_opts(score, n_group, topk_group, group_top, renorm, scale)
    with _On(dev) as stream:
        ids = torch.empty((T, max(k, 0)), dtype=torch.int32, device=dev)
        gates = torch.empty((T, max(k, 0)), dtype=torch.float32, device=dev)
        _check(lib().moe_route_scored(_at(logits), int(logits.dtype == torch.bfloat16),
                                      _at(bias), T, E, k, ctypes.byref(o), _at(ids), _at(gates),
                                      _at(err_flag), stream), "moe_route_scored")
    return ids, gates


def moe_route_scored_bwd(logits, topk_ids, dgates, score: str = "sigmoid", renorm: bool = True,
                         scale: float = 1.0):
    """dlogits [T,E] (the logits' dtype) from dgates fp32 [T,k], the choice topk_ids held fixed."""
    import torch
    _need("logits", logits, (torch.float32, torch.bfloat16), (-1, -1))
    T, E = logits.shape
    dev = logits.device
    _need("topk_ids", topk_ids, (torch.int32,), (T, -1), dev)
    k = topk_ids.shape[1]
    _need("dgates", dgates, (torch.float32,), (T, k), dev)
    o = _route_opts(score, 1, 1, 1, renorm, scale)
    with _On(dev) as stream:
        dl = torch.empty_like(logits)
        _check(lib().moe_route_scored_bwd(_at(logits), int(logits.dtype == torch.bfloat16),
                                          _at(topk_ids), _at(dgates), T, E, k, ctypes.byref(o),
                                          _at(dl), stream), "moe_route_scored_bwd")
    return dl


def fp8_quantize(x):
    """(codes float8_e4m3fn [M,C], scales float8_e8m0fnu [M,ceil(C/128)]) of BF16 rows x [M,C]."""
    import torch
    _need("x", x, (torch.bfloat16,), (-1, -1))
    M, C = x.shape
    with _On(x.device) as stream:
        codes = torch.empty((M, C), dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty((M, -(-C // SCALE_BLOCK)), dtype=torch.float8_e8m0fnu,
                             device=x.device)
        _check(lib().qgg_fp8_quantize(_at(x), M, C, _at(codes), _at(scales), stream),
               "qgg_fp8_quantize")
    return codes, scales


def fp8_dequantize(codes, scales):
    """BF16 rows [M,C] from codes [M,C] and scales [M,ceil(C/128)]."""
    import torch
    ct, st = _code_types()
    _need("codes", codes, ct, (-1, -1))
    M, C = codes.shape
    _need("scales", scales, st, (M, -(-C // SCALE_BLOCK)), codes.device)
    with _On(codes.device) as stream:
        x = torch.empty((M, C), dtype=torch.bfloat16, device=codes.device)
        _check(lib().qgg_fp8_dequantize(_at(codes), _at(scales), M, C, _at(x), stream),
               "qgg_fp8_dequantize")
    return x


@dataclass
class Fp8Weight:
    """Frozen 8-bit expert weights on the device: E4M3 codes [E,N,K] (float8_e4m3fn or uint8) and
    a scale per 128 x 128 block [E,ceil(N/128),K/128] (float8_e8m0fnu or uint8: E8M0; float32)."""
    codes: "object"
    scales: "object"

    def __post_init__(self):
        import torch
        ct, st = _code_types()
        _need("codes", self.codes, ct, (-1, -1, -1))
        E, N, K = self.codes.shape
        if K % SCALE_BLOCK:
            raise QggError(f"codes: K = {K}, want a multiple of {SCALE_BLOCK}")
        _need("scales", self.scales, (*st, torch.float32),
              (E, -(-N // SCALE_BLOCK), K // SCALE_BLOCK), self.codes.device)

    @property
    def E(self):
        return self.codes.shape[0]

    @property
    def N(self):
        return self.codes.shape[1]

    @property
    def K(self):
        return self.codes.shape[2]

    def c(self):
        import torch
        return _Fp8Weight(self.E, self.N, self.K, int(self.scales.dtype == torch.float32),
                          self.codes.data_ptr(), self.scales.data_ptr())


def fp8_grouped_gemm(w: Fp8Weight, a, a_scales, perm: Perm, T: int, k: int, flags: int = A_TOKENS,
                     out=None):
    """y [P,N] BF16 in sorted order for 8-bit rows a, a_scales (fp8_quantize) of K columns, or
    [P,K] for rows of N columns with TRANSPOSE_W; T rows with A_TOKENS, else P = T k."""
    import torch
    ct, st = _code_types()
    trans = bool(flags & TRANSPOSE_W)
    red, cols = (w.N, w.K) if trans else (w.K, w.N)
    P = T * k
    rows = T if flags & A_TOKENS else P
    dev = w.codes.device
    _need("a", a, ct, (rows, red), dev)
    _need("a_scales", a_scales, st, (rows, -(-red // SCALE_BLOCK)), dev)
    _need_perm(perm, P, dev, w.E)
    if out is not None:
        _need("out", out, (torch.bfloat16,), (P, cols), dev)
    with _On(dev) as stream:
        y = out if out is not None else torch.empty((P, cols), dtype=torch.bfloat16, device=dev)
        wc, pc = w.c(), perm.c()
        _check(lib().fp8_grouped_gemm(ctypes.byref(wc), _at(a), _at(a_scales), flags,
                                      ctypes.byref(pc), T, k, _at(y), stream),
               "fp8_grouped_gemm")
    return y


def swiglu_fp8(h, perm: Perm | None = None, want=("a8", "h8")):
    """SwiGLU of routed rows h [P,2I] BF16: {"a": BF16 [P,I], "a8"/"a8_scales": the output in 8
    bits, "h8"/"h8_scales": the rows' 8-bit checkpoint}, those in `want`.  With `perm`, rows
    past the permutation's last are left as they are."""
    import torch
    _need("h", h, (torch.bfloat16,), (-1, -1))
    P, width = h.shape
    inter = width // 2
    if width != 2 * inter or not set(want) <= {"a", "a8", "h8"}:
        raise QggError(f"h: {width} columns, want an even number; want: {want}")
    dev = h.device
    if perm is not None:
        _need_perm(perm, P, dev)
    nb = -(-inter // SCALE_BLOCK)
    r = dict.fromkeys(("a", "a8", "a8_scales", "h8", "h8_scales"))
    with _On(dev) as stream:
        if "a" in want:
            r["a"] = torch.empty((P, inter), dtype=torch.bfloat16, device=dev)
        for name, n in (("a8", 1), ("h8", 2)):
            if name in want:
                r[name] = torch.empty((P, n * inter), dtype=torch.float8_e4m3fn, device=dev)
                r[name + "_scales"] = torch.empty((P, n * nb), dtype=torch.float8_e8m0fnu,
                                                  device=dev)
        live = None if perm is None else ctypes.c_void_p(
            perm.offsets.data_ptr() + 4 * (perm.offsets.numel() - 1))
        _check(lib().moe_swiglu_fp8(_at(h), live, P, inter, _at(r["a"]), _at(r["a8"]),
                                    _at(r["a8_scales"]), _at(r["h8"]), _at(r["h8_scales"]),
                                    stream), "moe_swiglu_fp8")
    return r


def swiglu_fp8_bwd(da, h8, h8_scales, topk_gates, perm: Perm, want=("dh8", "dgates")):
    """From the checkpoint h8 [P,2I] and da [P,I] BF16 (the gradient of the SwiGLU output before
    the gate): {"dh": BF16 [P,2I], "dh8"/"dh8_scales": the same in 8 bits, "dgates": fp32
    [T,k]}, those in `want`; topk_gates fp32 [T,k]."""
    import torch
    ct, st = _code_types()
    _need("topk_gates", topk_gates, (torch.float32,), (-1, -1))
    T, k = topk_gates.shape
    P = T * k
    dev = topk_gates.device
    _need("da", da, (torch.bfloat16,), (P, -1), dev)
    inter = da.shape[1]
    nb = -(-inter // SCALE_BLOCK)
    _need("h8", h8, ct, (P, 2 * inter), dev)
    _need("h8_scales", h8_scales, st, (P, 2 * nb), dev)
    _need_perm(perm, P, dev)
    if not set(want) <= {"dh", "dh8", "dgates"}:
        raise QggError(f"want: {want}")
    r = dict.fromkeys(("dh", "dh8", "dh8_scales", "dgates"))
    with _On(dev) as stream:
        if "dh" in want:
            r["dh"] = torch.empty((P, 2 * inter), dtype=torch.bfloat16, device=dev)
        if "dh8" in want:
            r["dh8"] = torch.empty((P, 2 * inter), dtype=torch.float8_e4m3fn, device=dev)
            r["dh8_scales"] = torch.empty((P, 2 * nb), dtype=torch.float8_e8m0fnu, device=dev)
        if "dgates" in want:
            r["dgates"] = torch.empty((T, k), dtype=torch.float32, device=dev)
        pc = perm.c()
        _check(lib().moe_swiglu_fp8_bwd(_at(da), _at(h8), _at(h8_scales), _at(topk_gates),
                                        ctypes.byref(pc), T, k, inter, _at(r["dh"]),
                                        _at(r["dh8"]), _at(r["dh8_scales"]), _at(r["dgates"]),
                                        stream), "moe_swiglu_fp8_bwd")
    return r


def moe_combine(rows, perm: Perm, T: int, k: int, topk_gates=None):
    """y [T,d] BF16: the sorted rows [P,d] of each token's pairs, weighted by topk_gates [T,k] (or
    summed)."""
    import torch
    _need("rows", rows, (torch.bfloat16,), (T * k, -1))
    dev = rows.device
    _need_perm(perm, T * k, dev)
    if topk_gates is not None:
        _need("topk_gates", topk_gates, (torch.float32,), (T, k), dev)
    d = rows.shape[1]
    with _On(dev) as stream:
        y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
        pc = perm.c()
        _check(lib().moe_combine(_at(rows), d, ctypes.byref(pc), _at(topk_gates), T, k, _at(y),
                                 stream), "moe_combine")
    return y
