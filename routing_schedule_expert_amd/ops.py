"""Python binding of the C ABI in include/moe.h (ctypes; argument marshalling only).

Every function has the name of its C entry point and takes torch tensors for
the device buffers; the stream defaults to torch's current stream on the
tensors' device.  Each call returns after the launch (asynchronous) and raises
``MoeError`` if the library returns a negative code.  Every step of the layer
runs in the HIP library; if ``libmoe.so`` is missing or a device pointer is not
a CUDA(HIP) tensor, the call fails loudly - there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_EINVAL, MOE_ENOSPC, MOE_EUNSUPPORTED, MOE_EHIP = 0, -1, -2, -3, -4
(MOE_OP_SCHEDULE, MOE_OP_DISPATCH, MOE_OP_EXPERT_FFN, MOE_OP_COMBINE, MOE_OP_LAYER_FWD, MOE_OP_LAYER_BWD,
 MOE_OP_LAYER_FWD_SHARED, MOE_OP_LAYER_BWD_MX, MOE_OP_LAYER_BWD_CKPT) = range(9)
MOE_PERSISTENT = 1
MOE_WS_INVALID_IDS, MOE_WS_BARRIER_STATUS = 0, 1
(MOE_WS_MX_DHU, MOE_WS_MX_DO_Q, MOE_WS_MX_DO_S, MOE_WS_MX_DHU_Q, MOE_WS_MX_DHU_S, MOE_WS_MX_DOWT_Q, MOE_WS_MX_DOWT_S,
 MOE_WS_MX_AT_Q, MOE_WS_MX_AT_S, MOE_WS_MX_XDT_Q, MOE_WS_MX_XDT_S, MOE_WS_MX_DHUT_Q, MOE_WS_MX_DHUT_S) = range(2, 15)
MOE_WS_SINGLE_ROUTE = 15
MOE_GATE_NONE, MOE_GATE_TOKEN, MOE_GATE_ELEM = range(3)
CKPT_BLOCK = 128
MOE_TYPE_BF16, MOE_TYPE_FP16, MOE_TYPE_FP32 = range(3)
MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_GELU_TANH, MOE_ACT_RELU = range(4)
MOE_NORM_L2, MOE_NORM_MAX = range(2)

EXPORTED = (
    "moe_strerror", "moe_capacity_rows", "moe_workspace_bytes", "moe_workspace_field", "moe_schedule",
    "moe_dispatch",
    "moe_expert_ffn", "moe_combine", "moe_layer_fwd", "moe_layer_bwd", "moe_trace_enable", "moe_trace_read",
    "moe_quantize_mx", "moe_quantize_mx_t",
    "moe_layer_fwd_mx", "moe_layer_bwd_mx",
    "moe_ring_capacity_rows", "moe_ring_workspace_bytes", "moe_layer_fwd_ring", "moe_layer_bwd_ring",
    "moe_layer_fwd_shared", "moe_layer_fwd_noalloc",
    "moe_few_workspace_bytes", "moe_layer_fwd_few", "moe_layer_fwd_few_mx",
    "moe_block_norm_workspace_bytes", "moe_block_norm_fwd", "moe_block_norm_bwd",
    "moe_ckpt_pack", "moe_ckpt_swiglu_bwd", "moe_layer_bwd_ckpt",
    "moe_gated_ffn_workspace_bytes", "moe_gated_ffn_fwd", "moe_gated_ffn_bwd",
    "moe_layer_norm_workspace_bytes", "moe_layer_norm_fwd", "moe_layer_norm_bwd",
    "moe_grad_workspace_bytes", "moe_grad_norm", "moe_grad_clip", "moe_grad_scale",
)
MOE_NOALLOC_SCRATCH_BYTES = 8 << 20


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {strerror(code)} ({code})")
        self.code = code


class moe_desc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("P", "Np", "K", "E", "L", "expert_base", "pad_rows", "sched_threads", "H", "I", "num_batches")]


class moe_norm_desc(ctypes.Structure):
    _fields_ = ([("rows", ctypes.c_int64)] + [(n, ctypes.c_int32) for n in ("H", "gate", "res_fp32")] +
                [(n, ctypes.c_float) for n in ("alpha", "beta", "eps")])


class moe_ffn_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "ldx", "ldo")] + [(n, ctypes.c_int32) for n in ("H", "I", "act", "type")])


class moe_ln_desc(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("rows", "ldx", "ldy")] +
                [(n, ctypes.c_int32) for n in ("H", "x_type", "y_type")] + [("eps", ctypes.c_float)])


class moe_grad(ctypes.Structure):
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("numel", ctypes.c_int64), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


def make_desc(P, Np, K, E, L=None, expert_base=0, pad_rows=256, sched_threads=1024, H=0, I=0, num_batches=1):
    if L is None:
        L = E // P
    return moe_desc(P, Np, K, E, L, expert_base, pad_rows, sched_threads, H, I, num_batches)


_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree HIP library (fails loudly when it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with routing_schedule_expert_amd/build.py "
                          "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(LIB_PATH)
    P, D, N = ctypes.c_void_p, ctypes.POINTER(moe_desc), ctypes.POINTER(moe_norm_desc)
    F, LN, G = ctypes.POINTER(moe_ffn_desc), ctypes.POINTER(moe_ln_desc), ctypes.POINTER(moe_grad)
    i32, i64, sz, f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "moe_strerror": (ctypes.c_char_p, [ctypes.c_int]),
        "moe_capacity_rows": (i64, [D]),
        "moe_workspace_bytes": (i64, [D, ctypes.c_int]),
        "moe_workspace_field": (i64, [D, ctypes.c_int, ctypes.c_int]),
        "moe_schedule": (ctypes.c_int, [D, P, P, P, P, P, P, sz, P]),
        "moe_dispatch": (ctypes.c_int, [D, P, P, P, P, P]),
        "moe_expert_ffn": (ctypes.c_int, [D, P, P, P, P, P, P, P, i32, P, sz, P]),
        "moe_combine": (ctypes.c_int, [D, P, P, P, P, P]),
        "moe_layer_fwd": (ctypes.c_int, [D] + [P] * 14 + [i32, i32, P, sz, P]),
        "moe_layer_fwd_noalloc": (ctypes.c_int, [D] + [P] * 14 + [i32, i32, P, P]),
        "moe_quantize_mx": (ctypes.c_int, [P, i64, i32, P, P, P]),
        "moe_quantize_mx_t": (ctypes.c_int, [P, i64, i32, i32, P, P, P]),
        "moe_layer_fwd_mx": (ctypes.c_int, [D] + [P] * 19 + [sz, P]),
        "moe_layer_bwd_mx": (ctypes.c_int, [D] + [P] * 18 + [sz, P]),
        "moe_layer_bwd": (ctypes.c_int, [D] + [P] * 16 + [sz, P]),
        "moe_layer_fwd_shared": (ctypes.c_int, [D, i32] + [P] * 19 + [sz, P]),
        "moe_ring_capacity_rows": (i64, [D, i32]),
        "moe_ring_workspace_bytes": (i64, [D, i32, i32, ctypes.c_int]),
        "moe_layer_fwd_ring": (ctypes.c_int, [D, i32, i32] + [P] * 14 + [sz, P]),
        "moe_layer_bwd_ring": (ctypes.c_int, [D, i32, i32, i32] + [P] * 15 + [sz, P]),
        "moe_few_workspace_bytes": (i64, [D, i32]),
        "moe_layer_fwd_few": (ctypes.c_int, [D, i32] + [P] * 9 + [sz, P]),
        "moe_layer_fwd_few_mx": (ctypes.c_int, [D, i32] + [P] * 11 + [sz, P]),
        "moe_block_norm_workspace_bytes": (i64, [N]),
        "moe_block_norm_fwd": (ctypes.c_int, [N] + [P] * 9),
        "moe_block_norm_bwd": (ctypes.c_int, [N] + [P] * 14 + [sz, P]),
        "moe_ckpt_pack": (ctypes.c_int, [P, i64, i32, P, P, P, P]),
        "moe_ckpt_swiglu_bwd": (ctypes.c_int, [P, P, P, P, i64, i32, P, P, P, P, P]),
        "moe_layer_bwd_ckpt": (ctypes.c_int, [D] + [P] * 15 + [sz, P]),
        "moe_gated_ffn_workspace_bytes": (i64, [F, i32]),
        "moe_gated_ffn_fwd": (ctypes.c_int, [F] + [P] * 7 + [sz, P]),
        "moe_gated_ffn_bwd": (ctypes.c_int, [F] + [P] * 9 + [i32, i32, P, sz, P]),
        "moe_layer_norm_workspace_bytes": (i64, [LN]),
        "moe_layer_norm_fwd": (ctypes.c_int, [LN] + [P] * 6),
        "moe_layer_norm_bwd": (ctypes.c_int, [LN] + [P] * 9 + [sz, P]),
        "moe_grad_workspace_bytes": (i64, [i32]),
        "moe_grad_norm": (ctypes.c_int, [G, i32, i32, f32, f32, f32, P, P, sz, P]),
        "moe_grad_clip": (ctypes.c_int, [G, i32, i32, f32, f32, f32, P, P, sz, P]),
        "moe_grad_scale": (ctypes.c_int, [G, i32, P, f32, P]),
        "moe_trace_enable": (ctypes.c_int, [ctypes.c_int]),
        "moe_trace_read": (ctypes.c_int, [P, P, ctypes.c_int]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def strerror(code: int) -> str:
    return load().moe_strerror(code).decode()


def _check(rc: int, where: str) -> int:
    if rc != MOE_OK:
        raise MoeError(rc, where)
    return rc


def _dev(t):
    """Device pointer of a CUDA(HIP) tensor, or NULL for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("device buffers must be CUDA (HIP) torch tensors")
    if not t.is_contiguous():
        raise ValueError("device buffers must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _buf(name: str, t, dtype, n: int, dev: int):
    """Device pointer of a tensor that the call will touch n elements of: on GPU
    `dev`, contiguous, of dtype, at least that large; None stays NULL."""
    if t is None:
        return None
    if t.dtype != dtype or t.get_device() != dev or t.numel() < n or not t.is_contiguous():
        _dev(t)
        raise ValueError(f"{name}: needs {n} elements of {dtype} on cuda:{dev}, got {t.numel()} of {t.dtype} on {t.device}")
    return t.data_ptr()


def _run(where: str, dev: int, stream, *args) -> int:
    """Calls entry point `where` with GPU `dev` current, on `stream` or that
    device's current stream."""
    if dev < 0:
        raise TypeError("device buffers must be CUDA (HIP) torch tensors")
    if stream is not None and stream.device_index != dev:
        raise ValueError(f"{where}: the stream is on cuda:{stream.device_index}, the buffers on cuda:{dev}")
    fn = getattr(_lib or load(), where)
    stream = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == dev:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    return _check(rc, where)


def _stream(stream, ref: torch.Tensor):
    if stream is None:
        stream = torch.cuda.current_stream(ref.device)
    return ctypes.c_void_p(stream.cuda_stream)


def capacity_rows(d: moe_desc) -> int:
    n = load().moe_capacity_rows(ctypes.byref(d))
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_capacity_rows")
    return int(n)


def workspace_bytes(d: moe_desc, op: int) -> int:
    n = load().moe_workspace_bytes(ctypes.byref(d), op)
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_workspace_bytes")
    return int(n)


def workspace_field(d: moe_desc, op: int, field: int) -> int:
    """Byte offset of a status word (MOE_WS_*) in op's workspace; -1 if op has none."""
    return int(load().moe_workspace_field(ctypes.byref(d), op, field))


def read_ws_words(ws: torch.Tensor, offset: int, n: int = 1) -> list:
    """The n int32 words at byte `offset` of a workspace tensor (synchronises
    the tensor's stream by copying to the host)."""
    if offset < 0:
        raise ValueError("no such workspace field")
    return [int(v) for v in ws[offset:offset + 4 * n].cpu().view(torch.int32).tolist()]


def moe_schedule(d, routes, counts, seg_off, phi, route_row, ws, stream=None):
    rc = load().moe_schedule(ctypes.byref(d), _dev(routes), _dev(counts), _dev(seg_off), _dev(phi), _dev(route_row),
                             _dev(ws), ws.numel() * ws.element_size(), _stream(stream, routes))
    return _check(rc, "moe_schedule")


def moe_dispatch(d, X, phi, seg_off, Xd, stream=None):
    rc = load().moe_dispatch(ctypes.byref(d), _dev(X), _dev(phi), _dev(seg_off), _dev(Xd), _stream(stream, X))
    return _check(rc, "moe_dispatch")


def moe_expert_ffn(d, Xd, W13, W2, seg_off, HU, A, Y, chunk_rows=0, ws=None, stream=None):
    rc = load().moe_expert_ffn(ctypes.byref(d), _dev(Xd), _dev(W13), _dev(W2), _dev(seg_off), _dev(HU), _dev(A),
                               _dev(Y), chunk_rows, _dev(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                               _stream(stream, Xd))
    return _check(rc, "moe_expert_ffn")


def moe_combine(d, Y, route_row, w, out, stream=None):
    rc = load().moe_combine(ctypes.byref(d), _dev(Y), _dev(route_row), _dev(w), _dev(out), _stream(stream, Y))
    return _check(rc, "moe_combine")


def moe_layer_fwd(d, routes, w, X, W13, W2, counts, seg_off, phi, route_row, Xd, HU, A, Y, out, flags=0,
                  chunk_rows=0, ws=None, stream=None):
    rc = load().moe_layer_fwd(ctypes.byref(d), _dev(routes), _dev(w), _dev(X), _dev(W13), _dev(W2), _dev(counts),
                              _dev(seg_off), _dev(phi), _dev(route_row), _dev(Xd), _dev(HU), _dev(A), _dev(Y),
                              _dev(out), flags, chunk_rows, _dev(ws), ws.numel() * ws.element_size(),
                              _stream(stream, X))
    return _check(rc, "moe_layer_fwd")


def moe_layer_fwd_noalloc(d, routes, w, X, W13, W2, counts, seg_off, phi, route_row, Xd, HU, A, Y, out, flags=0,
                          chunk_rows=0, status=None, stream=None):
    rc = load().moe_layer_fwd_noalloc(ctypes.byref(d), _dev(routes), _dev(w), _dev(X), _dev(W13), _dev(W2),
                                      _dev(counts), _dev(seg_off), _dev(phi), _dev(route_row), _dev(Xd), _dev(HU),
                                      _dev(A), _dev(Y), _dev(out), flags, chunk_rows, _dev(status),
                                      _stream(stream, X))
    return _check(rc, "moe_layer_fwd_noalloc")


def moe_layer_bwd(d, dOut, routes, w, phi, route_row, seg_off, Xd, HU, A, W13, W2, dX, dW13, dW2, dw, ws,
                  stream=None):
    rc = load().moe_layer_bwd(ctypes.byref(d), _dev(dOut), _dev(routes), _dev(w), _dev(phi), _dev(route_row),
                              _dev(seg_off), _dev(Xd), _dev(HU), _dev(A), _dev(W13), _dev(W2), _dev(dX), _dev(dW13),
                              _dev(dW2), _dev(dw), _dev(ws), ws.numel() * ws.element_size(), _stream(stream, dOut))
    return _check(rc, "moe_layer_bwd")


def moe_trace_enable(max_records: int) -> None:
    _check(load().moe_trace_enable(max_records), "moe_trace_enable")


def moe_trace_read(max_records: int = 4096):
    """[(kernel name, ms)] of the recorded launches (synchronise first)."""
    names = ctypes.create_string_buffer(32 * max_records)
    ms = (ctypes.c_float * max_records)()
    n = load().moe_trace_read(names, ms, max_records)
    return [(names.raw[32 * i:32 * i + 32].split(b"\0", 1)[0].decode(), float(ms[i])) for i in range(n)]


# ---------------------------------------------------------------------------
# Buffer helpers (device memory via torch; no arithmetic).
# ---------------------------------------------------------------------------

@dataclass
class FwdBuffers:
    counts: torch.Tensor
    seg_off: torch.Tensor
    phi: torch.Tensor
    route_row: torch.Tensor
    Xd: torch.Tensor | None
    HU: torch.Tensor | None
    A: torch.Tensor
    Y: torch.Tensor
    out: torch.Tensor
    ws: torch.Tensor


def alloc_fwd(d: moe_desc, device, save_hu: bool = True, save_xd: bool = True) -> FwdBuffers:
    """Forward buffers.  save_xd=False leaves Xd out: moe_layer_fwd then pulls
    the gate/up rows straight from X (the dispatch fused into the GEMM loads)."""
    cap = capacity_rows(d)
    i32, bf = torch.int32, torch.bfloat16
    return FwdBuffers(
        counts=torch.empty((d.L, d.P), dtype=i32, device=device),
        seg_off=torch.empty(d.L + 1, dtype=i32, device=device),
        phi=torch.empty((cap, 2), dtype=i32, device=device),
        route_row=torch.empty((d.P, d.Np, d.K), dtype=i32, device=device),
        Xd=torch.empty((cap, d.H), dtype=bf, device=device) if save_xd else None,
        HU=torch.empty((cap, 2 * d.I), dtype=bf, device=device) if save_hu else None,
        A=torch.empty((cap, d.I), dtype=bf, device=device),
        Y=torch.empty((cap, d.H), dtype=bf, device=device),
        out=torch.empty((d.P, d.Np, d.H), dtype=bf, device=device),
        ws=torch.empty(max(workspace_bytes(d, MOE_OP_LAYER_FWD), 256), dtype=torch.uint8, device=device),
    )


def layer_fwd(d, routes, w, X, W13, W2, bufs: FwdBuffers, flags=0, chunk_rows=0, stream=None):
    return moe_layer_fwd(d, routes, w, X, W13, W2, bufs.counts, bufs.seg_off, bufs.phi, bufs.route_row, bufs.Xd,
                         bufs.HU, bufs.A, bufs.Y, bufs.out, flags, chunk_rows, bufs.ws, stream)


# ---------------------------------------------------------------------------
# MXFP8 routed experts.
# ---------------------------------------------------------------------------

def moe_quantize_mx(src, q, scales, stream=None):
    """Row-wise MX quantization of a bf16 tensor [..., K] into codes (uint8,
    same shape) and scale bytes (uint8 [..., K/32])."""
    K = src.shape[-1]
    rows = src.numel() // K if K else 0
    rc = load().moe_quantize_mx(_dev(src), rows, K, _dev(q), _dev(scales), _stream(stream, src))
    return _check(rc, "moe_quantize_mx")


def quantize_mx(src, stream=None):
    """Allocate and fill (codes, scales) for a bf16 tensor [..., K]."""
    q = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    s = torch.empty(src.shape[:-1] + (src.shape[-1] // 32,), dtype=torch.uint8, device=src.device)
    moe_quantize_mx(src, q, s, stream)
    return q, s


def moe_quantize_mx_t(src, q, scales, stream=None):
    """MX quantization of the columns of bf16 [..., R, C] along R into codes
    uint8 [..., C, R] and scale bytes uint8 [..., C, R/32]."""
    R, C = src.shape[-2], src.shape[-1]
    batch = src.numel() // (R * C) if R * C else 0
    rc = load().moe_quantize_mx_t(_dev(src), batch, R, C, _dev(q), _dev(scales), _stream(stream, src))
    return _check(rc, "moe_quantize_mx_t")


def quantize_mx_t(src, stream=None):
    """Allocate and fill (codes, scales) of src's columns along its rows."""
    R, C = src.shape[-2], src.shape[-1]
    q = torch.empty(src.shape[:-2] + (C, R), dtype=torch.uint8, device=src.device)
    s = torch.empty(src.shape[:-2] + (C, R // 32), dtype=torch.uint8, device=src.device)
    moe_quantize_mx_t(src, q, s, stream)
    return q, s


def moe_layer_fwd_mx(d, routes, w, X, W13q, W13s, W2q, W2s, counts, seg_off, phi, route_row, Xq, Xs, Aq, As, HU, Y,
                     out, ws, stream=None):
    rc = load().moe_layer_fwd_mx(ctypes.byref(d), _dev(routes), _dev(w), _dev(X), _dev(W13q), _dev(W13s), _dev(W2q),
                                 _dev(W2s), _dev(counts), _dev(seg_off), _dev(phi), _dev(route_row), _dev(Xq),
                                 _dev(Xs), _dev(Aq), _dev(As), _dev(HU), _dev(Y), _dev(out), _dev(ws),
                                 ws.numel() * ws.element_size(), _stream(stream, X))
    return _check(rc, "moe_layer_fwd_mx")


def moe_layer_bwd_mx(d, dOut, w, X, phi, route_row, seg_off, HU, Aq, As, W13tq, W13ts, W2tq, W2ts, dX, dW13, dW2, dw,
                     ws, stream=None):
    rc = load().moe_layer_bwd_mx(ctypes.byref(d), _dev(dOut), _dev(w), _dev(X), _dev(phi), _dev(route_row),
                                 _dev(seg_off), _dev(HU), _dev(Aq), _dev(As), _dev(W13tq), _dev(W13ts), _dev(W2tq),
                                 _dev(W2ts), _dev(dX), _dev(dW13), _dev(dW2), _dev(dw), _dev(ws),
                                 ws.numel() * ws.element_size(), _stream(stream, dOut))
    return _check(rc, "moe_layer_bwd_mx")


@dataclass
class MxFwdBuffers:
    counts: torch.Tensor
    seg_off: torch.Tensor
    phi: torch.Tensor
    route_row: torch.Tensor
    Xq: torch.Tensor
    Xs: torch.Tensor
    Aq: torch.Tensor
    As: torch.Tensor
    HU: torch.Tensor | None
    Y: torch.Tensor
    out: torch.Tensor
    ws: torch.Tensor


def alloc_fwd_mx(d: moe_desc, device, save_hu: bool = False) -> MxFwdBuffers:
    """MX forward buffers; save_hu keeps h and u (bf16) for moe_layer_bwd_mx."""
    cap = capacity_rows(d)
    i32, u8 = torch.int32, torch.uint8
    ntok = d.P * d.Np
    return MxFwdBuffers(
        counts=torch.empty((d.L, d.P), dtype=i32, device=device),
        seg_off=torch.empty(d.L + 1, dtype=i32, device=device),
        phi=torch.empty((cap, 2), dtype=i32, device=device),
        route_row=torch.empty((d.P, d.Np, d.K), dtype=i32, device=device),
        Xq=torch.empty((d.P, d.Np, d.H), dtype=u8, device=device),
        Xs=torch.empty((d.P, d.Np, d.H // 32), dtype=u8, device=device),
        Aq=torch.empty((cap, d.I), dtype=u8, device=device),
        As=torch.empty((cap, d.I // 32), dtype=u8, device=device),
        HU=torch.empty((cap, 2 * d.I), dtype=torch.bfloat16, device=device) if save_hu else None,
        Y=torch.empty((cap, d.H), dtype=torch.bfloat16, device=device),
        out=torch.empty((d.P, d.Np, d.H), dtype=torch.bfloat16, device=device),
        ws=torch.empty(max(workspace_bytes(d, MOE_OP_LAYER_FWD), 256), dtype=torch.uint8, device=device),
    )


def layer_fwd_mx(d, routes, w, X, W13q, W13s, W2q, W2s, bufs: MxFwdBuffers, stream=None):
    return moe_layer_fwd_mx(d, routes, w, X, W13q, W13s, W2q, W2s, bufs.counts, bufs.seg_off, bufs.phi,
                            bufs.route_row, bufs.Xq, bufs.Xs, bufs.Aq, bufs.As, bufs.HU, bufs.Y, bufs.out, bufs.ws,
                            stream)


@dataclass
class MxBwdGrads:
    dX: torch.Tensor
    dW13: torch.Tensor
    dW2: torch.Tensor
    dw: torch.Tensor
    ws: torch.Tensor


def alloc_bwd_mx(d: moe_desc, device) -> MxBwdGrads:
    return MxBwdGrads(
        dX=torch.empty((d.P, d.Np, d.H), dtype=torch.bfloat16, device=device),
        dW13=torch.empty((d.L, 2 * d.I, d.H), dtype=torch.float32, device=device),
        dW2=torch.empty((d.L, d.H, d.I), dtype=torch.float32, device=device),
        dw=torch.empty((d.P, d.Np, d.K), dtype=torch.float32, device=device),
        ws=torch.empty(workspace_bytes(d, MOE_OP_LAYER_BWD_MX), dtype=torch.uint8, device=device),
    )


def mx_bwd_views(d: moe_desc, ws: torch.Tensor) -> dict:
    """Views of moe_layer_bwd_mx's workspace buffers (the MOE_WS_MX_* fields):
    dHU bf16 [cap][2I]; row codes / scales (DO, DHU) [cap][C] / [cap][C/32];
    the column codes (DOWT, AT, XDT, DHUT) as flat (codes, scales) byte
    tensors, segment-major (mx_expert_block cuts one expert's block out)."""
    cap = capacity_rows(d)
    H, I2 = d.H, 2 * d.I

    def at(field, nbytes):
        off = workspace_field(d, MOE_OP_LAYER_BWD_MX, field)
        return ws[off:off + nbytes]

    v = {"dHU": at(MOE_WS_MX_DHU, cap * I2 * 2).view(torch.bfloat16).view(cap, I2)}
    for nm, f, C in (("DO", MOE_WS_MX_DO_Q, H), ("DHU", MOE_WS_MX_DHU_Q, I2)):
        v[nm] = (at(f, cap * C).view(cap, C), at(f + 1, cap * C // 32).view(cap, C // 32))
    for nm, f, C in (("DOWT", MOE_WS_MX_DOWT_Q, H), ("AT", MOE_WS_MX_AT_Q, d.I), ("XDT", MOE_WS_MX_XDT_Q, H),
                     ("DHUT", MOE_WS_MX_DHUT_Q, I2)):
        v[nm] = (at(f, cap * C), at(f + 1, cap * C // 32), C)
    return v


def mx_expert_block(view, S: int, n: int):
    """(codes [C][n], scales [C][n/32]) of the expert whose rows are [S, S+n)
    in a segment-major column-code view of mx_bwd_views."""
    q, s, C = view
    return q[C * S:C * (S + n)].view(C, n), s[C * S // 32:C * (S + n) // 32].view(C, n // 32)


def layer_bwd_mx(d, dOut, w, X, fwd: MxFwdBuffers, W13t, W2t, g: MxBwdGrads, stream=None):
    """moe_layer_bwd_mx on a forward's buffers; W13t / W2t are the (codes,
    scales) of quantize_mx_t(W13) and quantize_mx_t(W2)."""
    return moe_layer_bwd_mx(d, dOut, w, X, fwd.phi, fwd.route_row, fwd.seg_off, fwd.HU, fwd.Aq, fwd.As, W13t[0],
                            W13t[1], W2t[0], W2t[1], g.dX, g.dW13, g.dW2, g.dw, g.ws, stream)


# ---------------------------------------------------------------------------
# Macrobatch ring.
# ---------------------------------------------------------------------------

def ring_capacity_rows(d: moe_desc, mb_tokens: int) -> int:
    n = load().moe_ring_capacity_rows(ctypes.byref(d), mb_tokens)
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_ring_capacity_rows")
    return int(n)


def ring_workspace_bytes(d: moe_desc, mb_tokens: int, op: int, wgrad_group: int = 1) -> int:
    n = load().moe_ring_workspace_bytes(ctypes.byref(d), mb_tokens, wgrad_group, op)
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_ring_workspace_bytes")
    return int(n)


def moe_layer_fwd_ring(d, mb_tokens, ring_slots, routes, w, X, W13, W2, counts, seg_off, phi, route_row, HU, A, Y,
                       out, ws, stream=None):
    rc = load().moe_layer_fwd_ring(ctypes.byref(d), mb_tokens, ring_slots, _dev(routes), _dev(w), _dev(X), _dev(W13),
                                   _dev(W2), _dev(counts), _dev(seg_off), _dev(phi), _dev(route_row), _dev(HU),
                                   _dev(A), _dev(Y), _dev(out), _dev(ws), ws.numel() * ws.element_size(),
                                   _stream(stream, X))
    return _check(rc, "moe_layer_fwd_ring")


def moe_layer_bwd_ring(d, mb_tokens, ring_slots, dOut, w, X, W13, W2, phi, route_row, seg_off, HU, A, dX, dW13, dW2,
                       dw, ws, stream=None, wgrad_group=1):
    rc = load().moe_layer_bwd_ring(ctypes.byref(d), mb_tokens, ring_slots, wgrad_group, _dev(dOut), _dev(w), _dev(X),
                                   _dev(W13),
                                   _dev(W2), _dev(phi), _dev(route_row), _dev(seg_off), _dev(HU), _dev(A), _dev(dX),
                                   _dev(dW13), _dev(dW2), _dev(dw), _dev(ws), ws.numel() * ws.element_size(),
                                   _stream(stream, dOut))
    return _check(rc, "moe_layer_bwd_ring")


@dataclass
class RingBuffers:
    mb_tokens: int
    slots: int
    counts: torch.Tensor     # [M][L][P]
    seg_off: torch.Tensor    # [M][L+1]
    phi: torch.Tensor        # [M][capm][2]
    route_row: torch.Tensor  # [P][Np][K]
    HU: torch.Tensor         # [slots][capm][2I]
    A: torch.Tensor          # [slots][capm][I]
    Y: torch.Tensor          # [capm][H]
    out: torch.Tensor
    ws: torch.Tensor


def alloc_ring(d: moe_desc, mb_tokens: int, slots: int, device) -> RingBuffers:
    capm = ring_capacity_rows(d, mb_tokens)
    M = d.Np // mb_tokens
    i32, bf = torch.int32, torch.bfloat16
    return RingBuffers(
        mb_tokens=mb_tokens, slots=slots,
        counts=torch.empty((M, d.L, d.P), dtype=i32, device=device),
        seg_off=torch.empty((M, d.L + 1), dtype=i32, device=device),
        phi=torch.empty((M, capm, 2), dtype=i32, device=device),
        route_row=torch.empty((d.P, d.Np, d.K), dtype=i32, device=device),
        HU=torch.empty((slots, capm, 2 * d.I), dtype=bf, device=device),
        A=torch.empty((slots, capm, d.I), dtype=bf, device=device),
        Y=torch.empty((capm, d.H), dtype=bf, device=device),
        out=torch.empty((d.P, d.Np, d.H), dtype=bf, device=device),
        ws=torch.empty(max(ring_workspace_bytes(d, mb_tokens, MOE_OP_LAYER_FWD), 256), dtype=torch.uint8,
                       device=device),
    )


def layer_fwd_ring(d, routes, w, X, W13, W2, r: RingBuffers, stream=None):
    return moe_layer_fwd_ring(d, r.mb_tokens, r.slots, routes, w, X, W13, W2, r.counts, r.seg_off, r.phi,
                              r.route_row, r.HU, r.A, r.Y, r.out, r.ws, stream)


# ---------------------------------------------------------------------------
# Shared expert.
# ---------------------------------------------------------------------------

def moe_layer_fwd_shared(d, Is, routes, w, X, W13, W2, W13s, W2s, counts, seg_off, phi, route_row, HU, A, Y, HUs, As,
                         Ys, out, ws, stream=None):
    rc = load().moe_layer_fwd_shared(ctypes.byref(d), Is, _dev(routes), _dev(w), _dev(X), _dev(W13), _dev(W2),
                                     _dev(W13s), _dev(W2s), _dev(counts), _dev(seg_off), _dev(phi), _dev(route_row),
                                     _dev(HU), _dev(A), _dev(Y), _dev(HUs), _dev(As), _dev(Ys), _dev(out), _dev(ws),
                                     ws.numel() * ws.element_size(), _stream(stream, X))
    return _check(rc, "moe_layer_fwd_shared")


@dataclass
class SharedBuffers:
    Is: int
    HUs: torch.Tensor | None
    As: torch.Tensor
    Ys: torch.Tensor
    ws: torch.Tensor


def alloc_shared(d: moe_desc, Is: int, device, save_hu: bool = False) -> SharedBuffers:
    ntokp = (d.P * d.Np + 255) // 256 * 256
    bf = torch.bfloat16
    return SharedBuffers(
        Is=Is,
        HUs=torch.empty((ntokp, 2 * Is), dtype=bf, device=device) if save_hu else None,
        As=torch.empty((ntokp, Is), dtype=bf, device=device),
        Ys=torch.empty((ntokp, d.H), dtype=bf, device=device),
        ws=torch.empty(workspace_bytes(d, MOE_OP_LAYER_FWD_SHARED), dtype=torch.uint8, device=device),
    )


def layer_fwd_shared(d, routes, w, X, W13, W2, W13s, W2s, bufs: FwdBuffers, sh: SharedBuffers, stream=None):
    """Forward with a shared expert; bufs.Xd is not used (fused dispatch)."""
    return moe_layer_fwd_shared(d, sh.Is, routes, w, X, W13, W2, W13s, W2s, bufs.counts, bufs.seg_off, bufs.phi,
                                bufs.route_row, bufs.HU, bufs.A, bufs.Y, sh.HUs, sh.As, sh.Ys, bufs.out, sh.ws, stream)


# ---------------------------------------------------------------------------
# The layer forward for a few tokens.
# ---------------------------------------------------------------------------

def few_workspace_bytes(d: moe_desc, Is: int = 0) -> int:
    n = load().moe_few_workspace_bytes(ctypes.byref(d), Is)
    if n < 0:
        raise MoeError(MOE_EINVAL, "moe_few_workspace_bytes")
    return int(n)


def _few_args(d, Is, routes, w, X, S13, S2, out, ws):
    n, H, i32, f32, bf, dev = d.P * d.Np, d.H, torch.int32, torch.float32, torch.bfloat16, X.get_device()
    return ([_buf("routes", routes, i32, n * d.K, dev), _buf("w", w, f32, n * d.K, dev), _buf("X", X, bf, n * H, dev)],
            [_buf("S13", S13, bf, 2 * Is * H, dev), _buf("S2", S2, bf, Is * H, dev), _buf("out", out, bf, n * H, dev),
             _buf("ws", ws, torch.uint8, 0, dev), 0 if ws is None else ws.numel()])


def moe_layer_fwd_few(d, Is, routes, w, X, W13, W2, S13, S2, out, ws, stream=None):
    head, tail = _few_args(d, Is, routes, w, X, S13, S2, out, ws)
    n, bf, dev = d.L * d.I * d.H, torch.bfloat16, X.get_device()
    return _run("moe_layer_fwd_few", dev, stream, ctypes.byref(d), Is, *head, _buf("W13", W13, bf, 2 * n, dev),
                _buf("W2", W2, bf, n, dev), *tail)


def moe_layer_fwd_few_mx(d, Is, routes, w, X, W13q, W13s, W2q, W2s, S13, S2, out, ws, stream=None):
    head, tail = _few_args(d, Is, routes, w, X, S13, S2, out, ws)
    n, u8, dev = d.L * d.I * d.H, torch.uint8, X.get_device()
    return _run("moe_layer_fwd_few_mx", dev, stream, ctypes.byref(d), Is, *head, _buf("W13q", W13q, u8, 2 * n, dev),
                _buf("W13s", W13s, u8, 2 * n // 32, dev), _buf("W2q", W2q, u8, n, dev), _buf("W2s", W2s, u8, n // 32, dev), *tail)


@dataclass
class FewBuffers:
    Is: int
    out: torch.Tensor
    ws: torch.Tensor


def alloc_few(d: moe_desc, device, Is: int = 0) -> FewBuffers:
    """Output and workspace of the few-token forwards (Is: the shared expert's
    intermediate size, 0 without one)."""
    return FewBuffers(
        Is=Is,
        out=torch.empty((d.P, d.Np, d.H), dtype=torch.bfloat16, device=device),
        ws=torch.empty(few_workspace_bytes(d, Is), dtype=torch.uint8, device=device),
    )


def layer_fwd_few(d, routes, w, X, W13, W2, bufs: FewBuffers, S13=None, S2=None, stream=None):
    return moe_layer_fwd_few(d, bufs.Is, routes, w, X, W13, W2, S13, S2, bufs.out, bufs.ws, stream)


def layer_fwd_few_mx(d, routes, w, X, W13q, W13s, W2q, W2s, bufs: FewBuffers, S13=None, S2=None, stream=None):
    return moe_layer_fwd_few_mx(d, bufs.Is, routes, w, X, W13q, W13s, W2q, W2s, S13, S2, bufs.out, bufs.ws, stream)


# ---------------------------------------------------------------------------
# Norms before and after a block.
# ---------------------------------------------------------------------------

def make_norm_desc(rows, H, gate=MOE_GATE_NONE, res_fp32=False, alpha=1.0, beta=1.0, eps=1e-6):
    return moe_norm_desc(rows, H, gate, int(res_fp32), alpha, beta, eps)


def block_norm_workspace_bytes(n: moe_norm_desc) -> int:
    b = load().moe_block_norm_workspace_bytes(ctypes.byref(n))
    if b < 0:
        raise MoeError(MOE_EINVAL, "moe_block_norm_workspace_bytes")
    return int(b)


def _norm_inputs(n, y, r, z, g_post, g_pre):
    e, bf, f32, dev = n.rows * n.H, torch.bfloat16, torch.float32, r.get_device()
    elem = n.gate == MOE_GATE_ELEM
    return [_buf("y", y, bf, e, dev), _buf("r", r, f32 if n.res_fp32 else bf, e, dev),
            _buf("z", z, bf if elem else f32, e if elem else n.rows, dev), _buf("g_post", g_post, f32, n.H, dev),
            _buf("g_pre", g_pre, f32, n.H, dev)]


def moe_block_norm_fwd(n, y, r, z, g_post, g_pre, r_out, xn, stats, stream=None):
    e, dev = n.rows * n.H, r.get_device()
    args = _norm_inputs(n, y, r, z, g_post, g_pre)
    args += [_buf("r_out", r_out, r.dtype, e, dev), _buf("xn", xn, torch.bfloat16, e, dev),
             _buf("stats", stats, torch.float32, 2 * n.rows, dev)]
    return _run("moe_block_norm_fwd", dev, stream, ctypes.byref(n), *args)


def moe_block_norm_bwd(n, y, r, z, g_post, g_pre, stats, dr_out, dxn, dy, dr, dz, dg_post, dg_pre, ws, stream=None):
    e, bf, f32, dev = n.rows * n.H, torch.bfloat16, torch.float32, r.get_device()
    elem = n.gate == MOE_GATE_ELEM
    args = _norm_inputs(n, y, r, z, g_post, g_pre)
    args += [_buf("stats", stats, f32, 2 * n.rows, dev), _buf("dr_out", dr_out, r.dtype, e, dev), _buf("dxn", dxn, bf, e, dev),
             _buf("dy", dy, bf, e, dev), _buf("dr", dr, r.dtype, e, dev),
             _buf("dz", dz, bf if elem else f32, e if elem else n.rows, dev), _buf("dg_post", dg_post, f32, n.H, dev),
             _buf("dg_pre", dg_pre, f32, n.H, dev), _buf("ws", ws, torch.uint8, 0, dev)]
    return _run("moe_block_norm_bwd", dev, stream, ctypes.byref(n), *args, 0 if ws is None else ws.numel())


@dataclass
class NormGrads:
    dy: torch.Tensor | None
    dr: torch.Tensor
    dz: torch.Tensor | None
    dg_post: torch.Tensor | None
    dg_pre: torch.Tensor | None
    ws: torch.Tensor


def alloc_norm_bwd(n: moe_norm_desc, device, post: bool = True, pre: bool = True, y: bool = True) -> NormGrads:
    """Gradients and workspace of moe_block_norm_bwd for a block with or
    without a post-norm, a pre-norm and (y=False: a pre-norm alone) an output."""
    bf, f32 = torch.bfloat16, torch.float32
    shape = (n.rows, n.H)
    dz = {MOE_GATE_NONE: None, MOE_GATE_TOKEN: ((n.rows,), f32), MOE_GATE_ELEM: (shape, bf)}[n.gate]
    return NormGrads(
        dy=torch.empty(shape, dtype=bf, device=device) if y else None,
        dr=torch.empty(shape, dtype=f32 if n.res_fp32 else bf, device=device),
        dz=torch.empty(dz[0], dtype=dz[1], device=device) if dz else None,
        dg_post=torch.empty(n.H, dtype=f32, device=device) if post else None,
        dg_pre=torch.empty(n.H, dtype=f32, device=device) if pre else None,
        ws=torch.empty(max(block_norm_workspace_bytes(n), 256), dtype=torch.uint8, device=device),
    )


def block_norm_bwd(n, y, r, z, g_post, g_pre, stats, dr_out, dxn, b: NormGrads, stream=None):
    return moe_block_norm_bwd(n, y, r, z, g_post, g_pre, stats, dr_out, dxn, b.dy, b.dr, b.dz, b.dg_post, b.dg_pre, b.ws,
                              stream)


# ---------------------------------------------------------------------------
# Activation checkpoints in 8 bits.
# ---------------------------------------------------------------------------

def moe_ckpt_pack(src, q, scales, nrows=None, stream=None):
    """Pack a bf16 tensor [rows][cols] into int8 codes (same shape) and float
    scales [rows][cols/128]; nrows: a device int32 (one element, e.g.
    seg_off[L:]) that limits the rows packed."""
    (rows, cols), dev = src.shape, src.get_device()
    args = [_buf("src", src, torch.bfloat16, 0, dev), rows, cols, _buf("nrows", nrows, torch.int32, 1, dev),
            _buf("q", q, torch.int8, rows * cols, dev), _buf("scales", scales, torch.float32, rows * (cols // CKPT_BLOCK), dev)]
    return _run("moe_ckpt_pack", dev, stream, *args)


def ckpt_pack(src, nrows=None, stream=None):
    """Allocate and fill (codes, scales) of a bf16 tensor [rows][cols]."""
    # memory of the stream that writes it
    with torch.cuda.stream(stream):
        q = torch.empty(src.shape, dtype=torch.int8, device=src.device)
        s = torch.empty((src.shape[0], src.shape[1] // CKPT_BLOCK), dtype=torch.float32, device=src.device)
    moe_ckpt_pack(src, q, s, nrows, stream)
    return q, s


def moe_ckpt_swiglu_bwd(q, scales, dA, wrow, dHU, A, dw, nrows=None, stream=None):
    (rows, I), dev = dA.shape, dA.get_device()
    bf, f32 = torch.bfloat16, torch.float32
    args = [_buf("q", q, torch.int8, 2 * rows * I, dev), _buf("scales", scales, f32, 2 * rows * I // CKPT_BLOCK, dev),
            _buf("dA", dA, bf, 0, dev), _buf("wrow", wrow, f32, rows, dev), rows, I, _buf("nrows", nrows, torch.int32, 1, dev),
            _buf("dHU", dHU, bf, 2 * rows * I, dev), _buf("A", A, bf, rows * I, dev), _buf("dw", dw, f32, rows, dev)]
    return _run("moe_ckpt_swiglu_bwd", dev, stream, *args)


def moe_layer_bwd_ckpt(d, dOut, w, X, phi, route_row, seg_off, q, scales, W13, W2, dX, dW13, dW2, dw, ws, stream=None):
    cap, n, H, I = capacity_rows(d), d.P * d.Np, d.H, d.I
    bf, f32, i32, dev = torch.bfloat16, torch.float32, torch.int32, X.get_device()
    args = [_buf("dOut", dOut, bf, n * H, dev), _buf("w", w, f32, n * d.K, dev), _buf("X", X, bf, n * H, dev),
            _buf("phi", phi, i32, 2 * cap, dev), _buf("route_row", route_row, i32, n * d.K, dev),
            _buf("seg_off", seg_off, i32, d.L + 1, dev), _buf("q", q, torch.int8, cap * 2 * I, dev),
            _buf("scales", scales, f32, cap * 2 * I // CKPT_BLOCK, dev), _buf("W13", W13, bf, d.L * 2 * I * H, dev),
            _buf("W2", W2, bf, d.L * H * I, dev), _buf("dX", dX, bf, n * H, dev), _buf("dW13", dW13, f32, d.L * 2 * I * H, dev),
            _buf("dW2", dW2, f32, d.L * H * I, dev), _buf("dw", dw, f32, n * d.K, dev), _buf("ws", ws, torch.uint8, 0, dev)]
    return _run("moe_layer_bwd_ckpt", dev, stream, ctypes.byref(d), *args, 0 if ws is None else ws.numel())


# ---------------------------------------------------------------------------
# The gated feed-forward block.
# ---------------------------------------------------------------------------

_TYPES = {torch.bfloat16: MOE_TYPE_BF16, torch.float16: MOE_TYPE_FP16, torch.float32: MOE_TYPE_FP32}
_DTYPES = {v: k for k, v in _TYPES.items()}


def _type(dtype) -> int:
    if dtype not in _TYPES:
        raise ValueError(f"unsupported element type {dtype}")
    return _TYPES[dtype]


def make_ffn_desc(rows, H, I, act=MOE_ACT_SILU, dtype=torch.bfloat16, ldx=0, ldo=0):
    """ldx, ldo: elements from one row of X and dX, and of out and dOut, to the next (0: H)."""
    return moe_ffn_desc(rows, ldx, ldo, H, I, act, _type(dtype))


def gated_ffn_workspace_bytes(n: moe_ffn_desc, bwd: bool = False) -> int:
    b = load().moe_gated_ffn_workspace_bytes(ctypes.byref(n), int(bwd))
    if b < 0:
        raise MoeError(MOE_EINVAL, "moe_gated_ffn_workspace_bytes")
    return int(b)


def _rows(name: str, t, dtype, rows: int, H: int, ld: int, dev: int):
    """Device pointer of a tensor of `rows` rows of H elements, ld apart (0: H)."""
    if t is None:
        return None
    ld = ld or H
    if ld == H and t.is_contiguous():
        return _buf(name, t, dtype, rows * H, dev)
    if t.dim() != 2 or t.dtype != dtype or t.get_device() != dev or t.shape[0] < rows or t.shape[1] != H or t.stride(1) != 1 or (
            rows > 1 and t.stride(0) != ld):
        raise ValueError(f"{name}: needs {rows} rows of {H} elements of {dtype}, {ld} apart, on cuda:{dev}, got {tuple(t.shape)} with "
                         f"strides {t.stride()} of {t.dtype} on {t.device}")
    return t.data_ptr()


def moe_gated_ffn_fwd(n, X, W13, W2, HU, A, out, ws, stream=None):
    R, H, I, dev, dt = n.rows, n.H, n.I, X.get_device(), _DTYPES.get(n.type)
    args = [_rows("X", X, dt, R, H, n.ldx, dev), _buf("W13", W13, dt, 2 * I * H, dev), _buf("W2", W2, dt, H * I, dev),
            _buf("HU", HU, dt, 2 * R * I, dev), _buf("A", A, dt, R * I, dev), _rows("out", out, dt, R, H, n.ldo, dev),
            _buf("ws", ws, torch.uint8, 0, dev)]
    return _run("moe_gated_ffn_fwd", dev, stream, ctypes.byref(n), *args, 0 if ws is None else ws.numel())


def moe_gated_ffn_bwd(n, dOut, X, HU, A, W13, W2, dX, dW13, dW2, ws, accumulate=False, stream=None):
    R, H, I, dev, dt = n.rows, n.H, n.I, X.get_device(), _DTYPES.get(n.type)
    wt = next((t.dtype for t in (dW13, dW2) if t is not None), torch.float32)
    args = [_rows("dOut", dOut, dt, R, H, n.ldo, dev), _rows("X", X, dt, R, H, n.ldx, dev), _buf("HU", HU, dt, 2 * R * I, dev),
            _buf("A", A, dt, R * I, dev), _buf("W13", W13, dt, 2 * I * H, dev), _buf("W2", W2, dt, H * I, dev),
            _rows("dX", dX, dt, R, H, n.ldx, dev), _buf("dW13", dW13, wt, 2 * I * H, dev), _buf("dW2", dW2, wt, H * I, dev)]
    return _run("moe_gated_ffn_bwd", dev, stream, ctypes.byref(n), *args, _type(wt), int(accumulate), _buf("ws", ws, torch.uint8, 0, dev),
                0 if ws is None else ws.numel())


@dataclass
class FfnBuffers:
    out: torch.Tensor
    HU: torch.Tensor | None
    A: torch.Tensor
    ws: torch.Tensor


def _alloc_rows(rows, H, ld, dtype, device):
    return torch.empty((rows, ld or H), dtype=dtype, device=device)[:, :H]


def alloc_gated_ffn(n: moe_ffn_desc, device, save_hu: bool = True) -> FfnBuffers:
    """Outputs and workspace of the forward; save_hu=False: no pre-activations for a backward."""
    dt = _DTYPES[n.type]
    return FfnBuffers(
        out=_alloc_rows(n.rows, n.H, n.ldo, dt, device),
        HU=torch.empty((n.rows, 2 * n.I), dtype=dt, device=device) if save_hu else None,
        A=torch.empty((n.rows, n.I), dtype=dt, device=device),
        ws=torch.empty(max(gated_ffn_workspace_bytes(n), 256), dtype=torch.uint8, device=device),
    )


def gated_ffn_fwd(n, X, W13, W2, b: FfnBuffers, stream=None):
    return moe_gated_ffn_fwd(n, X, W13, W2, b.HU, b.A, b.out, b.ws, stream)


@dataclass
class FfnGrads:
    dX: torch.Tensor | None
    dW13: torch.Tensor | None
    dW2: torch.Tensor | None
    ws: torch.Tensor


def alloc_gated_ffn_bwd(n: moe_ffn_desc, device, dx: bool = True, dw: bool = True, dw_dtype=torch.float32) -> FfnGrads:
    """Gradients (dx=False, dw=False: without those of X, of the weights) and workspace of the backward."""
    return FfnGrads(
        dX=_alloc_rows(n.rows, n.H, n.ldx, _DTYPES[n.type], device) if dx else None,
        dW13=torch.empty((2 * n.I, n.H), dtype=dw_dtype, device=device) if dw else None,
        dW2=torch.empty((n.H, n.I), dtype=dw_dtype, device=device) if dw else None,
        ws=torch.empty(max(gated_ffn_workspace_bytes(n, True), 256), dtype=torch.uint8, device=device),
    )


def gated_ffn_bwd(n, dOut, X, HU, A, W13, W2, b: FfnGrads, accumulate=False, stream=None):
    """A=None: the activations are computed again from HU."""
    return moe_gated_ffn_bwd(n, dOut, X, HU, A, W13, W2, b.dX, b.dW13, b.dW2, b.ws, accumulate, stream)


# ---------------------------------------------------------------------------
# Layer norm.
# ---------------------------------------------------------------------------

def make_layer_norm_desc(rows, H, x_dtype=torch.bfloat16, y_dtype=None, eps=1e-5, ldx=0, ldy=0):
    """y_dtype: None for x's; ldx, ldy: elements from one row of x, dx, dres, and of y, dy, to the next (0: H)."""
    return moe_ln_desc(rows, ldx, ldy, H, _type(x_dtype), _type(y_dtype or x_dtype), eps)


def layer_norm_workspace_bytes(n: moe_ln_desc) -> int:
    b = load().moe_layer_norm_workspace_bytes(ctypes.byref(n))
    if b < 0:
        raise MoeError(MOE_EINVAL, "moe_layer_norm_workspace_bytes")
    return int(b)


def moe_layer_norm_fwd(n, x, g, b, y, stats, stream=None):
    R, H, dev, f32 = n.rows, n.H, x.get_device(), torch.float32
    args = [_rows("x", x, _DTYPES.get(n.x_type), R, H, n.ldx, dev), _buf("g", g, f32, H, dev), _buf("b", b, f32, H, dev),
            _rows("y", y, _DTYPES.get(n.y_type), R, H, n.ldy, dev), _buf("stats", stats, f32, 2 * R, dev)]
    return _run("moe_layer_norm_fwd", dev, stream, ctypes.byref(n), *args)


def moe_layer_norm_bwd(n, x, g, stats, dy, dres, dx, dg, db, ws, stream=None):
    R, H, dev, f32, tx = n.rows, n.H, x.get_device(), torch.float32, _DTYPES.get(n.x_type)
    args = [_rows("x", x, tx, R, H, n.ldx, dev), _buf("g", g, f32, H, dev), _buf("stats", stats, f32, 2 * R, dev),
            _rows("dy", dy, _DTYPES.get(n.y_type), R, H, n.ldy, dev), _rows("dres", dres, tx, R, H, n.ldx, dev),
            _rows("dx", dx, tx, R, H, n.ldx, dev), _buf("dg", dg, f32, H, dev), _buf("db", db, f32, H, dev),
            _buf("ws", ws, torch.uint8, 0, dev)]
    return _run("moe_layer_norm_bwd", dev, stream, ctypes.byref(n), *args, 0 if ws is None else ws.numel())


@dataclass
class LayerNormBuffers:
    y: torch.Tensor
    stats: torch.Tensor | None


def alloc_layer_norm(n: moe_ln_desc, device, stats: bool = True) -> LayerNormBuffers:
    return LayerNormBuffers(
        y=_alloc_rows(n.rows, n.H, n.ldy, _DTYPES[n.y_type], device),
        stats=torch.empty((n.rows, 2), dtype=torch.float32, device=device) if stats else None,
    )


def layer_norm_fwd(n, x, g, b, bufs: LayerNormBuffers, stream=None):
    return moe_layer_norm_fwd(n, x, g, b, bufs.y, bufs.stats, stream)


@dataclass
class LayerNormGrads:
    dx: torch.Tensor
    dg: torch.Tensor | None
    db: torch.Tensor | None
    ws: torch.Tensor | None
    both: torch.Tensor | None  # dg and db, which the call writes together
    rows_of_both: tuple  # the two, whether or not they are asked for


def alloc_layer_norm_bwd(n: moe_ln_desc, device, weight: bool = True, bias: bool = True) -> LayerNormGrads:
    """Gradients and workspace of moe_layer_norm_bwd; weight=False: of x alone, bias=False: no db to show."""
    both = torch.empty((2, n.H), dtype=torch.float32, device=device) if weight or bias else None
    return LayerNormGrads(
        dx=_alloc_rows(n.rows, n.H, n.ldx, _DTYPES[n.x_type], device),
        dg=both[0] if weight else None,
        db=both[1] if bias else None,
        ws=torch.empty(max(layer_norm_workspace_bytes(n), 256), dtype=torch.uint8, device=device) if both is not None else None,
        both=both,
        rows_of_both=(None, None) if both is None else tuple(both),
    )


def layer_norm_bwd(n, x, g, stats, dy, dres, b: LayerNormGrads, stream=None):
    return moe_layer_norm_bwd(n, x, g, stats, dy, dres, b.dx, *b.rows_of_both, b.ws, stream)


# ---------------------------------------------------------------------------
# Norm and clipping of gradients.
# ---------------------------------------------------------------------------

@dataclass
class GradList:
    """Gradients and where their scaled values go (out: the gradients themselves), as
    the library takes them, with the result and the workspace of its calls.  It holds
    the tensors; a gradient that is allocated anew each step needs a new list."""
    grads: list
    out: list
    table: object
    dev: int
    result: torch.Tensor  # 16 bytes, of which sum (float64), norm and coef (float32) are views
    sum: torch.Tensor
    norm: torch.Tensor
    coef: torch.Tensor
    ws: torch.Tensor


def make_grad_list(grads, out=None, device=None) -> GradList:
    """grads: contiguous fp32, bf16 or fp16 tensors of one GPU, none of which overlaps another;
    out: as many of the same types and sizes (None: the gradients themselves); device: needed
    where grads is empty."""
    grads = list(grads)
    out = grads if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"{len(grads)} gradients, {len(out)} outputs")
    dev = grads[0].get_device() if grads else torch.device(device).index
    if dev is None and torch.device(device).type == "cuda":
        dev = torch.cuda.current_device()
    if dev is None or dev < 0:
        raise TypeError("device buffers must be CUDA (HIP) torch tensors")
    table, spans = (moe_grad * max(1, len(grads)))(), []
    for i, (g, o) in enumerate(zip(grads, out)):
        if o.numel() != g.numel():
            raise ValueError(f"out {i}: {o.numel()} elements for a gradient of {g.numel()}")
        if o is not g and o.data_ptr() != g.data_ptr():
            spans.append((o.data_ptr(), o.data_ptr() + o.numel() * o.element_size(), f"out {i}"))
        spans.append((g.data_ptr(), g.data_ptr() + g.numel() * g.element_size(), f"gradient {i}"))
        table[i] = moe_grad(_buf(f"gradient {i}", g, g.dtype, 0, dev), _buf(f"out {i}", o, g.dtype, 0, dev), g.numel(), _type(g.dtype), 0)
    spans = sorted(s for s in spans if s[0] < s[1])
    for a, b in zip(spans, spans[1:]):
        if b[0] < a[1]:
            raise ValueError(f"{a[2]} and {b[2]} overlap")
    device = torch.device("cuda", dev)
    result = torch.empty(16, dtype=torch.uint8, device=device)  # no fill: it would run on this stream, a call perhaps on another
    floats = result.view(torch.float32)
    return GradList(grads, out, table, dev, result, result.view(torch.float64)[:1], floats[2:3], floats[3:4],
                    torch.empty(load().moe_grad_workspace_bytes(len(grads)), dtype=torch.uint8, device=device))


def _grad_call(name, gl, max_norm, kind, scale, eps, stream):
    _run(name, gl.dev, stream, gl.table, len(gl.grads), kind, scale, max_norm, eps, gl.result.data_ptr(), gl.ws.data_ptr(), gl.ws.numel())
    return gl


def grad_norm(gl: GradList, max_norm=1.0, kind=MOE_NORM_L2, scale=1.0, eps=1e-6, stream=None) -> GradList:
    """Leaves gl.sum, gl.norm and gl.coef."""
    return _grad_call("moe_grad_norm", gl, max_norm, kind, scale, eps, stream)


def grad_clip(gl: GradList, max_norm, kind=MOE_NORM_L2, scale=1.0, eps=1e-6, stream=None) -> GradList:
    """Leaves gl.sum, gl.norm, gl.coef and the scaled gradients in gl.out."""
    return _grad_call("moe_grad_clip", gl, max_norm, kind, scale, eps, stream)


def grad_scale(gl: GradList, coef, scale=1.0, stream=None) -> GradList:
    """Leaves scale * coef * gradient in gl.out; coef: a float on the device."""
    _run("moe_grad_scale", gl.dev, stream, gl.table, len(gl.grads), _buf("coef", coef, torch.float32, 1, gl.dev), scale)
    return gl
