"""ctypes binding of libnvfp4rac (the C ABI in include/nvfp4rac.h).

Argument marshalling only: tensors are passed as device pointers, outputs and
workspaces are allocated with torch on the tensors' device, and each call is
enqueued on torch's current HIP stream.  Every computation happens in the
library's HIP kernels; there is no CPU fallback -- importing this module
without the built library raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnvfp4rac.so")

NVFP4_IN_F32, NVFP4_IN_BF16 = 0, 1
NVFP4_EPI_F32, NVFP4_EPI_SILU_MUL_BF16, NVFP4_EPI_BF16 = 0, 1, 2
NVFP4_GEMM_SKIP_INACTIVE_BLOCKS = 1
NVFP4_GEMM_PER_GROUP_SCALES = 2

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t


class GemmArgs(ctypes.Structure):
    """Mirror of w4a4_gemm_args_t."""
    _fields_ = [
        ("num_groups", _I64), ("N", _I64), ("K", _I64), ("total_rows", _I64),
        ("group_offsets", _P), ("gather_rows", _P),
        ("a_codes", _P), ("a_scales", _P), ("a_tscale", _P),
        ("r_codes", _P), ("r_scales", _P), ("r_tscale", _P),
        ("kblock_active", _P),
        ("w_codes", _P), ("w_scales", _P), ("w_tscale", _P),
        ("epilogue", _I64), ("out", _P), ("out_amax", _P), ("flags", _I64),
        ("out_y", _P),
    ]


class Fp8GemmArgs(ctypes.Structure):
    """Mirror of fp8_gemm_args_t."""
    _fields_ = [
        ("num_groups", _I64), ("N", _I64), ("K", _I64), ("total_rows", _I64),
        ("group_offsets", _P), ("gather_rows", _P),
        ("a_codes", _P), ("a_scales", _P), ("w_codes", _P), ("w_scales", _P),
        ("epilogue", _I64), ("out", _P),
    ]


class MoEDecodeArgs(ctypes.Structure):
    """Mirror of nvfp4_moe_decode_args_t."""
    _fields_ = [
        ("T", _I64), ("E", _I64), ("k", _I64), ("H", _I64), ("I", _I64),
        ("x", _P), ("x_dtype", _I64), ("ldx", _I64),
        ("logits", _P), ("ld_logits", _I64),
        ("gu_codes", _P), ("gu_scales", _P), ("gu_tscale", _P),
        ("d_codes", _P), ("d_scales", _P), ("d_tscale", _P),
        ("out", _P), ("ldo", _I64), ("topk_ids", _P), ("topk_weights", _P),
    ]


class Int8GemmArgs(ctypes.Structure):
    """Mirror of int8_gemm_args_t."""
    _fields_ = [
        ("num_groups", _I64), ("N", _I64), ("K", _I64), ("total_rows", _I64),
        ("group_offsets", _P), ("gather_rows", _P),
        ("a_codes", _P), ("a_scales", _P),
        ("x", _P), ("x_dtype", _I64), ("ldx", _I64), ("src_rows", _I64),
        ("w_codes", _P), ("w_scales", _P), ("epilogue", _I64), ("out", _P),
    ]


_SIGS = {
    "nvfp4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "nvfp4_quantize_workspace_size": (_SZ, [_I64, _I64]),
    "nvfp4_quantize": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P, _P,
                                      _P, _P, _P, _SZ, _P]),
    "rac_select_residual_workspace_size": (_SZ, [_I64, _I64]),
    "rac_select_residual": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P,
                                           _P, _P, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_route_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "moe_route": (ctypes.c_int, [_P, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "w4a4_grouped_gemm_rac_workspace_size": (_SZ, [ctypes.POINTER(GemmArgs)]),
    "w4a4_grouped_gemm_rac": (ctypes.c_int, [ctypes.POINTER(GemmArgs), _P, _SZ, _P]),
    "moe_combine": (ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P, _P]),
    "nvfp4_quantize_grouped_workspace_size": (_SZ, [_I64, _I64]),
    "nvfp4_quantize_grouped": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _I64, _I64, _P,
                                              _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "rac_select_residual_grouped_workspace_size": (_SZ, [_I64, _I64]),
    "rac_select_residual_grouped": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _I64, _I64,
                                                   _P, _P, _P, _P, _P, _I64, _P, _P, _P, _P, _P,
                                                   _P, _SZ, _P]),
    "nvfp4_qdq_workspace_size": (_SZ, [_I64, _I64]),
    "nvfp4_qdq": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, ctypes.c_int, _P, _P,
                                 _P, _SZ, _P]),
    "nvfp4_dequantize": (ctypes.c_int, [_P, _P, _P, _I64, _I64, ctypes.c_int, _P, _P]),
    "fp8_quantize_rows": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _P, _P, _P]),
    "fp8_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(Fp8GemmArgs), _P]),
    "nvfp4_check_groups": (ctypes.c_int, [_P, _I64, _I64, _P, _I64]),
    "nvfp4_quantize_rac_static": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P,
                                                 _P, _P, _P, _I64, _P, _P, _P, _P, _P, _P]),
    "nvfp4_moe_decode_workspace_size": (_SZ, [ctypes.POINTER(MoEDecodeArgs)]),
    "nvfp4_moe_decode": (ctypes.c_int, [ctypes.POINTER(MoEDecodeArgs), _P, _SZ, _P]),
    "token_logprobs_workspace_size": (_SZ, [_I64, _I64, _I64]),
    "token_logprobs": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _I64, _P, _P,
                                      _P, _P, _P, _P, _SZ, _P]),
    "token_logprobs_backward": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P,
                                               _P, _P, _P, _P, _I64, _P]),
    "int8_quantize_rows": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _P, _P]),
    "int8_grouped_gemm_workspace_size": (_SZ, [ctypes.POINTER(Int8GemmArgs)]),
    "int8_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(Int8GemmArgs), _P, _SZ, _P]),
    "moe_balance_loss_workspace_size": (_SZ, [_I64, _I64]),
    "moe_balance_loss": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _P, _I64, _P, _P, _P,
                                        _P, _P, _P, _SZ, _P]),
    "moe_balance_loss_backward": (ctypes.c_int, [_P, ctypes.c_int, _I64, _I64, _I64, _I64, _P, _P,
                                                 _P, _P, _P, _I64, _P]),
}
EXPORTS = tuple(_SIGS)


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is missing: build the HIP library first "
            "(python -m nvfp4_w4a4_moe_quant_amd.build)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib: Optional[ctypes.CDLL] = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        _lib = load()
    return _lib


class NVFP4Error(RuntimeError):
    pass


def _check(status: int):
    if status != 0:
        raise NVFP4Error(f"status {status}: {lib().nvfp4_status_string(status).decode()}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _ws(nbytes: int, dev) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=dev)


def _dtype_code(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return NVFP4_IN_BF16
    if x.dtype == torch.float32:
        return NVFP4_IN_F32
    raise TypeError(f"unsupported dtype {x.dtype}")


class NVFP4(NamedTuple):
    codes: torch.Tensor    # uint8 [rows, K/2]
    scales: torch.Tensor   # uint8 [rows, K/16]
    tscale: torch.Tensor   # float32 [1]


class QuantOut(NamedTuple):
    q: NVFP4
    channel_score: Optional[torch.Tensor]  # int64 [K]
    channel_max: Optional[torch.Tensor]    # float32 [K]


class RacOut(NamedTuple):
    r: NVFP4
    selected: torch.Tensor       # int32 [n_select]
    kblock_active: torch.Tensor  # uint8 [K/16]


class MoEDecodeOut(NamedTuple):
    out: torch.Tensor           # [T, H], x's dtype
    topk_ids: torch.Tensor      # int32 [T, k]
    topk_weights: torch.Tensor  # float32 [T, k]


class LogprobsOut(NamedTuple):
    logprobs: Optional[torch.Tensor]      # float32 [T]
    entropy: torch.Tensor                 # float32 [T]
    norm: torch.Tensor                    # float32 [T, 2], for the backward call
    top_ids: Optional[torch.Tensor]       # int32 [T, top_k]
    top_logprobs: Optional[torch.Tensor]  # float32 [T, top_k]


class BalanceOut(NamedTuple):
    losses: torch.Tensor      # float32 [2]: balance loss, z-loss
    counts: torch.Tensor      # int32 [E]
    mean_probs: torch.Tensor  # float32 [E]
    tokens: torch.Tensor      # int32 [1]: rows counted, for the backward call


class RouteOut(NamedTuple):
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    expert_offsets: torch.Tensor
    gather_rows: torch.Tensor
    row_of: torch.Tensor


def nvfp4_quantize(x: torch.Tensor, *, amax_in: Optional[torch.Tensor] = None,
                   stats: bool = False, channel_max: bool = True) -> QuantOut:
    """NVFP4-quantize a 2-D bf16/fp32 device tensor (row stride honoured).
    stats: the RAC channel scores; channel_max (with stats): also max|e| per
    channel, which the selection does not need."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, K = x.shape
    dev = x.device
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    score = torch.empty(K, dtype=torch.int64, device=dev) if stats else None
    chmax = torch.empty(K, dtype=torch.float32, device=dev) if stats and channel_max else None
    L = lib()
    ws = _ws(L.nvfp4_quantize_workspace_size(rows, K), dev)
    _check(L.nvfp4_quantize(_ptr(x), _dtype_code(x), rows, K, x.stride(0), _ptr(amax_in),
                            _ptr(codes), _ptr(scales), _ptr(ts), _ptr(score), _ptr(chmax),
                            _ptr(ws), ws.numel(), _stream(dev)))
    return QuantOut(NVFP4(codes, scales, ts), score, chmax)


def rac_select_residual(x: torch.Tensor, qo: QuantOut, n_select: int) -> RacOut:
    assert qo.channel_score is not None, "quantize with stats=True first"
    rows, K = x.shape
    dev = x.device
    q = qo.q
    sel = torch.empty(max(n_select, 1), dtype=torch.int32, device=dev)[:n_select]
    kact = torch.empty(K // 16, dtype=torch.uint8, device=dev)
    rc = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    rs = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev)
    rts = torch.empty(1, dtype=torch.float32, device=dev)
    L = lib()
    ws = _ws(L.rac_select_residual_workspace_size(rows, K), dev)
    _check(L.rac_select_residual(_ptr(x), _dtype_code(x), rows, K, x.stride(0), _ptr(q.codes),
                                 _ptr(q.scales), _ptr(q.tscale), _ptr(qo.channel_score),
                                 _ptr(qo.channel_max), n_select, _ptr(sel), _ptr(kact),
                                 _ptr(rc), _ptr(rs), _ptr(rts), _ptr(ws), ws.numel(),
                                 _stream(dev)))
    return RacOut(NVFP4(rc, rs, rts), sel, kact)


def nvfp4_quantize_rac_static(x: torch.Tensor, n_select: int, *,
                              amax_in: Optional[torch.Tensor] = None, channel_max: bool = True):
    """nvfp4_quantize (with statistics) + rac_select_residual in one call that
    takes no workspace (the library's per-device scratch).  Returns
    (QuantOut, RacOut)."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, K = x.shape
    dev = x.device
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    score = torch.empty(K, dtype=torch.int64, device=dev)
    chmax = torch.empty(K, dtype=torch.float32, device=dev) if channel_max else None
    sel = torch.empty(max(n_select, 1), dtype=torch.int32, device=dev)[:n_select]
    kact = torch.empty(K // 16, dtype=torch.uint8, device=dev)
    rc = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    rs = torch.empty((rows, K // 16), dtype=torch.uint8, device=dev)
    rts = torch.empty(1, dtype=torch.float32, device=dev)
    _check(lib().nvfp4_quantize_rac_static(
        _ptr(x), _dtype_code(x), rows, K, x.stride(0), _ptr(amax_in), _ptr(codes), _ptr(scales),
        _ptr(ts), _ptr(score), _ptr(chmax), n_select, _ptr(sel), _ptr(kact), _ptr(rc), _ptr(rs),
        _ptr(rts), _stream(dev)))
    return (QuantOut(NVFP4(codes, scales, ts), score, chmax),
            RacOut(NVFP4(rc, rs, rts), sel, kact))


def nvfp4_quantize_grouped(x: torch.Tensor, group_offsets: torch.Tensor, total_rows: int, *,
                           gather_rows: Optional[torch.Tensor] = None,
                           stats: bool = False, channel_max: bool = True) -> QuantOut:
    """Per-expert quantization: each group's rows (x[gather[j]] or x[j]) as
    their own tensor.  Returns grouped-order codes/scales, tscale [G] and, with
    stats, score [G, K] and channel max [G, K]."""
    assert x.dim() == 2 and x.stride(1) == 1
    K = x.shape[1]
    G = group_offsets.numel() - 1
    dev = x.device
    codes = torch.empty((total_rows, K // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((total_rows, K // 16), dtype=torch.uint8, device=dev)
    ts = torch.empty(G, dtype=torch.float32, device=dev)
    score = torch.empty((G, K), dtype=torch.int64, device=dev) if stats else None
    chmax = (torch.empty((G, K), dtype=torch.float32, device=dev) if stats and channel_max
             else None)
    L = lib()
    ws = _ws(L.nvfp4_quantize_grouped_workspace_size(G, K), dev)
    _check(L.nvfp4_quantize_grouped(_ptr(x), _dtype_code(x), K, x.stride(0), _ptr(group_offsets),
                                    G, total_rows, _ptr(gather_rows), _ptr(codes), _ptr(scales),
                                    _ptr(ts), _ptr(score), _ptr(chmax), _ptr(ws), ws.numel(),
                                    _stream(dev)))
    return QuantOut(NVFP4(codes, scales, ts), score, chmax)


def rac_select_residual_grouped(x: torch.Tensor, qo: QuantOut, group_offsets: torch.Tensor,
                                total_rows: int, n_select: int, *,
                                gather_rows: Optional[torch.Tensor] = None) -> RacOut:
    """Per-expert RAC: selection, masks and residual per group."""
    K = x.shape[1]
    G = group_offsets.numel() - 1
    dev = x.device
    sel = torch.empty((G, max(n_select, 1)), dtype=torch.int32, device=dev)
    kact = torch.empty((G, K // 16), dtype=torch.uint8, device=dev)
    rc = torch.empty((total_rows, K // 2), dtype=torch.uint8, device=dev)
    rs = torch.empty((total_rows, K // 16), dtype=torch.uint8, device=dev)
    rts = torch.empty(G, dtype=torch.float32, device=dev)
    L = lib()
    ws = _ws(L.rac_select_residual_grouped_workspace_size(G, K), dev)
    _check(L.rac_select_residual_grouped(
        _ptr(x), _dtype_code(x), K, x.stride(0), _ptr(group_offsets), G, total_rows,
        _ptr(gather_rows), _ptr(qo.q.scales), _ptr(qo.q.tscale), _ptr(qo.channel_score),
        _ptr(qo.channel_max), n_select, _ptr(sel), _ptr(kact), _ptr(rc), _ptr(rs), _ptr(rts),
        _ptr(ws), ws.numel(), _stream(dev)))
    return RacOut(NVFP4(rc, rs, rts), sel[:, :n_select], kact)


def moe_route(logits: torch.Tensor, k: int) -> RouteOut:
    assert logits.dtype == torch.float32 and logits.is_contiguous()
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    wts = torch.empty((T, k), dtype=torch.float32, device=dev)
    off = torch.empty(E + 1, dtype=torch.int32, device=dev)
    gather = torch.empty(T * k, dtype=torch.int32, device=dev)
    row_of = torch.empty((T, k), dtype=torch.int32, device=dev)
    L = lib()
    ws = _ws(L.moe_route_workspace_size(T, E, k), dev)
    _check(L.moe_route(_ptr(logits), T, E, k, _ptr(ids), _ptr(wts), _ptr(off), _ptr(gather),
                       _ptr(row_of), _ptr(ws), ws.numel(), _stream(dev)))
    return RouteOut(ids, wts, off, gather, row_of)


def w4a4_grouped_gemm_rac(a: NVFP4, w: NVFP4, group_offsets: torch.Tensor, *, N: int, K: int,
                          total_rows: int, gather_rows: Optional[torch.Tensor] = None,
                          r: Optional[NVFP4] = None,
                          kblock_active: Optional[torch.Tensor] = None,
                          epilogue: int = NVFP4_EPI_F32,
                          out: Optional[torch.Tensor] = None,
                          out_amax: Optional[torch.Tensor] = None,
                          skip_inactive: bool = False,
                          per_group_scales: bool = False,
                          out_y: Optional[torch.Tensor] = None,
                          validate: bool = False) -> torch.Tensor:
    """w: codes [G, N, K/2], scales [G, N, K/16], tscale [G].  With the SiLU*mul
    epilogue, out_y (float32 [total_rows, N]) also receives the FP32 gate/up
    values before the SiLU.  validate=True checks the offsets and gather
    indices on the host first (check_groups; synchronizes)."""
    dev = a.codes.device
    G = group_offsets.numel() - 1
    if validate:
        check_groups(group_offsets, total_rows, gather_rows, a.codes.shape[0])
    if out is None:
        if epilogue == NVFP4_EPI_F32:
            out = torch.empty((total_rows, N), dtype=torch.float32, device=dev)
        else:
            out = torch.empty((total_rows, N // 2), dtype=torch.bfloat16, device=dev)
    args = GemmArgs(
        num_groups=G, N=N, K=K, total_rows=total_rows,
        group_offsets=_ptr(group_offsets), gather_rows=_ptr(gather_rows),
        a_codes=_ptr(a.codes), a_scales=_ptr(a.scales), a_tscale=_ptr(a.tscale),
        r_codes=_ptr(r.codes if r else None), r_scales=_ptr(r.scales if r else None),
        r_tscale=_ptr(r.tscale if r else None), kblock_active=_ptr(kblock_active),
        w_codes=_ptr(w.codes), w_scales=_ptr(w.scales), w_tscale=_ptr(w.tscale),
        epilogue=epilogue, out=_ptr(out), out_amax=_ptr(out_amax),
        flags=(NVFP4_GEMM_SKIP_INACTIVE_BLOCKS if skip_inactive else 0) |
              (NVFP4_GEMM_PER_GROUP_SCALES if per_group_scales else 0),
        out_y=_ptr(out_y))
    L = lib()
    nbytes = L.w4a4_grouped_gemm_rac_workspace_size(ctypes.byref(args))
    ws = _ws(nbytes, dev) if nbytes else None
    _check(L.w4a4_grouped_gemm_rac(ctypes.byref(args), _ptr(ws), 0 if ws is None else ws.numel(),
                                   _stream(dev)))
    return out


def check_groups(group_offsets: torch.Tensor, total_rows: int,
                 gather_rows: Optional[torch.Tensor] = None, src_rows: int = 0) -> None:
    """Checks the grouped GEMM's offsets and gather indices on host copies
    (nvfp4_check_groups); raises NVFP4Error on a violation.  Synchronizes with
    the device to copy the arrays."""
    import numpy as np
    offs = np.ascontiguousarray(group_offsets.cpu().numpy(), np.int32)
    gat = None if gather_rows is None else \
        np.ascontiguousarray(gather_rows.cpu().numpy(), np.int32)
    if gat is not None and gat.size < total_rows:
        raise NVFP4Error(f"gather_rows has {gat.size} entries, total_rows is {total_rows}")
    _check(lib().nvfp4_check_groups(
        offs.ctypes.data_as(ctypes.c_void_p), offs.size - 1, total_rows,
        None if gat is None else gat.ctypes.data_as(ctypes.c_void_p), src_rows))


def moe_combine(y: torch.Tensor, row_of: torch.Tensor, topk_weights: torch.Tensor, *,
                out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """Token-order output [T, H] from the grouped expert outputs y [rows, H]."""
    T, k = row_of.shape
    H = y.shape[1]
    dev = y.device
    out = torch.empty((T, H), dtype=out_dtype, device=dev)
    _check(lib().moe_combine(_ptr(y), _ptr(row_of), _ptr(topk_weights), T, k, H,
                             _dtype_code(out), _ptr(out), _stream(dev)))
    return out


# ------------------------------------ trainer-side weight fake-quant
def nvfp4_qdq(x: torch.Tensor, *, out_dtype: torch.dtype = torch.bfloat16,
              amax_in: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rollout's NVFP4 quantize-dequantize of a 2-D bf16/fp32 tensor,
    returned as bf16 or FP32 [rows, K]."""
    assert x.dim() == 2 and x.stride(1) == 1
    rows, K = x.shape
    dev = x.device
    out = torch.empty((rows, K), dtype=out_dtype, device=dev)
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    L = lib()
    ws = _ws(L.nvfp4_qdq_workspace_size(rows, K), dev)
    _check(L.nvfp4_qdq(_ptr(x), _dtype_code(x), rows, K, x.stride(0), _ptr(amax_in),
                       _dtype_code(out), _ptr(out), _ptr(ts), _ptr(ws), ws.numel(),
                       _stream(dev)))
    return out


def nvfp4_dequantize(q: NVFP4, *, out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Dequantized values of an NVFP4 tensor (codes [rows, K/2])."""
    rows, K = q.codes.shape[0], q.codes.shape[1] * 2
    dev = q.codes.device
    out = torch.empty((rows, K), dtype=out_dtype, device=dev)
    _check(lib().nvfp4_dequantize(_ptr(q.codes), _ptr(q.scales), _ptr(q.tscale), rows, K,
                                  _dtype_code(out), _ptr(out), _stream(dev)))
    return out


# ------------------------------------------------- FP8 W8A8 comparator
class FP8(NamedTuple):
    codes: torch.Tensor    # uint8 [rows, K] (E4M3), or [G, N, K] for weights
    scales: torch.Tensor   # float32 [rows], or [G, N]


def fp8_quantize_rows(x: torch.Tensor, out: Optional[FP8] = None) -> FP8:
    """Per-row E4M3 quantization of x [rows, K] (bf16 or FP32)."""
    assert x.dim() == 2 and x.is_contiguous()
    rows, K = x.shape
    dev = x.device
    if out is None:
        out = FP8(torch.empty((rows, K), dtype=torch.uint8, device=dev),
                  torch.empty(rows, dtype=torch.float32, device=dev))
    _check(lib().fp8_quantize_rows(_ptr(x), _dtype_code(x), rows, K, _ptr(out.codes),
                                   _ptr(out.scales), _stream(dev)))
    return out


def fp8_grouped_gemm(a: FP8, w: FP8, group_offsets: torch.Tensor, *, N: int, K: int,
                     total_rows: int, gather_rows: Optional[torch.Tensor] = None,
                     epilogue: int = NVFP4_EPI_F32,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """w: codes [G, N, K], scales [G, N].  epilogue F32, SILU_MUL_BF16 or BF16."""
    dev = a.codes.device
    G = group_offsets.numel() - 1
    if out is None:
        if epilogue == NVFP4_EPI_F32:
            out = torch.empty((total_rows, N), dtype=torch.float32, device=dev)
        elif epilogue == NVFP4_EPI_BF16:
            out = torch.empty((total_rows, N), dtype=torch.bfloat16, device=dev)
        else:
            out = torch.empty((total_rows, N // 2), dtype=torch.bfloat16, device=dev)
    args = Fp8GemmArgs(
        num_groups=G, N=N, K=K, total_rows=total_rows,
        group_offsets=_ptr(group_offsets), gather_rows=_ptr(gather_rows),
        a_codes=_ptr(a.codes), a_scales=_ptr(a.scales),
        w_codes=_ptr(w.codes), w_scales=_ptr(w.scales),
        epilogue=epilogue, out=_ptr(out))
    _check(lib().fp8_grouped_gemm(ctypes.byref(args), _stream(dev)))
    return out


# --------------------------------------------- decode step: layer and tokens
# These calls take a few microseconds on the GPU, so the host side is kept to
# plain attribute checks; messages are only built for a call that is refused.
def _refuse(what: str):
    raise ValueError(what)


def _vector(t: Optional[torch.Tensor], n: int, dtype: torch.dtype, dev, name: str):
    """Address of a contiguous [n] tensor of one dtype on one device (or None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.dim() != 1 or t.numel() != n or t.device != dev \
            or not t.is_contiguous():
        _refuse(f"{name}: contiguous {dtype} [{n}] on {dev}")
    return t.data_ptr()


def _row_stride(t: torch.Tensor, name: str) -> int:
    """Row stride of a 2-D tensor whose rows are contiguous and do not overlap."""
    rows, cols = t.shape
    if rows <= 1:
        if rows and cols > 1 and t.stride(1) != 1:
            _refuse(f"{name}: contiguous rows")
        return cols + -cols % 8
    st, one = t.stride()
    if cols > 1 and one != 1:
        _refuse(f"{name}: contiguous rows")
    if st < cols:
        _refuse(f"{name}: rows overlap")
    return st


def _call(dev: torch.device, fn, *args):
    """Runs fn(*args, stream) with dev current, on its current stream."""
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev.index))
    if status:
        _check(status)


def _nvfp4_experts(w: NVFP4, E: int, N: int, K: int, dev, name: str):
    for t, shape, dt in ((w.codes, (E, N, K // 2), torch.uint8),
                         (w.scales, (E, N, K // 16), torch.uint8),
                         (w.tscale, (E,), torch.float32)):
        if t.shape != shape or t.dtype != dt or t.device != dev or not t.is_contiguous():
            _refuse(f"{name}: contiguous {dt} {shape} on {dev}")


def nvfp4_moe_decode(x: torch.Tensor, logits: torch.Tensor, wgu: NVFP4, wd: NVFP4, k: int, *,
                     out: Optional[torch.Tensor] = None) -> MoEDecodeOut:
    """The whole MoE FFN layer for up to 64 tokens on NVFP4 expert weights
    wgu [E, 2I, H] (gate rows first) and wd [E, H, I], with unquantized
    activations x [T, H] (bf16 or FP32, row stride honoured) and router logits
    [T, E] (FP32, row stride honoured).  Rows whose logits are all -inf cost
    nothing and give 0."""
    if x.dim() != 2 or logits.dim() != 2 or x.shape[0] != logits.shape[0]:
        _refuse("x [T, H] and logits [T, E]")
    T, H = x.shape
    E = logits.shape[1]
    dev = x.device
    xd = _dtype_code(x)
    if dev.type != "cuda" or logits.device != dev:
        _refuse("x and logits on one GPU")
    if logits.dtype != torch.float32:
        _refuse("logits are float32")
    if wd.codes.dim() != 3:
        _refuse("wd codes [E, H, I/2]")
    I = wd.codes.shape[2] * 2
    _nvfp4_experts(wgu, E, 2 * I, H, dev, "wgu")
    _nvfp4_experts(wd, E, H, I, dev, "wd")
    if out is None:
        out = torch.empty(T, H, dtype=x.dtype, device=dev)
    elif out.shape != x.shape or out.dtype != x.dtype or out.device != dev:
        _refuse("out like x")
    ids = torch.empty(T, k, dtype=torch.int32, device=dev)
    wts = torch.empty(T, k, dtype=torch.float32, device=dev)
    args = MoEDecodeArgs(
        T, E, k, H, I, x.data_ptr(), xd, _row_stride(x, "x"),
        logits.data_ptr(), _row_stride(logits, "logits"),
        wgu.codes.data_ptr(), wgu.scales.data_ptr(), wgu.tscale.data_ptr(),
        wd.codes.data_ptr(), wd.scales.data_ptr(), wd.tscale.data_ptr(),
        out.data_ptr(), _row_stride(out, "out"), ids.data_ptr(), wts.data_ptr())
    L = lib()
    ref = ctypes.byref(args)
    ws = _ws(L.nvfp4_moe_decode_workspace_size(ref), dev)
    _call(dev, L.nvfp4_moe_decode, ref, ws.data_ptr(), ws.numel())
    return MoEDecodeOut(out, ids, wts)


def token_logprobs(logits: torch.Tensor, targets: Optional[torch.Tensor] = None, *,
                   top_k: int = 0, inv_temperature: Optional[torch.Tensor] = None) -> LogprobsOut:
    """Log-probability of targets [T] (int64; negative = ignored, giving 0),
    entropy and the top_k largest alternatives of each row of logits [T, V]
    (bf16 or FP32, row stride honoured), at a temperature per row
    (inv_temperature, float32 [T]).  Logits of -inf are masked tokens."""
    if logits.dim() != 2:
        _refuse("logits [T, V]")
    T, V = logits.shape
    dev = logits.device
    dt = _dtype_code(logits)
    if dev.type != "cuda":
        _refuse("logits on a GPU")
    y = _vector(targets, T, torch.int64, dev, "targets")
    it = _vector(inv_temperature, T, torch.float32, dev, "inv_temperature")
    lp = torch.empty(T, dtype=torch.float32, device=dev) if targets is not None else None
    ent = torch.empty(T, dtype=torch.float32, device=dev)
    norm = torch.empty(T, 2, dtype=torch.float32, device=dev)
    ids = torch.empty(T, top_k, dtype=torch.int32, device=dev) if top_k > 0 else None
    tlp = torch.empty(T, top_k, dtype=torch.float32, device=dev) if top_k > 0 else None
    L = lib()
    n = L.token_logprobs_workspace_size(T, V, top_k)
    ws = _ws(n, dev) if n else None
    _call(dev, L.token_logprobs, logits.data_ptr(), dt, T, V, _row_stride(logits, "logits"),
          y, it, top_k, None if lp is None else lp.data_ptr(), ent.data_ptr(), norm.data_ptr(),
          None if ids is None else ids.data_ptr(), None if tlp is None else tlp.data_ptr(),
          None if ws is None else ws.data_ptr(), n)
    return LogprobsOut(lp, ent, norm, ids, tlp)


def token_logprobs_backward(logits: torch.Tensor, targets: Optional[torch.Tensor],
                            norm: torch.Tensor, entropy: Optional[torch.Tensor],
                            grad_logprobs: Optional[torch.Tensor],
                            grad_entropy: Optional[torch.Tensor] = None, *,
                            inv_temperature: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits from those of token_logprobs's logprobs and
    entropy (either may be None), with its norm and entropy.  out: where to
    write it, which may be logits itself."""
    if logits.dim() != 2:
        _refuse("logits [T, V]")
    T, V = logits.shape
    dev = logits.device
    dt = _dtype_code(logits)
    if dev.type != "cuda":
        _refuse("logits on a GPU")
    f32 = torch.float32
    y = _vector(targets, T, torch.int64, dev, "targets")
    it = _vector(inv_temperature, T, f32, dev, "inv_temperature")
    h = _vector(entropy, T, f32, dev, "entropy")
    ga = _vector(grad_logprobs, T, f32, dev, "grad_logprobs")
    gb = _vector(grad_entropy, T, f32, dev, "grad_entropy")
    if norm.shape != (T, 2) or norm.dtype != f32 or norm.device != dev or not norm.is_contiguous():
        _refuse("norm: float32 [T, 2]")
    if out is None:
        out = torch.empty(T, V, dtype=logits.dtype, device=dev)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
        _refuse("out like logits")
    _call(dev, lib().token_logprobs_backward, logits.data_ptr(), dt, T, V,
          _row_stride(logits, "logits"), y, it, norm.data_ptr(), h, ga, gb, out.data_ptr(),
          _row_stride(out, "out"))
    return out


# ------------------------------------------------- INT8 W8A8 comparator
class INT8(NamedTuple):
    codes: torch.Tensor    # int8 [rows, K], or [G, N, K] for weights
    scales: torch.Tensor   # float32 [rows], or [G, N]


def int8_quantize_rows(x: torch.Tensor, out: Optional[INT8] = None) -> INT8:
    """Per-row quantization of x [rows, K] (bf16 or FP32, row stride honoured)
    to 8-bit integers: scale amax / 127."""
    if x.dim() != 2:
        _refuse("x [rows, K]")
    rows, K = x.shape
    dev = x.device
    dt = _dtype_code(x)
    if dev.type != "cuda":
        _refuse("x on a GPU")
    if out is None:
        out = INT8(torch.empty(rows, K, dtype=torch.int8, device=dev),
                   torch.empty(rows, dtype=torch.float32, device=dev))
    else:
        _int8(out, (rows, K), dev, "out")
    _call(dev, lib().int8_quantize_rows, x.data_ptr(), dt, rows, K, _row_stride(x, "x"),
          out.codes.data_ptr(), out.scales.data_ptr())
    return out


def _int8(q: INT8, shape, dev, name: str):
    c, s = q
    if c.shape != shape or c.dtype != torch.int8 or c.device != dev or not c.is_contiguous():
        _refuse(f"{name}: contiguous int8 codes {shape} on {dev}")
    if s.shape != shape[:-1] or s.dtype != torch.float32 or s.device != dev \
            or not s.is_contiguous():
        _refuse(f"{name}: contiguous float32 scales {shape[:-1]} on {dev}")


def int8_grouped_gemm(a, w: INT8, group_offsets: Optional[torch.Tensor] = None, *, N: int, K: int,
                      total_rows: int, gather_rows: Optional[torch.Tensor] = None,
                      epilogue: int = NVFP4_EPI_F32, out: Optional[torch.Tensor] = None,
                      validate: bool = False) -> torch.Tensor:
    """a: INT8 rows, or x [src_rows, K] (bf16 or FP32, row stride honoured), which
    the call quantizes as int8_quantize_rows does.  w: codes [G, N, K], scales
    [G, N].  group_offsets [G + 1] may be None for one group.  epilogue F32,
    SILU_MUL_BF16 or BF16.  validate=True checks the offsets, which may end before
    total_rows, and the groups' gather indices on the host first (check_groups;
    synchronizes)."""
    quantized = isinstance(a, INT8)
    x = a.codes if quantized else a
    shape, dev = x.shape, x.device
    if len(shape) != 2 or shape[1] != K:
        _refuse("activations [src_rows, K]")
    src_rows = shape[0]
    if dev.type != "cuda":
        _refuse("activations on a GPU")
    G = 1 if group_offsets is None else group_offsets.numel() - 1
    _int8(w, (G, N, K), dev, "w")
    offs = gat = codes = scales = xp = None
    xd = ldx = 0
    if group_offsets is not None:
        offs = _vector(group_offsets, G + 1, torch.int32, dev, "group_offsets")
    if gather_rows is not None:
        gat = _vector(gather_rows, total_rows, torch.int32, dev, "gather_rows")
    elif src_rows < total_rows:
        _refuse("activations of at least total_rows rows")
    if quantized:
        _int8(a, (src_rows, K), dev, "a")
        codes, scales = x.data_ptr(), a.scales.data_ptr()
    else:
        xp, xd, ldx = x.data_ptr(), _dtype_code(x), _row_stride(x, "x")
    if validate:
        ends = torch.tensor([0, total_rows], dtype=torch.int32) if group_offsets is None \
            else group_offsets.cpu()
        rows = int(ends[-1])  # those behind the last group are not touched
        if rows > total_rows:
            raise NVFP4Error(f"group_offsets end at {rows}, total_rows is {total_rows}")
        check_groups(ends, rows, None if gather_rows is None else gather_rows[:rows], src_rows)
    odt = torch.float32 if epilogue == NVFP4_EPI_F32 else torch.bfloat16
    cols = N // 2 if epilogue == NVFP4_EPI_SILU_MUL_BF16 else N
    if out is None:
        out = torch.empty(total_rows, cols, dtype=odt, device=dev)
    elif out.shape != (total_rows, cols) or out.dtype != odt or out.device != dev \
            or not out.is_contiguous():
        _refuse(f"out: contiguous {odt} {(total_rows, cols)} on {dev}")
    args = Int8GemmArgs(G, N, K, total_rows, offs, gat, codes, scales, xp, xd, ldx, src_rows,
                        w.codes.data_ptr(), w.scales.data_ptr(), epilogue, out.data_ptr())
    L = lib()
    ref = ctypes.byref(args)
    n = L.int8_grouped_gemm_workspace_size(ref)
    ws = _ws(n, dev) if n else None
    _call(dev, L.int8_grouped_gemm, ref, None if ws is None else ws.data_ptr(), n)
    return out


# ------------------------------------------------- the router's balance loss
def _mask(mask: Optional[torch.Tensor], T: int, dev):
    if mask is None:
        return None
    if mask.dtype != torch.bool and mask.dtype != torch.uint8:
        _refuse("mask: bool [T]")
    return _vector(mask, T, mask.dtype, dev, "mask")


def moe_balance_loss(logits: torch.Tensor, topk_ids: torch.Tensor, *,
                     mask: Optional[torch.Tensor] = None) -> BalanceOut:
    """Slots per expert, mean router probabilities, balance loss and z-loss of
    logits [T, E] (bf16 or FP32, row stride honoured) and topk_ids [T, k]
    (int32, moe_route's; an id outside [0, E) is a dropped slot).  Rows with
    mask [T] (bool) false, or whose logits are all -inf, do not count."""
    if logits.dim() != 2 or topk_ids.dim() != 2 or topk_ids.shape[0] != logits.shape[0]:
        _refuse("logits [T, E] and topk_ids [T, k]")
    T, E = logits.shape
    k = topk_ids.shape[1]
    dev = logits.device
    dt = _dtype_code(logits)
    if dev.type != "cuda":
        _refuse("logits on a GPU")
    if topk_ids.dtype != torch.int32 or topk_ids.device != dev or not topk_ids.is_contiguous():
        _refuse(f"topk_ids: contiguous int32 [T, k] on {dev}")
    m = _mask(mask, T, dev)
    losses = torch.empty(2, dtype=torch.float32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    mean = torch.empty(E, dtype=torch.float32, device=dev)
    tokens = torch.empty(1, dtype=torch.int32, device=dev)
    L = lib()
    ws = _ws(L.moe_balance_loss_workspace_size(T, E), dev)
    _call(dev, L.moe_balance_loss, logits.data_ptr(), dt, T, E, _row_stride(logits, "logits"),
          topk_ids.data_ptr(), k, m, counts.data_ptr(), tokens.data_ptr(), mean.data_ptr(),
          losses.data_ptr(), ws.data_ptr(), ws.numel())
    return BalanceOut(losses, counts, mean, tokens)


def moe_balance_loss_backward(logits: torch.Tensor, k: int, counts: torch.Tensor,
                              tokens: torch.Tensor, grad_losses: torch.Tensor, *,
                              mask: Optional[torch.Tensor] = None,
                              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of the logits from that of moe_balance_loss's losses (float32
    [2]), with its counts and tokens.  out: where to write it, which may be
    logits itself."""
    if logits.dim() != 2:
        _refuse("logits [T, E]")
    T, E = logits.shape
    dev = logits.device
    dt = _dtype_code(logits)
    if dev.type != "cuda":
        _refuse("logits on a GPU")
    m = _mask(mask, T, dev)
    c = _vector(counts, E, torch.int32, dev, "counts")
    n = _vector(tokens, 1, torch.int32, dev, "tokens")
    g = _vector(grad_losses, 2, torch.float32, dev, "grad_losses")
    if out is None:
        out = torch.empty(T, E, dtype=logits.dtype, device=dev)
    elif out.shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
        _refuse("out like logits")
    _call(dev, lib().moe_balance_loss_backward, logits.data_ptr(), dt, T, E,
          _row_stride(logits, "logits"), k, m, c, n, g, out.data_ptr(), _row_stride(out, "out"))
    return out
