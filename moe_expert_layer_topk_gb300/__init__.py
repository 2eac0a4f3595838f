"""GB300 (sm_103a) MoE expert layer: router top-k -> dispatch -> grouped
gate/up GEMM + SwiGLU -> grouped down GEMM -> weighted combine, forward and
backward, as a C-ABI CUDA library (include/moe_topk.h).

This module is the thin Python binding: it loads libmoe_topk.so and exposes
every C entry point under the same name, taking torch tensors (device
memory) and passing their pointers, sizes and the current CUDA stream.  All
arithmetic runs in the library's kernels; nothing here computes the layer,
and there is no fallback -- calls fail loudly when the library is missing.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

import torch

from . import build as _build_mod

__all__ = ["lib", "MoEError", "LIB_PATH", "ENTRY_POINTS",
           "moe_route_topk", "moe_route_topk_chunks", "moe_route_topk_chunks_workspace_size",
           "moe_dispatch", "moe_dispatch_chunked", "moe_dispatch_e4m3_chunked", "moe_dispatch_no_alloc",
           "moe_grouped_gemm_swiglu",
           "moe_grouped_gemm_swiglu_gather", "moe_grouped_gemm_down", "moe_grouped_gemm_down_combine",
           "moe_quantize_rows_e4m3", "moe_dispatch_e4m3", "moe_grouped_gemm_swiglu_fp8",
           "moe_grouped_gemm_down_fp8",
           "moe_combine", "moe_combine_bwd", "moe_grouped_gemm_down_bwd",
           "moe_grouped_gemm_swiglu_bwd", "moe_grouped_gemm_down_bwd_dx", "moe_grouped_gemm_down_bwd_dw",
           "moe_grouped_gemm_swiglu_bwd_dx", "moe_grouped_gemm_swiglu_bwd_dw",
           "moe_dispatch_bwd", "moe_route_topk_bwd",
           "moe_route_topk_workspace_size", "moe_dispatch_workspace_size",
           "moe_route_topk_bwd_workspace_size", "moe_grouped_gemm_bwd_workspace_size",
           "moe_route_topk_logits", "moe_route_topk_logits_bwd",
           "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_balance_loss_bwd",
           "moe_dropout", "moe_combine_dropout", "moe_combine_dropout_bwd",
           "moe_adapter_hidden_size", "moe_adapter_linear", "moe_adapter_linear_bwd_workspace_size",
           "moe_adapter_linear_bwd",
           "moe_pre_norm", "moe_pre_norm_bwd_workspace_size", "moe_pre_norm_bwd", "moe_post_norm",
           "moe_combine_post_norm", "moe_post_norm_bwd_workspace_size", "moe_post_norm_bwd",
           "moe_ckpt_pack", "moe_ckpt_unpack", "moe_dispatch_rows", "moe_grouped_gemm_swiglu_ckpt",
           "moe_grouped_gemm_down_bwd_ckpt_workspace_size", "moe_grouped_gemm_down_bwd_ckpt",
           "moe_read_device_status", "moe_abi_version", "moe_probe_fma", "moe_set_gemm_sm_limit", "sm_count"]

LIB_PATH: Path = _build_mod.LIB

_P, _I, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
_L, _F, _D = ctypes.c_longlong, ctypes.c_float, ctypes.c_double

# name -> (argtypes, restype); mirrors include/moe_topk.h
# the ABI version of include/moe_topk.h these signatures follow
ABI_VERSION = 103

ENTRY_POINTS = {
    "moe_abi_version": ([], _I),
    "moe_last_error_string": ([], ctypes.c_char_p),
    "moe_read_device_status": ([_P, _I, _P], _I),
    "moe_route_topk_workspace_size": ([_I, _I, _I], _Z),
    "moe_route_topk": ([_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_route_topk_chunks_workspace_size": ([_I, _I, _I], _Z),
    "moe_route_topk_chunks": ([_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_dispatch_workspace_size": ([_I, _I, _I], _Z),
    "moe_dispatch_chunked": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_dispatch_e4m3_chunked": ([_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P], _I),
    "moe_dispatch": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P], _I),
    "moe_dispatch_no_alloc_max_scratch": ([], _Z),
    "moe_dispatch_no_alloc": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_grouped_gemm_swiglu": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _Z, _P], _I),
    "moe_grouped_gemm_swiglu_gather": ([_P, _P, _I, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P], _I),
    "moe_grouped_gemm_down": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _Z, _P], _I),
    "moe_grouped_gemm_down_combine": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P, _P, _P], _I),
    "moe_quantize_rows_e4m3": ([_P, _I, _I, _P, _P, _P], _I),
    "moe_dispatch_e4m3": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_grouped_gemm_swiglu_fp8": ([_P, _P, _P, _I, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_grouped_gemm_down_fp8": ([_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_combine": ([_P, _P, _P, _I, _I, _I, _P, _P], _I),
    "moe_combine_bwd": ([_P, _P, _P, _P, _I, _I, _I, _P, _P, _P], _I),
    "moe_grouped_gemm_bwd_workspace_size": ([_I], _Z),
    "moe_grouped_gemm_down_bwd": ([_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _Z, _P], _I),
    "moe_grouped_gemm_swiglu_bwd": ([_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _Z, _P],
                                    _I),
    "moe_grouped_gemm_down_bwd_dx": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_grouped_gemm_down_bwd_dw": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _I, _P, _Z, _P], _I),
    "moe_grouped_gemm_swiglu_bwd_dx": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P], _I),
    "moe_grouped_gemm_swiglu_bwd_dw": ([_P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _Z, _P], _I),
    "moe_dispatch_bwd": ([_P, _P, _I, _I, _I, _P, _P], _I),
    "moe_route_topk_bwd_workspace_size": ([_I, _I, _I], _Z),
    "moe_route_topk_bwd": ([_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _Z, _P], _I),
    "moe_route_topk_logits": ([_P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P], _I),
    "moe_route_topk_logits_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _Z, _P], _I),
    "moe_balance_loss_workspace_size": ([_I, _I, _I], _Z),
    "moe_balance_loss": ([_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _F, _F, _P, _P, _Z, _P], _I),
    "moe_balance_loss_bwd": ([_P, _P, _I, _I, _I, _I, _P, _P, _P, _F, _F, _P, _P, _P], _I),
    "moe_dropout": ([_P, _P, _L, _I, _D, _P, _P, _P], _I),
    "moe_combine_dropout": ([_P, _P, _P, _P, _I, _I, _I, _D, _P, _P, _P], _I),
    "moe_combine_dropout_bwd": ([_P, _P, _P, _P, _I, _I, _I, _D, _P, _P, _P, _P], _I),
    "moe_adapter_hidden_size": ([_I, _I], _Z),
    "moe_adapter_linear": ([_P, _L, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _Z, _P, _L, _P], _I),
    "moe_adapter_linear_bwd_workspace_size": ([_I, _I, _I, _I, _I], _Z),
    "moe_adapter_linear_bwd": ([_P, _L, _P, _L, _P, _P, _P, _P, _P, _Z, _I, _P, _P, _I, _I, _I, _I, _I, _P, _L, _P, _P,
                                _I, _P, _Z, _P], _I),
    "moe_pre_norm": ([_P, _L, _I, _P, _F, _I, _I, _P, _L, _P, _P], _I),
    "moe_pre_norm_bwd_workspace_size": ([_I, _I], _Z),
    "moe_pre_norm_bwd": ([_P, _L, _P, _L, _I, _P, _P, _P, _L, _F, _I, _I, _P, _L, _P, _I, _P, _Z, _P], _I),
    "moe_post_norm": ([_P, _P, _I, _P, _I, _F, _I, _P, _F, _F, _I, _I, _P, _P, _P, _P, _P, _P], _I),
    "moe_combine_post_norm": ([_P, _P, _P, _P, _I, _P, _I, _F, _I, _P, _F, _F, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P], _I),
    "moe_post_norm_bwd_workspace_size": ([_I, _I], _Z),
    "moe_post_norm_bwd": ([_P, _I, _P, _P, _I, _P, _I, _P, _F, _I, _I, _P, _P, _P, _I, _P, _Z, _P], _I),
    "moe_ckpt_pack": ([_P, _I, _I, _P, _P, _P], _I),
    "moe_ckpt_unpack": ([_P, _P, _I, _I, _P, _P], _I),
    "moe_dispatch_rows": ([_P, _P, _P, _P, _I, _I, _I, _P, _P, _P], _I),
    "moe_grouped_gemm_swiglu_ckpt": ([_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P], _I),
    "moe_grouped_gemm_down_bwd_ckpt_workspace_size": ([_I, _I], _Z),
    "moe_grouped_gemm_down_bwd_ckpt": ([_P, _P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P, _P, _Z,
                                        _P], _I),
    "moe_probe_fma": ([_I, _I, _I, _P, ctypes.POINTER(ctypes.c_longlong), _P], _I),
    "moe_set_gemm_sm_limit": ([_I, ctypes.POINTER(ctypes.c_int)], _I),
}

_lib = None


class MoEError(RuntimeError):
    def __init__(self, name: str, code: int, msg: str):
        super().__init__(f"{name} failed with code {code}: {msg}")
        self.code = code


def lib(path: Path | str | None = None) -> ctypes.CDLL:
    """The loaded CUDA library.  Raises if it has not been built."""
    global _lib
    if _lib is None or path is not None:
        p = Path(path) if path is not None else LIB_PATH
        if not p.exists():
            raise RuntimeError(f"CUDA library {p} is not built: run "
                               f"`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(str(p))
        version = getattr(L, "moe_abi_version", None)
        if version is None or version() != ABI_VERSION:
            raise RuntimeError(f"CUDA library {p} has ABI version {version and version()}, this binding "
                               f"expects {ABI_VERSION}: rebuild it")
        for name, (args, res) in ENTRY_POINTS.items():
            f = getattr(L, name, None)
            if f is None:  # added calls leave the version as it is
                raise RuntimeError(f"CUDA library {p} has no {name}, it is older than this binding: rebuild it")
            f.argtypes = args
            f.restype = res
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    raise ValueError("tensor arguments must be contiguous")


# the raw handle of the current stream without building a Stream object
# (torch.cuda.current_stream() costs about 3 us a call, a third of a small
# kernel call's host time)
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_current_stream is not None:
            return _raw_current_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _call(name, *args):
    rc = getattr(_lib or lib(), name)(*args)
    if rc != 0:
        raise MoEError(name, rc, lib().moe_last_error_string().decode(errors="replace"))


def _nbytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# ------------------------------------------------- entry points (same names)

def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_route_topk_workspace_size(T, H, E) -> int:
    return lib().moe_route_topk_workspace_size(T, H, E)


def moe_route_topk_chunks_workspace_size(T, H, E) -> int:
    return lib().moe_route_topk_chunks_workspace_size(T, H, E)


def moe_dispatch_workspace_size(T, E, k) -> int:
    return lib().moe_dispatch_workspace_size(T, E, k)


def moe_route_topk_bwd_workspace_size(T, H, E) -> int:
    return lib().moe_route_topk_bwd_workspace_size(T, H, E)


def moe_grouped_gemm_bwd_workspace_size(num_seg) -> int:
    return lib().moe_grouped_gemm_bwd_workspace_size(num_seg)


def moe_read_device_status(reset: bool = True, stream=None) -> int:
    v = ctypes.c_int(0)
    _call("moe_read_device_status", ctypes.addressof(v), int(reset), _stream(stream))
    return v.value


def moe_route_topk(x, Wr, bias, T, H, E, k, ep_size, topk_idx, topk_w, counts, offsets,
                   rank_offsets, ws, stream=None):
    _call("moe_route_topk", _ptr(x), _ptr(Wr), _ptr(bias), T, H, E, k, ep_size, _ptr(topk_idx),
          _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(rank_offsets), _ptr(ws), _nbytes(ws),
          _stream(stream))


def moe_route_topk_chunks(x, Wr, bias, T, H, E, k, ep_size, topk_idx, topk_w, counts, offsets,
                          rank_offsets, chunk_prefix, ws, stream=None):
    _call("moe_route_topk_chunks", _ptr(x), _ptr(Wr), _ptr(bias), T, H, E, k, ep_size, _ptr(topk_idx),
          _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(rank_offsets), _ptr(chunk_prefix), _ptr(ws),
          _nbytes(ws), _stream(stream))


def moe_dispatch_chunked(x, topk_idx, offsets, chunk_prefix, T, H, E, k, x_perm, row_of_slot, token_of_row,
                         stream=None):
    _call("moe_dispatch_chunked", _ptr(x), _ptr(topk_idx), _ptr(offsets), _ptr(chunk_prefix), T, H, E, k,
          _ptr(x_perm), _ptr(row_of_slot), _ptr(token_of_row), _stream(stream))


def moe_dispatch_e4m3_chunked(x, topk_idx, offsets, chunk_prefix, T, H, E, k, xq_perm, xs_perm, row_of_slot,
                              token_of_row, stream=None):
    _call("moe_dispatch_e4m3_chunked", _ptr(x), _ptr(topk_idx), _ptr(offsets), _ptr(chunk_prefix), T, H, E, k,
          _ptr(xq_perm), _ptr(xs_perm), _ptr(row_of_slot), _ptr(token_of_row), _stream(stream))


def moe_dispatch(x, topk_idx, offsets, T, H, E, k, x_perm, row_of_slot, token_of_row, ws,
                 stream=None):
    _call("moe_dispatch", _ptr(x), _ptr(topk_idx), _ptr(offsets), T, H, E, k, _ptr(x_perm),
          _ptr(row_of_slot), _ptr(token_of_row), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_dispatch_no_alloc(x, topk_idx, offsets, T, H, E, k, x_perm, row_of_slot, token_of_row,
                          stream=None):
    """moe_dispatch with the library's built-in scratch instead of a workspace."""
    _call("moe_dispatch_no_alloc", _ptr(x), _ptr(topk_idx), _ptr(offsets), T, H, E, k, _ptr(x_perm),
          _ptr(row_of_slot), _ptr(token_of_row), _stream(stream))


def moe_grouped_gemm_swiglu(x_perm, Wg, Wu, num_seg, seg_offsets, seg_expert, R, H, I, E, h,
                            gu_save=None, ws=None, stream=None):
    _call("moe_grouped_gemm_swiglu", _ptr(x_perm), _ptr(Wg), _ptr(Wu), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(h), _ptr(gu_save), _ptr(ws), _nbytes(ws),
          _stream(stream))


def moe_grouped_gemm_swiglu_gather(x, token_of_row, T, Wg, Wu, num_seg, seg_offsets, seg_expert, R, H,
                                   I, E, h, gu_save=None, stream=None):
    _call("moe_grouped_gemm_swiglu_gather", _ptr(x), _ptr(token_of_row), T, _ptr(Wg), _ptr(Wu), num_seg,
          _ptr(seg_offsets), _ptr(seg_expert), R, H, I, E, _ptr(h), _ptr(gu_save), _stream(stream))


def moe_grouped_gemm_down(h, Wd, num_seg, seg_offsets, seg_expert, R, H, I, E, y_perm, ws=None,
                          stream=None):
    _call("moe_grouped_gemm_down", _ptr(h), _ptr(Wd), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(y_perm), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_grouped_gemm_down_combine(h, Wd, num_seg, seg_offsets, seg_expert, R, H, I, E, token_of_row,
                                  row_of_slot, topk_w, T, k, y_acc, y, stream=None):
    _call("moe_grouped_gemm_down_combine", _ptr(h), _ptr(Wd), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(token_of_row), _ptr(row_of_slot), _ptr(topk_w), T, k,
          _ptr(y_acc), _ptr(y), _stream(stream))


def moe_quantize_rows_e4m3(a, rows, cols, q, scale, stream=None):
    _call("moe_quantize_rows_e4m3", _ptr(a), rows, cols, _ptr(q), _ptr(scale), _stream(stream))


def moe_dispatch_e4m3(x, topk_idx, offsets, T, H, E, k, xq_perm, xs_perm, row_of_slot, token_of_row, ws,
                      stream=None):
    _call("moe_dispatch_e4m3", _ptr(x), _ptr(topk_idx), _ptr(offsets), T, H, E, k, _ptr(xq_perm), _ptr(xs_perm),
          _ptr(row_of_slot), _ptr(token_of_row), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_grouped_gemm_swiglu_fp8(a, a_scale, token_of_row, T, Wg, Wg_scale, Wu, Wu_scale, num_seg,
                                seg_offsets, seg_expert, R, H, I, E, h, stream=None):
    _call("moe_grouped_gemm_swiglu_fp8", _ptr(a), _ptr(a_scale), _ptr(token_of_row), T, _ptr(Wg),
          _ptr(Wg_scale), _ptr(Wu), _ptr(Wu_scale), num_seg, _ptr(seg_offsets), _ptr(seg_expert), R, H,
          I, E, _ptr(h), _stream(stream))


def moe_grouped_gemm_down_fp8(h, h_scale, Wd, Wd_scale, num_seg, seg_offsets, seg_expert, R, H, I, E,
                              y_perm, stream=None):
    _call("moe_grouped_gemm_down_fp8", _ptr(h), _ptr(h_scale), _ptr(Wd), _ptr(Wd_scale), num_seg,
          _ptr(seg_offsets), _ptr(seg_expert), R, H, I, E, _ptr(y_perm), _stream(stream))


def moe_combine(y_perm, topk_w, row_of_slot, T, H, k, y, stream=None):
    _call("moe_combine", _ptr(y_perm), _ptr(topk_w), _ptr(row_of_slot), T, H, k, _ptr(y),
          _stream(stream))


def moe_combine_bwd(dy, y_perm, topk_w, row_of_slot, T, H, k, dy_perm, d_w, stream=None):
    _call("moe_combine_bwd", _ptr(dy), _ptr(y_perm), _ptr(topk_w), _ptr(row_of_slot), T, H, k,
          _ptr(dy_perm), _ptr(d_w), _stream(stream))


def moe_grouped_gemm_down_bwd(dy_perm, h, gu_save, Wd, num_seg, seg_offsets, seg_expert, R, H, I,
                              E, dgu, dWd, accumulate=0, ws=None, stream=None):
    _call("moe_grouped_gemm_down_bwd", _ptr(dy_perm), _ptr(h), _ptr(gu_save), _ptr(Wd), num_seg,
          _ptr(seg_offsets), _ptr(seg_expert), R, H, I, E, _ptr(dgu), _ptr(dWd), int(accumulate),
          _ptr(ws), _nbytes(ws), _stream(stream))


def moe_grouped_gemm_swiglu_bwd(dgu, x_perm, Wg, Wu, num_seg, seg_offsets, seg_expert, R, H, I, E,
                                dx_perm, dWg, dWu, accumulate=0, ws=None, stream=None):
    _call("moe_grouped_gemm_swiglu_bwd", _ptr(dgu), _ptr(x_perm), _ptr(Wg), _ptr(Wu), num_seg,
          _ptr(seg_offsets), _ptr(seg_expert), R, H, I, E, _ptr(dx_perm), _ptr(dWg), _ptr(dWu),
          int(accumulate), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_grouped_gemm_down_bwd_dx(dy_perm, gu_save, Wd, num_seg, seg_offsets, seg_expert, R, H, I, E, dgu,
                                 stream=None):
    _call("moe_grouped_gemm_down_bwd_dx", _ptr(dy_perm), _ptr(gu_save), _ptr(Wd), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(dgu), _stream(stream))


def moe_grouped_gemm_down_bwd_dw(dy_perm, h, num_seg, seg_offsets, seg_expert, R, H, I, E, dWd, accumulate=0,
                                 ws=None, stream=None):
    _call("moe_grouped_gemm_down_bwd_dw", _ptr(dy_perm), _ptr(h), num_seg, _ptr(seg_offsets), _ptr(seg_expert),
          R, H, I, E, _ptr(dWd), int(accumulate), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_grouped_gemm_swiglu_bwd_dx(dgu, Wg, Wu, num_seg, seg_offsets, seg_expert, R, H, I, E, dx_perm,
                                   stream=None):
    _call("moe_grouped_gemm_swiglu_bwd_dx", _ptr(dgu), _ptr(Wg), _ptr(Wu), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(dx_perm), _stream(stream))


def moe_grouped_gemm_swiglu_bwd_dw(dgu, x_perm, num_seg, seg_offsets, seg_expert, R, H, I, E, dWg, dWu,
                                   accumulate=0, ws=None, stream=None):
    _call("moe_grouped_gemm_swiglu_bwd_dw", _ptr(dgu), _ptr(x_perm), num_seg, _ptr(seg_offsets),
          _ptr(seg_expert), R, H, I, E, _ptr(dWg), _ptr(dWu), int(accumulate), _ptr(ws), _nbytes(ws),
          _stream(stream))


def moe_dispatch_bwd(dx_perm, row_of_slot, T, H, k, dx_acc, stream=None):
    _call("moe_dispatch_bwd", _ptr(dx_perm), _ptr(row_of_slot), T, H, k, _ptr(dx_acc),
          _stream(stream))


def moe_route_topk_bwd(d_w, topk_w, topk_idx, x, Wr, dx_acc, T, H, E, k, dWr, dx, accumulate=0,
                       ws=None, stream=None):
    _call("moe_route_topk_bwd", _ptr(d_w), _ptr(topk_w), _ptr(topk_idx), _ptr(x), _ptr(Wr),
          _ptr(dx_acc), T, H, E, k, _ptr(dWr), _ptr(dx), int(accumulate), _ptr(ws), _nbytes(ws),
          _stream(stream))


def moe_route_topk_logits(x, Wr, bias, T, H, E, k, ep_size, topk_idx, topk_w, counts, offsets, rank_offsets,
                          chunk_prefix, logits, ws, stream=None):
    _call("moe_route_topk_logits", _ptr(x), _ptr(Wr), _ptr(bias), T, H, E, k, ep_size, _ptr(topk_idx),
          _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(rank_offsets), _ptr(chunk_prefix), _ptr(logits),
          _ptr(ws), _nbytes(ws), _stream(stream))


def moe_route_topk_logits_bwd(d_w, topk_w, topk_idx, dlogits, x, Wr, dx_acc, T, H, E, k, dWr, dx, accumulate=0,
                              ws=None, stream=None):
    _call("moe_route_topk_logits_bwd", _ptr(d_w), _ptr(topk_w), _ptr(topk_idx), _ptr(dlogits), _ptr(x),
          _ptr(Wr), _ptr(dx_acc), T, H, E, k, _ptr(dWr), _ptr(dx), int(accumulate), _ptr(ws), _nbytes(ws),
          _stream(stream))


def moe_balance_loss_workspace_size(T, E, num_seg=1) -> int:
    return lib().moe_balance_loss_workspace_size(T, E, num_seg)


def moe_balance_loss(logits, topk_idx, mask, T, E, k, num_seg, seg_offsets, counts, tokens, prob_sum, loss,
                     balance_coef, z_coef, dlogits, ws, stream=None):
    _call("moe_balance_loss", _ptr(logits), _ptr(topk_idx), _ptr(mask), T, E, k, num_seg, _ptr(seg_offsets),
          _ptr(counts), _ptr(tokens), _ptr(prob_sum), _ptr(loss), balance_coef, z_coef, _ptr(dlogits), _ptr(ws),
          _nbytes(ws), _stream(stream))


def moe_balance_loss_bwd(logits, mask, T, E, k, num_seg, seg_offsets, counts, tokens, balance_coef, z_coef, dloss,
                         dlogits, stream=None):
    _call("moe_balance_loss_bwd", _ptr(logits), _ptr(mask), T, E, k, num_seg, _ptr(seg_offsets), _ptr(counts),
          _ptr(tokens), balance_coef, z_coef, _ptr(dloss), _ptr(dlogits), _stream(stream))


def _dropout_type(x, out) -> int:
    """0 for bf16 tensors, 1 for fp32 ones."""
    if x.dtype != out.dtype or x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x and out must both be bf16 or both fp32")
    return int(x.dtype == torch.float32)


def moe_dropout(x, residual, n, p, rng, out, stream=None):
    """out = residual + D(x) over n elements, bf16 or fp32 by x's type; rng: int64 [2] {seed, offset}."""
    if residual is not None and residual.dtype != x.dtype:
        raise ValueError("residual must have x's type")
    _call("moe_dropout", _ptr(x), _ptr(residual), n, _dropout_type(x, out), p, _ptr(rng), _ptr(out), _stream(stream))


def moe_combine_dropout(y_perm, topk_w, row_of_slot, residual, T, H, k, p, rng, y, stream=None):
    _call("moe_combine_dropout", _ptr(y_perm), _ptr(topk_w), _ptr(row_of_slot), _ptr(residual), T, H, k, p,
          _ptr(rng), _ptr(y), _stream(stream))


def moe_combine_dropout_bwd(dy, y_perm, topk_w, row_of_slot, T, H, k, p, rng, dy_perm, d_w, stream=None):
    _call("moe_combine_dropout_bwd", _ptr(dy), _ptr(y_perm), _ptr(topk_w), _ptr(row_of_slot), T, H, k, p,
          _ptr(rng), _ptr(dy_perm), _ptr(d_w), _stream(stream))


def _rows(t, dtype=None):
    """Pointer and row stride of a 2-D tensor (of that type) whose rows may lie apart."""
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"a tensor of {t.dtype} where {dtype} is read or written")
    st = t.stride()
    if len(st) != 2 or st[1] != 1:
        raise ValueError("row tensors must be 2-D with contiguous rows")
    if not t.is_cuda:
        raise ValueError("tensor arguments must live on the GPU")
    n, cols = t.shape
    return t.data_ptr(), st[0] if n > 1 else cols


def moe_adapter_hidden_size(T, r) -> int:
    return lib().moe_adapter_hidden_size(T, r)


def moe_adapter_linear_bwd_workspace_size(T, K, N, r, num_seg) -> int:
    return lib().moe_adapter_linear_bwd_workspace_size(T, K, N, r, num_seg)


def moe_adapter_linear(x, W, A, B, scale, num_seg, seg_offsets, seg_adapter, T, K, N, r, num_adapters, hidden, y,
                       stream=None):
    """y = x W^T plus each request's adapter; x and y may be row slices of wider tensors."""
    px, ldx = _rows(x)
    py, ldy = _rows(y)
    _call("moe_adapter_linear", px, ldx, _ptr(W), _ptr(A), _ptr(B), _ptr(scale), num_seg, _ptr(seg_offsets),
          _ptr(seg_adapter), T, K, N, r, num_adapters, _ptr(hidden), _nbytes(hidden), py, ldy, _stream(stream))


def moe_adapter_linear_bwd(dy, x, W, A, B, scale, hidden, num_seg, seg_offsets, seg_adapter, T, K, N, r, num_adapters,
                           dx, dA, dB, accumulate=0, ws=None, stream=None):
    pd, lddy = _rows(dy)
    px, ldx = _rows(x)
    po, lddx = _rows(dx)
    _call("moe_adapter_linear_bwd", pd, lddy, px, ldx, _ptr(W), _ptr(A), _ptr(B), _ptr(scale), _ptr(hidden),
          _nbytes(hidden), num_seg, _ptr(seg_offsets), _ptr(seg_adapter), T, K, N, r, num_adapters, po, lddx, _ptr(dA),
          _ptr(dB), int(accumulate), _ptr(ws), _nbytes(ws), _stream(stream))


def _stream_type(*tensors) -> int:
    """0 where the residual stream's tensors are bf16, 1 where they are fp32."""
    dt = tensors[0].dtype
    for t in tensors:
        if t is not None and t.dtype is not dt:
            raise ValueError("the residual stream's tensors must all be bf16 or all fp32")
    if dt is torch.bfloat16:
        return 0
    if dt is torch.float32:
        return 1
    raise ValueError("the residual stream's tensors must all be bf16 or all fp32")


def _gate_kind(gate, T, H) -> int:
    """0 without a gate, 1 for fp32 logits of T tokens, 2 for bf16 logits of T x H elements."""
    if gate is None:
        return 0
    if gate.dtype == torch.float32 and gate.numel() == T:
        return 1
    if gate.dtype == torch.bfloat16 and gate.numel() == T * H:
        return 2
    raise ValueError("gate must be fp32 logits of the tokens or bf16 logits of their elements")


def _pointer_of(dtype, what):
    """_ptr for tensors that are read or written as dtype."""
    def pointer(t):
        if t is None:
            return None
        try:
            if t.dtype is dtype and t.is_cuda and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:  # an address
            return _ptr(t)
        if t.dtype is not dtype:
            raise ValueError(f"{what}, not {t.dtype}")
        return _ptr(t)
    return pointer


_bf16 = _pointer_of(torch.bfloat16, "what enters and leaves a block or an expert is bf16")
_f32 = _pointer_of(torch.float32, "rows' statistics, weights and their gradients are fp32")
_fp32 = _pointer_of(torch.float32, "gains and their gradients are fp32")


def _codes(q, scale):
    """Pointers of 8-bit codes and their bf16 scales."""
    if q.element_size() != 1 or scale.dtype is not torch.bfloat16:
        raise ValueError("codes are 8-bit, their scales bf16")
    return _ptr(q), _ptr(scale)


def moe_pre_norm(x, gain, eps, T, H, y, rstd=None, stream=None):
    """y = x / rms(x) * gain; x bf16 or fp32, x and y may be row slices of wider tensors."""
    px, ldx = _rows(x)
    py, ldy = _rows(y, torch.bfloat16)
    _call("moe_pre_norm", px, ldx, _stream_type(x), _fp32(gain), eps, T, H, py, ldy, _f32(rstd), _stream(stream))


def moe_pre_norm_bwd_workspace_size(T, H) -> int:
    return lib().moe_pre_norm_bwd_workspace_size(T, H)


def moe_pre_norm_bwd(dy, x, gain, rstd, dres, res_scale, T, H, dx, dgain=None, accumulate=0, ws=None, stream=None):
    pd, lddy = _rows(dy, torch.bfloat16)
    px, ldx = _rows(x)
    pr, lddres = (None, H) if dres is None else _rows(dres)
    po, lddx = _rows(dx)
    _call("moe_pre_norm_bwd", pd, lddy, px, ldx, _stream_type(x, dres, dx), _fp32(gain), _f32(rstd), pr, lddres, res_scale,
          T, H, po, lddx, _fp32(dgain), int(accumulate), _ptr(ws), _nbytes(ws), _stream(stream))


def moe_post_norm(z, residual, gain, norm, eps, gate, res_scale, out_scale, T, H, out, rstd=None, next_gain=None,
                  next_y=None, next_rstd=None, stream=None):
    """out = res_scale residual + out_scale sigmoid(gate) norm(z) gain, and the next norm of out where next_y is given;
    the stream's type is out's, the gate's kind its own (fp32 [T] or bf16 [T,H])."""
    _call("moe_post_norm", _bf16(z), _ptr(residual), _stream_type(out, residual), _fp32(gain), int(norm), eps,
          _gate_kind(gate, T, H), _ptr(gate), res_scale, out_scale, T, H, _ptr(out), _f32(rstd), _fp32(next_gain),
          _bf16(next_y), _f32(next_rstd), _stream(stream))


def moe_combine_post_norm(y_perm, topk_w, row_of_slot, residual, gain, norm, eps, gate, res_scale, out_scale, T, H, k, z,
                          out, rstd=None, next_gain=None, next_y=None, next_rstd=None, stream=None):
    _call("moe_combine_post_norm", _bf16(y_perm), _f32(topk_w), _ptr(row_of_slot), _ptr(residual),
          _stream_type(out, residual), _fp32(gain), int(norm), eps, _gate_kind(gate, T, H), _ptr(gate), res_scale, out_scale,
          T, H, k, _bf16(z), _ptr(out), _f32(rstd), _fp32(next_gain), _bf16(next_y), _f32(next_rstd), _stream(stream))


def moe_post_norm_bwd_workspace_size(T, H) -> int:
    return lib().moe_post_norm_bwd_workspace_size(T, H)


def moe_post_norm_bwd(dout, z, gain, norm, rstd, gate, out_scale, T, H, dz, dgain=None, dgate=None, accumulate=0, ws=None,
                      stream=None):
    if dgate is not None and (gate is None or dgate.dtype != gate.dtype):
        raise ValueError("dgate must have the gate's type")
    _call("moe_post_norm_bwd", _ptr(dout), _stream_type(dout), _bf16(z), _fp32(gain), int(norm), _f32(rstd),
          _gate_kind(gate, T, H), _ptr(gate), out_scale, T, H, _bf16(dz), _fp32(dgain), _ptr(dgate), int(accumulate), _ptr(ws),
          _nbytes(ws), _stream(stream))


def moe_ckpt_pack(a, rows, cols, q, scale, stream=None):
    _call("moe_ckpt_pack", _bf16(a), rows, cols, *_codes(q, scale), _stream(stream))


def moe_ckpt_unpack(q, scale, rows, cols, a, stream=None):
    _call("moe_ckpt_unpack", *_codes(q, scale), rows, cols, _bf16(a), _stream(stream))


def moe_dispatch_rows(x, scale, row_of_slot, topk_w, T, H, k, x_perm, row_w=None, stream=None):
    """x: bf16 tokens (scale None), or int8 codes with their scales."""
    if x.dtype is not torch.bfloat16 if scale is None else x.element_size() != 1:
        raise ValueError("x must be bf16 tokens, or 8-bit codes with their scales")
    _call("moe_dispatch_rows", _ptr(x), _bf16(scale), _ptr(row_of_slot), _f32(topk_w), T, H, k, _bf16(x_perm), _f32(row_w),
          _stream(stream))


def moe_grouped_gemm_swiglu_ckpt(x_perm, Wg, Wu, num_seg, seg_offsets, seg_expert, R, H, I, E, h, gu_q, gu_scale,
                                 stream=None):
    _call("moe_grouped_gemm_swiglu_ckpt", _bf16(x_perm), _bf16(Wg), _bf16(Wu), num_seg, _ptr(seg_offsets), _ptr(seg_expert),
          R, H, I, E, _bf16(h), *_codes(gu_q, gu_scale), _stream(stream))


def moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I) -> int:
    return lib().moe_grouped_gemm_down_bwd_ckpt_workspace_size(R, I)


def moe_grouped_gemm_down_bwd_ckpt(dy_perm, row_w, gu_q, gu_scale, Wd, num_seg, seg_offsets, seg_expert, R, H, I, E, dgu,
                                   h_w, d_w, row_of_slot=None, T=0, k=0, ws=None, stream=None):
    _call("moe_grouped_gemm_down_bwd_ckpt", _bf16(dy_perm), _f32(row_w), *_codes(gu_q, gu_scale), _bf16(Wd), num_seg,
          _ptr(seg_offsets), _ptr(seg_expert), R, H, I, E, _bf16(dgu), _bf16(h_w), _ptr(row_of_slot), T, k, _f32(d_w), _ptr(ws),
          _nbytes(ws), _stream(stream))


def moe_set_gemm_sm_limit(max_sms: int) -> int:
    """Limit the grouped GEMMs issued from this thread to max_sms SMs (0 = all);
    returns the previous limit."""
    prev = ctypes.c_int(0)
    _call("moe_set_gemm_sm_limit", int(max_sms), ctypes.byref(prev))
    return prev.value


def sm_count(device=None) -> int:
    return torch.cuda.get_device_properties(device if device is not None else torch.cuda.current_device()) \
        .multi_processor_count


from .layer import AdapterLinear, MoEBlock, MoELayer  # noqa: E402  (buffers + call sequence over the entry points)

__all__ += ["MoELayer", "MoEBlock", "AdapterLinear"]


def moe_probe_fma(packed, per_sm, iters, out, stream=None) -> int:
    """Launch the FMA-rate probe; returns the number of FMAs it performs."""
    n = ctypes.c_longlong(0)
    _call("moe_probe_fma", int(packed), int(per_sm), int(iters), _ptr(out), ctypes.byref(n), _stream(stream))
    return int(n.value)

