"""GB300-native (sm_103a) FlashAttention-2-style attention forward.

The compute lives in ``_build/libfa_gb300.so`` (hand-written CUDA: TMA,
tcgen05 MMAs into tensor memory, online softmax).  This module is a thin
ctypes binding with the C ABI's names (``include/fa.h``): it only marshals
arguments.  torch is used for device memory and streams.  There is no CPU
or library fallback: if the shared library cannot be built or loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import threading

from . import build as _build

__all__ = ["fa_fwd", "fa_fwd_raw", "fa_fwd_window", "fa_fwd_window_raw", "fa_strerror", "fa_device_status",
           "fa_selftest_bounded_wait", "fa_selftest_fwd_timeout", "fa_selftest_bwd_timeout", "fa_selftest_splitkv_timeout",
           "fa_selftest_paged_chunk_timeout", "fa_version", "FAError", "lib", "library_path",
           "FA_OK", "FA_ERR_NULLPTR", "FA_ERR_BAD_SHAPE", "FA_ERR_UNSUPPORTED_D",
           "FA_ERR_UNSUPPORTED_CAUSAL", "FA_ERR_MISALIGNED", "FA_ERR_BAD_SCALE", "FA_ERR_CUDA",
           "FA_ERR_TIMEOUT", "FA_ERR_ALIAS", "FA_ERR_BAD_WINDOW", "FA_ERR_WORKSPACE",
           "fa_fwd_splitkv", "fa_fwd_splitkv_raw", "fa_fwd_splitkv_workspace_bytes",
           "fa_splitkv_num_splits", "FA_ERR_SCRATCH_LIMIT",
           "fa_bwd", "fa_bwd_raw", "fa_fwd_fp8", "fa_fwd_fp8_raw",
           "fa_fwd_blockmask", "fa_fwd_blockmask_raw", "FA_ERR_BAD_MASK", "FA_BLOCK_M", "FA_BLOCK_N",
           "fa_kv_plan", "fa_kv_plan_raw", "fa_kv_append", "fa_kv_append_raw", "fa_page_select", "fa_page_select_raw",
           "fa_fwd_paged", "fa_fwd_paged_raw", "fa_fwd_paged_workspace_bytes", "FA_ERR_BAD_PAGE", "FA_PAGE_SIZES",
           "fa_kv_plan_positions_raw", "fa_kv_append_rope", "fa_kv_append_rope_raw",
           "fa_fwd_paged_chunk", "fa_fwd_paged_chunk_raw", "fa_fwd_paged_chunk_workspace_bytes",
           "fa_rope", "fa_rope_raw", "fa_rope_bwd", "fa_rope_bwd_raw", "fa_rope_phases", "FA_ROPE_SCALINGS"]

FA_OK = 0
FA_ERR_NULLPTR = -1
FA_ERR_BAD_SHAPE = -2
FA_ERR_UNSUPPORTED_D = -3
FA_ERR_UNSUPPORTED_CAUSAL = -4
FA_ERR_MISALIGNED = -5
FA_ERR_BAD_SCALE = -6
FA_ERR_CUDA = -7
FA_ERR_TIMEOUT = -8
FA_ERR_ALIAS = -9
FA_ERR_BAD_WINDOW = -10
FA_ERR_WORKSPACE = -11
FA_ERR_SCRATCH_LIMIT = -12
FA_ERR_BAD_MASK = -13
FA_ERR_BAD_PAGE = -14
FA_BLOCK_M = 128  # query rows per block-mask row
FA_BLOCK_N = 128  # keys per block-mask column
FA_PAGE_SIZES = (16, 32, 64, 128)  # tokens per page of the paged cache
FA_ROPE_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}  # how fa_rope_phases stretches frequencies

_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i = ctypes.c_int
_ll = ctypes.c_longlong
_d = ctypes.c_double

# name -> (restype, argtypes), mirroring include/fa.h
_SIGNATURES = {
    "fa_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _vp]),
    "fa_fwd_window": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i,
                           _vp]),
    "fa_fwd_blockmask": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _i,
                              _vp, _i, _i, _vp]),
    "fa_fwd_splitkv": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i, _vp,
                            ctypes.c_size_t, _vp]),
    "fa_fwd_splitkv_workspace_bytes": (ctypes.c_size_t, [_i, _i, _i, _i, _i, _i]),
    "fa_fwd_splitkv_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float,
                                    _i, _vp]),
    "fa_splitkv_num_splits": (_i, [_i, _i, _i, _i, _i]),
    "fa_bwd": (_i, [_vp] * 10 + [_i, _i, _i, _i, _i, ctypes.c_float, _i, _vp]),
    "fa_fwd_fp8": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float, _i,
                        ctypes.c_float, ctypes.c_float, ctypes.c_float, _vp]),
    "fa_kv_plan": (_i, [_vp] * 9 + [_i] * 6 + [_vp]),
    "fa_kv_append": (_i, [_vp] * 9 + [_i] * 3 + [_ll] * 2 + [_i] * 2 + [_vp]),
    "fa_page_select": (_i, [_vp] * 8 + [_i] * 5 + [_ll] + [_i] * 6 + [_vp]),
    "fa_fwd_paged": (_i, [_vp] * 12 + [_i] * 5 + [ctypes.c_float, _ll] + [_i] * 4 + [_vp, ctypes.c_size_t, _vp]),
    "fa_fwd_paged_workspace_bytes": (ctypes.c_size_t, [_i] * 5),
    "fa_kv_plan_positions": (_i, [_vp] * 10 + [_i] * 6 + [_vp]),
    "fa_kv_append_rope": (_i, [_vp] * 13 + [_i] * 6 + [ctypes.c_float] + [_ll] * 4 + [_i] * 2 + [_vp]),
    "fa_fwd_paged_chunk": (_i, [_vp] * 10 + [_i] * 5 + [ctypes.c_float, _ll] + [_i] * 3 + [_vp, ctypes.c_size_t, _vp]),
    "fa_fwd_paged_chunk_workspace_bytes": (ctypes.c_size_t, [_i] * 5),
    "fa_rope": (_i, [_vp] * 6 + [_i] * 6 + [_vp, _ll, _i, ctypes.c_float, _vp]),
    "fa_rope_bwd": (_i, [_vp] * 6 + [_i] * 6 + [_vp, _ll, _i, ctypes.c_float, _vp]),
    "fa_rope_phases": (_i, [_vp, _vp, _i, _d, _i, _d, _d, _d, _d, _vp]),
    "fa_strerror": (ctypes.c_char_p, [_i]),
    "fa_device_status": (_i, [_vp]),
    "fa_selftest_bounded_wait": (_i, [_i, _vp]),
    "fa_selftest_fwd_timeout": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, ctypes.c_float,
                                     _i, ctypes.c_ulonglong, _vp]),
    "fa_selftest_bwd_timeout": (_i, [_vp] * 10 + [_i, _i, _i, _i, _i, ctypes.c_float, _i, ctypes.c_ulonglong,
                                                  _vp]),
    "fa_selftest_splitkv_timeout": (_i, [_vp] * 5 + [_i] * 5 + [ctypes.c_float, _i, _vp, ctypes.c_size_t,
                                                               ctypes.c_ulonglong, _vp]),
    "fa_selftest_paged_chunk_timeout": (_i, [_vp] * 10 + [_i] * 5 + [ctypes.c_float, _ll] + [_i] * 3 +
                                        [_vp, ctypes.c_size_t, ctypes.c_ulonglong, _vp]),
    "fa_version": (_i, []),
}


class FAError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = status
        msg = fa_strerror(status)
        super().__init__(f"{where}: {msg} (status {status})" if where else msg)


def library_path() -> str:
    return _build.LIB_PATH


def lib():
    """The loaded shared library (built in-tree with nvcc on first use)."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build()
            handle = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(handle, name)
                fn.restype = res
                fn.argtypes = args
            _lib = handle
        return _lib


def fa_strerror(status: int) -> str:
    return lib().fa_strerror(int(status)).decode()


def fa_version() -> int:
    return lib().fa_version()


def _stream_ptr(stream) -> int:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def fa_fwd_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, H: int,
               Sq: int, Sk: int, D: int, scale: float, causal: int, stream_ptr: int) -> int:
    """The C call with raw device pointers; returns the status code."""
    return lib().fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Sq, Sk, D, float(scale),
                        int(causal), stream_ptr)


def fa_fwd_window_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int,
                      H: int, Sq: int, Sk: int, D: int, scale: float, window_left: int,
                      window_right: int, stream_ptr: int) -> int:
    """The windowed C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_window(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Sq, Sk, D, float(scale),
                               int(window_left), int(window_right), stream_ptr)


def fa_fwd_blockmask_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int,
                         H: int, Sq: int, Sk: int, D: int, scale: float, window_left: int,
                         window_right: int, mask_ptr: int, mask_heads: int, pair_stride: int,
                         stream_ptr: int) -> int:
    """The block-mask C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_blockmask(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Sq, Sk, D, float(scale),
                                  int(window_left), int(window_right), mask_ptr, int(mask_heads),
                                  int(pair_stride), stream_ptr)


def _prepare(q, k, v, o, lse):
    import torch

    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    if o is None:
        o = torch.empty((B, H, Sq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16),
                        ("v", v, torch.bfloat16), ("o", o, torch.bfloat16),
                        ("lse", lse, torch.float32)):
        if t.dtype != dt or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA {dt} tensor")
    if tuple(k.shape) != (B, H, Sk, D) or tuple(v.shape) != (B, H, Sk, D):
        raise ValueError("k and v must be [B, H, Sk, D] matching q")
    if tuple(o.shape) != (B, H, Sq, D) or tuple(lse.shape) != (B, H, Sq):
        raise ValueError("o must be [B, H, Sq, D] and lse [B, H, Sq]")
    return o, lse, B, H, Sq, Sk, D


def fa_fwd(q, k, v, o=None, lse=None, scale: float | None = None, causal: bool = False,
           stream=None):
    """Attention forward on torch CUDA tensors.

    q: bf16 [B,H,Sq,D]; k, v: bf16 [B,H,Sk,D] (contiguous, same device).
    o (bf16 [B,H,Sq,D]) and lse (fp32 [B,H,Sq]) are allocated if not given.
    scale defaults to 1/sqrt(D).  Launches on ``stream`` (default: torch's
    current stream) and returns (o, lse) without synchronising.
    """
    o, lse, B, H, Sq, Sk, D = _prepare(q, k, v, o, lse)
    if scale is None:
        scale = D ** -0.5
    st = fa_fwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                    B, H, Sq, Sk, D, scale, int(bool(causal)), _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd")
    return o, lse


def fa_fwd_window(q, k, v, window_left: int, window_right: int, o=None, lse=None,
                  scale: float | None = None, stream=None):
    """Banded attention: key j allowed for query i iff i-window_left <= j <= i+window_right
    (-1 = unbounded on that side).  Same tensors and return value as fa_fwd."""
    o, lse, B, H, Sq, Sk, D = _prepare(q, k, v, o, lse)
    if scale is None:
        scale = D ** -0.5
    st = fa_fwd_window_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                           lse.data_ptr(), B, H, Sq, Sk, D, scale, window_left, window_right,
                           _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_window")
    return o, lse


def fa_fwd_blockmask(q, k, v, block_mask, window_left: int = -1, window_right: int = -1, o=None,
                     lse=None, scale: float | None = None, pair_stride: int = 1, stream=None):
    """Attention over the key blocks ``block_mask`` keeps (uint8 or bool CUDA tensor
    ``[mask_heads, ceil(Sq/128), ceil(Sk/128)]``, ``mask_heads`` 1 or B*H; nonzero
    keeps a 128-row x 128-key block), within the band of fa_fwd_window.  Rows with
    no allowed key get O = 0, LSE = -inf.  ``pair_stride``: query blocks a and
    a + pair_stride are computed together (a hint; the stride of a dilated
    pattern suits it).  Same tensors and return value as fa_fwd."""
    import torch

    o, lse, B, H, Sq, Sk, D = _prepare(q, k, v, o, lse)
    if scale is None:
        scale = D ** -0.5
    n_qb, n_kb = -(-Sq // FA_BLOCK_M), -(-Sk // FA_BLOCK_N)
    if (block_mask.dtype not in (torch.uint8, torch.bool) or not block_mask.is_cuda
            or not block_mask.is_contiguous() or block_mask.dim() != 3
            or tuple(block_mask.shape[1:]) != (n_qb, n_kb)):
        raise ValueError(f"block_mask must be a contiguous CUDA uint8/bool tensor [mask_heads, {n_qb}, {n_kb}]")
    st = fa_fwd_blockmask_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                              B, H, Sq, Sk, D, scale, window_left, window_right,
                              block_mask.data_ptr(), block_mask.shape[0], pair_stride, _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_blockmask")
    return o, lse


def fa_fwd_splitkv_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int,
                       H: int, Sq: int, Sk: int, D: int, scale: float, num_splits: int,
                       ws_ptr: int, ws_bytes: int, stream_ptr: int) -> int:
    """The split-KV C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_splitkv(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Sq, Sk, D, float(scale),
                                int(num_splits), ws_ptr, int(ws_bytes), stream_ptr)


def fa_fwd_splitkv_workspace_bytes(B: int, H: int, Sq: int, Sk: int, D: int,
                                   num_splits: int = 0) -> int:
    return lib().fa_fwd_splitkv_workspace_bytes(B, H, Sq, Sk, D, num_splits)


def fa_splitkv_num_splits(B: int, H: int, Sq: int, Sk: int, D: int) -> int:
    return lib().fa_splitkv_num_splits(B, H, Sq, Sk, D)


def fa_fwd_splitkv(q, k, v, o=None, lse=None, scale: float | None = None, num_splits: int = 0,
                   workspace=None, stream=None):
    """Decode attention (1..8 query rows per head, every key visible) with the keys
    of each head split across CTAs.  ``workspace`` is a CUDA uint8 tensor of at
    least fa_fwd_splitkv_workspace_bytes(...) bytes (allocated here if None)."""
    import torch

    o, lse, B, H, Sq, Sk, D = _prepare(q, k, v, o, lse)
    if scale is None:
        scale = D ** -0.5
    need = fa_fwd_splitkv_workspace_bytes(B, H, Sq, Sk, D, num_splits)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    st = fa_fwd_splitkv_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                            lse.data_ptr(), B, H, Sq, Sk, D, scale, num_splits,
                            workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                            _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_splitkv")
    return o, lse


def fa_fwd_fp8_raw(q_ptr: int, k_ptr: int, v_ptr: int, o_ptr: int, lse_ptr: int, B: int, H: int,
                   Sq: int, Sk: int, D: int, scale: float, causal: int, descale_q: float,
                   descale_k: float, descale_v: float, stream_ptr: int) -> int:
    """The 8-bit C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_fp8(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Sq, Sk, D, float(scale),
                            int(causal), float(descale_q), float(descale_k), float(descale_v),
                            stream_ptr)


def fa_fwd_fp8(q, k, v, descale_q: float, descale_k: float, descale_v: float, o=None, lse=None,
               scale: float | None = None, causal: bool = False, stream=None):
    """Attention forward on e4m3 inputs with per-tensor scales (real value = code * descale).

    q: [B,H,Sq,128], k, v: [B,H,Sk,128], each a contiguous CUDA tensor of dtype uint8
    (the codes) or torch.float8_e4m3fn.  o (bf16 [B,H,Sq,128]) and lse (fp32 [B,H,Sq])
    are allocated if not given.  Returns (o, lse) without synchronising."""
    import torch

    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dtype not in (torch.uint8, torch.float8_e4m3fn) or not t.is_cuda or \
                not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA uint8 / float8_e4m3fn tensor")
    if tuple(k.shape) != (B, H, Sk, D) or tuple(v.shape) != (B, H, Sk, D):
        raise ValueError("k and v must be [B, H, Sk, D] matching q")
    if o is None:
        o = torch.empty((B, H, Sq, D), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    if o.dtype != torch.bfloat16 or tuple(o.shape) != (B, H, Sq, D) or not o.is_contiguous() \
            or lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, Sq) or \
            not lse.is_contiguous() or not o.is_cuda or not lse.is_cuda:
        raise ValueError("o must be contiguous CUDA bf16 [B,H,Sq,D] and lse fp32 [B,H,Sq]")
    if scale is None:
        scale = D ** -0.5
    st = fa_fwd_fp8_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                        B, H, Sq, Sk, D, scale, int(bool(causal)), descale_q, descale_k,
                        descale_v, _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_fwd_fp8")
    return o, lse


def fa_bwd_raw(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, do_ptr, dq_ptr, dk_ptr, dv_ptr, delta_ptr,
               B, H, Sq, Sk, D, scale, causal, stream_ptr) -> int:
    """The backward C call with raw device pointers; returns the status code."""
    return lib().fa_bwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, do_ptr, dq_ptr, dk_ptr, dv_ptr,
                        delta_ptr, B, H, Sq, Sk, D, float(scale), int(causal), stream_ptr)


def fa_bwd(q, k, v, o, lse, dout, dq=None, dk=None, dv=None, delta=None,
           scale: float | None = None, causal: bool = False, stream=None):
    """Gradients (dq, dk, dv) of fa_fwd for output gradient ``dout`` (torch CUDA tensors;
    o and lse are fa_fwd's outputs).  Outputs and the fp32 ``delta`` scratch [B,H,Sq] are
    allocated if not given.  Returns (dq, dk, dv) without synchronising."""
    import torch

    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if delta is None:
        delta = torch.empty((B, H, Sq), dtype=torch.float32, device=q.device)
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout), ("dq", dq),
                    ("dk", dk), ("dv", dv)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA bfloat16 tensor")
    for name, t in (("lse", lse), ("delta", delta)):
        if t.dtype != torch.float32 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous CUDA float32 tensor")
    if scale is None:
        scale = D ** -0.5
    st = fa_bwd_raw(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                    dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                    delta.data_ptr(), B, H, Sq, Sk, D, scale, int(bool(causal)),
                    _stream_ptr(stream))
    if st != FA_OK:
        raise FAError(st, "fa_bwd")
    return dq, dk, dv


# ------------------------------------------------------ the paged 8-bit cache
def fa_kv_plan_raw(cached_ptr, new_ptr, free_ptr, count_ptr, table_ptr, cu_q_ptr, lens_ptr, slots_ptr, left_ptr, B, T,
                   max_pages, num_free, num_pages, page_size, stream_ptr) -> int:
    """The plan C call with raw device pointers; returns the status code."""
    return lib().fa_kv_plan(cached_ptr, new_ptr, free_ptr, count_ptr, table_ptr, cu_q_ptr, lens_ptr, slots_ptr, left_ptr,
                            B, T, max_pages, num_free, num_pages, page_size, stream_ptr)


def fa_kv_append_raw(k_ptr, v_ptr, slots_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr, k_mean_ptr,
                     k_mean_scale_ptr, T, Hkv, D, k_stride, v_stride, num_pages, page_size, stream_ptr) -> int:
    """The append C call with raw device pointers; returns the status code."""
    return lib().fa_kv_append(k_ptr, v_ptr, slots_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr, k_mean_ptr,
                              k_mean_scale_ptr, T, Hkv, D, k_stride, v_stride, num_pages, page_size, stream_ptr)


def fa_page_select_raw(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_mean_ptr, k_mean_scale_ptr, sel_ptr, count_ptr, B, T, Hq,
                       Hkv, D, q_stride, max_pages, num_pages, page_size, top_k, keep_first, keep_last,
                       stream_ptr) -> int:
    """The page selection C call with raw device pointers; returns the status code."""
    return lib().fa_page_select(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_mean_ptr, k_mean_scale_ptr, sel_ptr, count_ptr, B,
                                T, Hq, Hkv, D, q_stride, max_pages, num_pages, page_size, top_k, keep_first, keep_last,
                                stream_ptr)


def fa_fwd_paged_raw(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr, sel_ptr,
                     count_ptr, o_ptr, lse_ptr, B, T, Hq, Hkv, D, scale, q_stride, max_pages, num_pages, page_size,
                     sel_width, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The paged attention C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_paged(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr,
                              sel_ptr, count_ptr, o_ptr, lse_ptr, B, T, Hq, Hkv, D, scale, q_stride, max_pages, num_pages,
                              page_size, sel_width, ws_ptr, ws_bytes, stream_ptr)


def fa_fwd_paged_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace that fa_fwd_paged needs for these sizes on the current device."""
    return lib().fa_fwd_paged_workspace_bytes(B, T, Hq, Hkv, D)


def fa_kv_plan_positions_raw(cached_ptr, new_ptr, free_ptr, count_ptr, table_ptr, cu_q_ptr, lens_ptr, slots_ptr, positions_ptr,
                             left_ptr, B, T, max_pages, num_free, num_pages, page_size, stream_ptr) -> int:
    """The plan C call that writes positions too, with raw device pointers; returns the status code."""
    return lib().fa_kv_plan_positions(cached_ptr, new_ptr, free_ptr, count_ptr, table_ptr, cu_q_ptr, lens_ptr, slots_ptr,
                                      positions_ptr, left_ptr, B, T, max_pages, num_free, num_pages, page_size, stream_ptr)


def fa_kv_append_rope_raw(k_ptr, v_ptr, positions_ptr, phases_ptr, slots_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr,
                          k_mean_ptr, k_mean_scale_ptr, q_ptr, q_out_ptr, T, Hkv, Hq, D, rot_dim, interleaved, amplitude, k_stride,
                          v_stride, q_stride, q_out_stride, num_pages, page_size, stream_ptr) -> int:
    """The rotating append C call with raw device pointers; returns the status code."""
    return lib().fa_kv_append_rope(k_ptr, v_ptr, positions_ptr, phases_ptr, slots_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr,
                                   v_scale_ptr, k_mean_ptr, k_mean_scale_ptr, q_ptr, q_out_ptr, T, Hkv, Hq, D, rot_dim,
                                   int(interleaved), float(amplitude), k_stride, v_stride, q_stride, q_out_stride, num_pages,
                                   page_size, stream_ptr)


def fa_fwd_paged_chunk_raw(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr, o_ptr, lse_ptr,
                           B, T, Hq, Hkv, D, scale, q_stride, max_pages, num_pages, page_size, ws_ptr, ws_bytes, stream_ptr) -> int:
    """The paged attention of chunks C call with raw device pointers; returns the status code."""
    return lib().fa_fwd_paged_chunk(q_ptr, cu_q_ptr, lens_ptr, table_ptr, k_pages_ptr, v_pages_ptr, k_scale_ptr, v_scale_ptr, o_ptr,
                                    lse_ptr, B, T, Hq, Hkv, D, scale, q_stride, max_pages, num_pages, page_size, ws_ptr, ws_bytes,
                                    stream_ptr)


def fa_fwd_paged_chunk_workspace_bytes(B: int, T: int, Hq: int, Hkv: int, D: int) -> int:
    """Bytes of workspace that fa_fwd_paged_chunk needs for these sizes on the current device."""
    return lib().fa_fwd_paged_chunk_workspace_bytes(B, T, Hq, Hkv, D)


_binding_module = None


def _binding():
    """The extension module that makes the paged cache's calls on tensors."""
    global _binding_module
    if _binding_module is None:
        import importlib.machinery
        import importlib.util

        import torch  # noqa: F401  (its libraries, which the module links, are loaded)

        lib()
        with _lock:
            if _binding_module is None:
                _build.build_binding()
                loader = importlib.machinery.ExtensionFileLoader("fa_binding", _build.BINDING_PATH)
                module = importlib.util.module_from_spec(importlib.util.spec_from_loader("fa_binding", loader))
                loader.exec_module(module)
                _binding_module = module
    return _binding_module


def _stream_of(stream, device):
    """A stream argument as the extension takes it: None (torch's current one) or an address."""
    if stream is None or isinstance(stream, int):
        return stream
    if stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {device}")
    return stream.cuda_stream


def _allocating(device, stream):
    """A context in which new tensors belong to the stream that the call is launched on."""
    import contextlib

    import torch

    if device.type != "cuda":
        raise ValueError("the tensors must be CUDA tensors")
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


def fa_kv_plan(cached_lens, new_lens, free_pages, free_count, block_table, num_pages: int, page_size: int, cu_q=None,
               seq_lens=None, slot_map=None, free_left=None, num_tokens: int | None = None, stream=None, positions=None):
    """Block tables and slot maps from request lengths, first come, first served.

    cached_lens, new_lens: int32 [B]; free_pages: int32 [num_free], of which the first free_count
    (int32 [1]) are free and are taken from the end; block_table: int32 [B, max_pages], to which the
    new pages are added.  slot_map (int32 [T]) or num_tokens says how many tokens there are room for.
    Returns (cu_q [B+1], seq_lens [B], slot_map [T], free_left [1]), all int32, without synchronising;
    a request that is not served gets seq_lens 0 and slots of -1.  positions (int32 [T], if given) is
    written too: each token's position in its sequence, for fa_rope and fa_kv_append_rope, -1 behind the
    last token."""
    if cu_q is None or seq_lens is None or slot_map is None or free_left is None:
        import torch

        dev, B = cached_lens.device, cached_lens.shape[0]
        if slot_map is None and num_tokens is None:
            raise ValueError("give slot_map or num_tokens")
        with _allocating(dev, stream):
            cu_q = torch.empty(B + 1, dtype=torch.int32, device=dev) if cu_q is None else cu_q
            seq_lens = torch.empty(B, dtype=torch.int32, device=dev) if seq_lens is None else seq_lens
            slot_map = torch.empty(num_tokens, dtype=torch.int32, device=dev) if slot_map is None else slot_map
            free_left = torch.empty(1, dtype=torch.int32, device=dev) if free_left is None else free_left
    rc = _binding().kv_plan(cached_lens, new_lens, free_pages, free_count, block_table, num_pages, page_size, cu_q, seq_lens,
                            slot_map, free_left, positions, stream if stream is None else _stream_of(stream, cached_lens.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv_plan")
    return cu_q, seq_lens, slot_map, free_left


def fa_kv_append(k, v, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean=None, k_mean_scale=None, stream=None):
    """Rounds a step's keys and values into the paged 8-bit cache, in place.

    k, v: bf16 [T, Hkv, D], strided over tokens or contiguous; slot_map: int32 [T] (negative: skipped);
    k_pages, v_pages: uint8 or float8_e4m3fn [num_pages, Hkv, page_size, D]; k_scale, v_scale: fp32
    [num_pages, Hkv]; k_mean (int8 [num_pages, Hkv, D]) and k_mean_scale (fp32 [num_pages, Hkv]), both or
    neither, are the pages' mean keys for fa_page_select.  Does not synchronise."""
    rc = _binding().kv_append(k, v, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean, k_mean_scale,
                              stream if stream is None else _stream_of(stream, k.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv_append")


def fa_kv_append_rope(k, v, positions, phases, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean=None, k_mean_scale=None, q=None,
                      q_out=None, interleaved: bool = False, amplitude: float = 1.0, stream=None):
    """fa_kv_append with the keys rotated on the way (in fp32, rounded once, to codes), and, where q is
    given, the step's queries rotated beside.

    positions: int32 [T] (fa_kv_plan's); phases, interleaved, amplitude: as in fa_rope; q: bf16 [T, Hq, D],
    strided over tokens or contiguous; q_out: the same shape (allocated if not given; may be q itself).
    Other arguments are fa_kv_append's.  Returns q_out (None without q); does not synchronise."""
    if q is not None and q_out is None:
        import torch

        with _allocating(q.device, stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device)
    rc = _binding().kv_append_rope(k, v, positions, phases, slot_map, k_pages, v_pages, k_scale, v_scale, k_mean, k_mean_scale, q, q_out,
                                   interleaved, amplitude, stream if stream is None else _stream_of(stream, k.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_kv_append_rope")
    return q_out


def fa_page_select(q, cu_q, seq_lens, block_table, k_mean, k_mean_scale, page_size: int, top_k: int, keep_first: int = 1,
                   keep_last: int = 1, sel=None, sel_count=None, stream=None):
    """The top_k pages of each sequence and key/value head by the 8-bit score of its queries against
    the pages' mean keys; the first keep_first and the last keep_last pages are always among them.

    q: bf16 [T, Hq, D], strided over tokens or contiguous; cu_q: int32 [B+1]; seq_lens: int32 [B];
    block_table: int32 [B, max_pages]; k_mean, k_mean_scale: fa_kv_append's.  Returns (sel, sel_count):
    int32 [B, Hkv, top_k] of positions in the block table, ascending, -1 behind the last, and int32
    [B, Hkv].  Does not synchronise."""
    if sel is None or sel_count is None:
        import torch

        shape = (seq_lens.shape[0], k_mean.shape[1])
        with _allocating(q.device, stream):
            sel = torch.empty((*shape, top_k), dtype=torch.int32, device=q.device) if sel is None else sel
            sel_count = torch.empty(shape, dtype=torch.int32, device=q.device) if sel_count is None else sel_count
    rc = _binding().page_select(q, cu_q, seq_lens, block_table, k_mean, k_mean_scale, page_size, top_k, keep_first, keep_last, sel,
                                sel_count, stream if stream is None else _stream_of(stream, q.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_page_select")
    return sel, sel_count


def fa_fwd_paged(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, sel=None, sel_count=None, o=None,
                 lse=None, scale: float | None = None, workspace=None, stream=None):
    """Attention of a step's query tokens (the last ones of their sequences, causal) over the paged
    8-bit cache, or over the pages that fa_page_select chose.

    q: bf16 [T, Hq, D], strided over tokens or contiguous; cu_q: int32 [B+1]; seq_lens: int32 [B], this
    step's tokens included; block_table: int32 [B, max_pages]; the cache as in fa_kv_append; sel,
    sel_count: both or neither.  o (bf16 [T, Hq, D]), lse (fp32 [T, Hq]) and workspace (a CUDA uint8
    tensor of at least fa_fwd_paged_workspace_bytes(...) bytes) are allocated if not given; rows from
    cu_q[B] on are not written.  Returns (o, lse) without synchronising."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if o is None or lse is None or workspace is None:
        import torch

        dev = q.device
        with _allocating(dev, stream):
            o = torch.empty(q.shape, dtype=torch.bfloat16, device=dev) if o is None else o
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if lse is None else lse
            if workspace is None:
                with torch.cuda.device(dev):
                    need = fa_fwd_paged_workspace_bytes(seq_lens.shape[0], q.shape[0], q.shape[1], k_pages.shape[1], q.shape[-1])
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = _binding().fwd_paged(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, sel, sel_count, o, lse, scale,
                              workspace, stream if stream is None else _stream_of(stream, q.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_paged")
    return o, lse


def fa_fwd_paged_chunk(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o=None, lse=None, scale: float | None = None,
                       workspace=None, stream=None):
    """fa_fwd_paged (over all pages) made for many query tokens a sequence: prompts, or chunks of them behind
    what is cached, beside sequences with a single token.

    Arguments and results are fa_fwd_paged's, but workspace has at least fa_fwd_paged_chunk_workspace_bytes(...)
    bytes.  Returns (o, lse) without synchronising."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if o is None or lse is None or workspace is None:
        import torch

        dev = q.device
        with _allocating(dev, stream):
            o = torch.empty(q.shape, dtype=torch.bfloat16, device=dev) if o is None else o
            lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if lse is None else lse
            if workspace is None:
                with torch.cuda.device(dev):
                    need = fa_fwd_paged_chunk_workspace_bytes(seq_lens.shape[0], q.shape[0], q.shape[1], k_pages.shape[1], q.shape[-1])
                workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    rc = _binding().fwd_paged_chunk(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o, lse, scale, workspace,
                                    stream if stream is None else _stream_of(stream, q.device))
    if rc != FA_OK:
        raise FAError(rc, "fa_fwd_paged_chunk")
    return o, lse


# ------------------------------------------------------------ rotary positions
def fa_rope_raw(q_ptr, k_ptr, q_out_ptr, k_out_ptr, positions_ptr, phases_ptr, B, S, Hq, Hk, D, rot_dim, strides, positions_stride,
                interleaved, amplitude, stream_ptr) -> int:
    """The rotation C call with raw device pointers and 12 strides (a sequence of integers, or None); returns the status code."""
    array = None if strides is None else (_ll * 12)(*strides)
    return lib().fa_rope(q_ptr, k_ptr, q_out_ptr, k_out_ptr, positions_ptr, phases_ptr, B, S, Hq, Hk, D, rot_dim, array,
                         positions_stride, int(interleaved), float(amplitude), stream_ptr)


def fa_rope_bwd_raw(dq_out_ptr, dk_out_ptr, dq_ptr, dk_ptr, positions_ptr, phases_ptr, B, S, Hq, Hk, D, rot_dim, strides,
                    positions_stride, interleaved, amplitude, stream_ptr) -> int:
    """The rotation's gradient C call with raw device pointers and 12 strides; returns the status code."""
    array = None if strides is None else (_ll * 12)(*strides)
    return lib().fa_rope_bwd(dq_out_ptr, dk_out_ptr, dq_ptr, dk_ptr, positions_ptr, phases_ptr, B, S, Hq, Hk, D, rot_dim, array,
                             positions_stride, int(interleaved), float(amplitude), stream_ptr)


def fa_rope_phases(rot_dim: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0, span: float = 0.0,
                   fast: float = 32.0, slow: float = 1.0, frequencies=None, device="cuda"):
    """The frequencies of rotary positions as fa_rope takes them: (phases, amplitude), phases an int64 tensor
    [rot_dim / 2] on ``device`` in units of 2^-64 turns a position, amplitude a float.

    Pair i turns by base^(-2 i / rot_dim) radians a position, or by frequencies[i]; scaling "linear" divides
    by factor, "ntk" stretches the base by factor, "yarn" divides the pairs that make fewer than ``slow``
    turns in ``span`` positions by factor, keeps those with more than ``fast`` and mixes between (the
    amplitude is then 0.1 ln(factor) + 1).  Computed on the host; meant to be called once."""
    import torch

    if scaling not in FA_ROPE_SCALINGS:
        raise ValueError(f"scaling must be one of {tuple(FA_ROPE_SCALINGS)}")
    if frequencies is not None:
        frequencies = [float(f) for f in frequencies]
        if len(frequencies) != rot_dim // 2:
            raise ValueError("frequencies must have rot_dim / 2 elements")
    phases = (ctypes.c_ulonglong * max(1, rot_dim // 2))()
    amplitude = ctypes.c_float()
    st = lib().fa_rope_phases(phases, ctypes.byref(amplitude), rot_dim, base, FA_ROPE_SCALINGS[scaling], factor, span, fast, slow,
                              None if frequencies is None else (_d * len(frequencies))(*frequencies))
    if st != FA_OK:
        raise FAError(st, "fa_rope_phases")
    signed = [x - (1 << 64) if x >= 1 << 63 else x for x in phases]
    return torch.tensor(signed, dtype=torch.int64, device=device), amplitude.value


def _rope(name, inverse, q, k, phases, positions, interleaved, amplitude, q_out, k_out, stream):
    if q_out is None or (k is not None and k_out is None):
        import torch

        with _allocating(q.device, stream):
            q_out = torch.empty(q.shape, dtype=torch.bfloat16, device=q.device) if q_out is None else q_out
            k_out = torch.empty(k.shape, dtype=torch.bfloat16, device=q.device) if k is not None and k_out is None else k_out
    rc = _binding().rope(q, k, phases, positions, interleaved, amplitude, q_out, k_out, inverse,
                         stream if stream is None else _stream_of(stream, q.device))
    if rc != FA_OK:
        raise FAError(rc, name)
    return q_out, k_out


def fa_rope(q, k, phases, positions=None, interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_out=None, stream=None):
    """Rotary positions of queries and keys.

    q: bf16 [B, Hq, S, D] or [T, Hq, D], k: the same with Hk heads, or None; any strides but a contiguous
    last dimension (views of a fused projection); positions: int32 [S] or [B, S] ([T] for packed tokens),
    or None: 0, 1, ..; phases, amplitude: fa_rope_phases'.  The first 2 * len(phases) elements of each head
    are rotated, in pairs i and i + len(phases), or, ``interleaved``, 2 i and 2 i + 1; the others are copied.
    q_out and k_out (allocated contiguous if not given) may be q and k, or views of a fused tensor.
    Returns (q_out, k_out) without synchronising."""
    return _rope("fa_rope", False, q, k, phases, positions, interleaved, amplitude, q_out, k_out, stream)


def fa_rope_bwd(dq_out, dk_out, phases, positions=None, interleaved: bool = False, amplitude: float = 1.0, q_out=None, k_out=None,
                stream=None):
    """Gradients (dq, dk) of fa_rope for the gradients of its outputs, written to q_out and k_out (allocated if
    not given); other arguments as for fa_rope."""
    return _rope("fa_rope_bwd", True, dq_out, dk_out, phases, positions, interleaved, amplitude, q_out, k_out, stream)


def fa_device_status(stream=None) -> int:
    """Synchronise the stream, return and clear the kernels' status word."""
    return lib().fa_device_status(_stream_ptr(stream))


def fa_selftest_bounded_wait(timeout_us: int, stream=None) -> int:
    return lib().fa_selftest_bounded_wait(int(timeout_us), _stream_ptr(stream))


def fa_selftest_fwd_timeout(q, k, v, o, lse, scale, causal, timeout_ns: int, stream=None) -> int:
    """fa_fwd with every on-chip wait bounded by `timeout_ns` (tests of the give-up
    path); returns the launch status.  q, k, v, o, lse: contiguous CUDA tensors."""
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    return lib().fa_selftest_fwd_timeout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                         lse.data_ptr(), B, H, Sq, Sk, D, float(scale),
                                         int(bool(causal)), int(timeout_ns), _stream_ptr(stream))


def fa_selftest_bwd_timeout(q, k, v, o, lse, dout, dq, dk, dv, delta, scale, causal, timeout_ns: int,
                            stream=None) -> int:
    """fa_bwd with every on-chip wait of both kernels bounded by `timeout_ns`
    (tests of the give-up path); returns the launch status.  All arguments are
    contiguous CUDA tensors as for fa_bwd."""
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    return lib().fa_selftest_bwd_timeout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                         lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                         dv.data_ptr(), delta.data_ptr(), B, H, Sq, Sk, D, float(scale),
                                         int(bool(causal)), int(timeout_ns), _stream_ptr(stream))


def fa_selftest_splitkv_timeout(q, k, v, o, lse, workspace, scale, timeout_ns: int, num_splits: int = 0,
                                stream=None) -> int:
    """fa_fwd_splitkv with every on-chip wait of the partial kernel bounded by
    `timeout_ns` (tests of the give-up path); returns the launch status.  All
    arguments are contiguous CUDA tensors as for fa_fwd_splitkv; ``workspace`` is a
    byte tensor of at least fa_fwd_splitkv_workspace_bytes."""
    B, H, Sq, D = q.shape
    Sk = k.shape[2]
    return lib().fa_selftest_splitkv_timeout(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                             lse.data_ptr(), B, H, Sq, Sk, D, float(scale), int(num_splits),
                                             workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                             int(timeout_ns), _stream_ptr(stream))


def fa_selftest_paged_chunk_timeout(q, cu_q, seq_lens, block_table, k_pages, v_pages, k_scale, v_scale, o, lse, workspace, scale,
                                    timeout_ns: int, stream=None) -> int:
    """fa_fwd_paged_chunk with every on-chip wait bounded by `timeout_ns` (tests of the give-up path); returns
    the launch status.  All arguments are tensors as for fa_fwd_paged_chunk, none of them optional."""
    T, Hq, D = q.shape
    num_pages, Hkv, page, _ = k_pages.shape
    return lib().fa_selftest_paged_chunk_timeout(q.data_ptr(), cu_q.data_ptr(), seq_lens.data_ptr(), block_table.data_ptr(),
                                                 k_pages.data_ptr(), v_pages.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                                 o.data_ptr(), lse.data_ptr(), seq_lens.shape[0], T, Hq, Hkv, D, float(scale),
                                                 q.stride(0) if T > 1 else Hq * D, block_table.shape[1], num_pages, page,
                                                 workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                                 int(timeout_ns), _stream_ptr(stream))
