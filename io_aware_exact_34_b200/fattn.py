"""Python binding of libfattn: argument marshalling over the C ABI only.

Every function here takes torch tensors, checks their dtype / device / layout,
passes raw pointers, sizes and the current CUDA stream to the library of the
same name, and raises ``FattnError`` on a non-zero status.  All arithmetic runs
in the library's CUDA kernels; there is no fallback of any kind.  If the
shared library is missing, importing this module fails.
"""
from __future__ import annotations

import ctypes
import importlib.util
import operator
import os
import warnings

import torch

from . import calls_path

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libfattn.so")
if not os.path.exists(_LIB_PATH):
    raise ImportError(f"libfattn.so is not built ({_LIB_PATH}); run "
                      "`python -m io_aware_exact_34_b200.build`")
lib = ctypes.CDLL(_LIB_PATH)

_vp, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_ll = ctypes.c_longlong
_llp = ctypes.POINTER(ctypes.c_longlong)
lib.attn_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp]
lib.attn_fwd.restype = _i
lib.attn_fwd_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp, ctypes.c_size_t, _vp]
lib.attn_fwd_host.restype = _i
lib.attn_fwd_host_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.attn_fwd_host_workspace_bytes.restype = ctypes.c_size_t
lib.attn_fwd_counted.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _vp]
lib.attn_fwd_counted.restype = _i
lib.attn_fwd_varlen.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp]
lib.attn_fwd_varlen.restype = _i
lib.attn_fwd_varlen_counted.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f, _i, _i, _i,
                                        _vp, _vp]
lib.attn_fwd_varlen_counted.restype = _i
lib.attn_fwd_f32.argtypes = [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp]
lib.attn_fwd_f32.restype = _i
lib.attn_decode_splitkv.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp, _sz, _vp]
lib.attn_decode_splitkv.restype = _i
lib.attn_decode_splitkv_noalloc.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _vp]
lib.attn_decode_splitkv_noalloc.restype = _i
lib.attn_decode_paged.argtypes = [_vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _i, _i, _i, _f, _i, _vp, _sz, _vp]
lib.attn_decode_paged.restype = _i
lib.attn_paged_plan.argtypes = [_vp, _vp, _i, _vp, _i, _vp, _i, _i, _vp, _i, _vp, _vp, _vp, _vp]
lib.attn_paged_plan.restype = _i
lib.attn_append_paged_fp8.argtypes = [_vp, _vp, _ll, _ll, _vp, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _vp]
lib.attn_append_paged_fp8.restype = _i
lib.attn_decode_paged_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _i, _i, _i, _i, _f, _i, _i,
                                      _vp, _sz, _vp]
lib.attn_decode_paged_fp8.restype = _i
lib.attn_decode_paged_fp8_auto_splits.argtypes = [_i, _i, _i, _i, _i]
lib.attn_decode_paged_fp8_auto_splits.restype = _i
lib.attn_fwd_paged_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _i, _f,
                                   _i, _i, _i, _vp, _sz, _vp]
lib.attn_fwd_paged_fp8.restype = _i
lib.attn_fwd_paged_fp8_workspace_bytes.argtypes = [_i, _i, _i, _i, _i, _i, _i]
lib.attn_fwd_paged_fp8_workspace_bytes.restype = _sz
lib.attn_decode_auto_splits.argtypes = [_i, _i, _i, _i]
lib.attn_decode_auto_splits.restype = _i
lib.attn_decode_workspace_bytes.argtypes = [_i, _i, _i, _i, _i]
lib.attn_decode_workspace_bytes.restype = _sz
lib.attn_count_blocks.argtypes = [_i, _i, _i, _i, _i, _i, _i, _llp, _llp, _llp, _llp]
lib.attn_count_blocks.restype = _i
lib.attn_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp, _sz, _vp]
lib.attn_bwd.restype = _i
lib.attn_bwd_counted.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp,
                                 _sz, _vp, _vp]
lib.attn_bwd_counted.restype = _i
lib.attn_bwd_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.attn_bwd_workspace_bytes.restype = _sz
lib.attn_bwd_count_blocks.argtypes = [_i, _i, _i, _i, _i, _i, _i, _llp]
lib.attn_bwd_count_blocks.restype = _i
lib.attn_fwd_fp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp]
lib.attn_fwd_fp8.restype = _i
lib.attn_fwd_fp8_counted.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _f, _i, _i, _i, _vp,
                                     _vp]
lib.attn_fwd_fp8_counted.restype = _i
lib.attn_fp8_ld.argtypes = [_i]
lib.attn_fp8_ld.restype = _i
lib.attn_quantize_fp8.argtypes = [_vp, _vp, _vp, _i, _i, _i, _i, _i, _vp]
lib.attn_quantize_fp8.restype = _i
lib.fattn_status_string.argtypes = [_i]
lib.fattn_status_string.restype = ctypes.c_char_p
lib.fattn_device_status.argtypes = [_vp]
lib.fattn_device_status.restype = _i
lib.fattn_debug_inject_stall.argtypes = [_i]
lib.fattn_debug_inject_stall.restype = _i

FATTN_OK = 0
FATTN_ERR_INVALID_ARG = -1
FATTN_ERR_UNSUPPORTED = -2
FATTN_ERR_MISALIGNED = -3
FATTN_ERR_WORKSPACE = -4
FATTN_ERR_CUDA = -5
FATTN_ERR_TIMEOUT = -6
FATTN_ERR_NO_DEVICE = -7


class FattnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {lib.fattn_status_string(status).decode()}")


def _check(status: int, where: str) -> None:
    if status != FATTN_OK:
        raise FattnError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _want(t, dtype, ndim, name, shape=None, device=None):
    """Every pointer the library receives comes from a tensor checked here:
    dtype, rank, contiguity, CUDA residency and, where given, the exact shape
    and the device of the first input (the kernels trust all of these)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.dim() != ndim or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} CUDA tensor with {ndim} dims, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _want_counter(counter, device):
    if counter is not None:
        if not isinstance(counter, torch.Tensor) or counter.dtype not in (torch.int64, torch.uint64) \
                or counter.numel() != 1 or not counter.is_cuda or counter.device != device:
            raise ValueError(f"counter: expected a one-element int64 tensor on {device}")


def _want_workspace(ws, device):
    if ws is not None:
        if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.device != device or not ws.is_contiguous():
            raise ValueError(f"workspace: expected a contiguous CUDA tensor on {device}")


def attn_fwd(q, k, v, o=None, lse=None, scale=None, causal=False, window_left=-1, window_right=-1,
             need_lse=True, counter=None):
    """bf16 prefill forward.  q: [B,H,Lq,d], k, v: [B,H,Lk,d] -> (o, lse).
    ``counter`` (optional, a zeroed one-element int64 CUDA tensor) receives the
    number of KV tiles visited."""
    _want(q, torch.bfloat16, 4, "q")
    B, H, Lq, d = q.shape
    dev = q.device
    _want(k, torch.bfloat16, 4, "k", device=dev)
    Lk = k.shape[2]
    _want(k, torch.bfloat16, 4, "k", shape=(B, H, Lk, d))  # same batch, heads and head dim as q
    _want(v, torch.bfloat16, 4, "v", shape=(B, H, Lk, d), device=dev)
    _want_counter(counter, dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.bfloat16, 4, "o", shape=(B, H, Lq, d), device=dev)
    if lse is None and need_lse:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev)
    if lse is not None:
        _want(lse, torch.float32, 3, "lse", shape=(B, H, Lq), device=dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, scale, int(bool(causal)),
            int(window_left), int(window_right))
    if counter is None:
        _check(lib.attn_fwd(*args, _stream()), "attn_fwd")
    else:
        _check(lib.attn_fwd_counted(*args, _ptr(counter), _stream()), "attn_fwd_counted")
    return o, lse


def attn_fwd_counted(q, k, v, counter, o=None, lse=None, scale=None, causal=False, window_left=-1,
                     window_right=-1):
    """attn_fwd that adds the number of KV tiles visited to ``counter``
    (a zeroed uint64/int64 CUDA tensor with one element)."""
    return attn_fwd(q, k, v, o, lse, scale, causal, window_left, window_right, counter=counter)


def attn_fwd_host_workspace_bytes(B, H, Lq, Lk, d) -> int:
    return lib.attn_fwd_host_workspace_bytes(B, H, Lq, Lk, d)


def _want_host(t, dtype, ndim, name, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype or t.dim() != ndim or t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} host tensor with {ndim} dims, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def attn_fwd_host(q, k, v, o=None, lse=None, scale=None, causal=False, window_left=-1, window_right=-1,
                  need_lse=True, workspace=None):
    """attn_fwd on host tensors (pin them for the copies to overlap the
    kernels): q [B,H,Lq,d], k, v [B,H,Lk,d] bf16 on the CPU -> (o, lse) on the
    CPU.  The device workspace is allocated here unless given (a uint8 CUDA
    tensor of attn_fwd_host_workspace_bytes).  Returns once the results are in
    o and lse (the current stream is synchronised)."""
    _want_host(q, torch.bfloat16, 4, "q")
    B, H, Lq, d = q.shape
    Lk = k.shape[2] if k.dim() == 4 else -1
    _want_host(k, torch.bfloat16, 4, "k", shape=(B, H, Lk, d))
    _want_host(v, torch.bfloat16, 4, "v", shape=(B, H, Lk, d))
    if o is None:
        o = torch.empty_like(q, pin_memory=True)
    _want_host(o, torch.bfloat16, 4, "o", shape=(B, H, Lq, d))
    if lse is None and need_lse:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, pin_memory=True)
    if lse is not None:
        _want_host(lse, torch.float32, 3, "lse", shape=(B, H, Lq))
    dev = torch.device("cuda", torch.cuda.current_device())
    need = attn_fwd_host_workspace_bytes(B, H, Lq, Lk, d)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _want_workspace(workspace, dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    _check(lib.attn_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, scale,
                             int(bool(causal)), int(window_left), int(window_right), _ptr(workspace),
                             workspace.numel() * workspace.element_size(), _stream()), "attn_fwd_host")
    torch.cuda.current_stream().synchronize()
    return o, lse


def attn_fwd_varlen(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, o=None, lse=None, scale=None,
                    causal=False, window_left=-1, window_right=-1, counter=None):
    """Packed variable-length prefill.  q: [total_q, H, d], k, v: [total_k, H, d]
    bf16; cu_seqlens_*: int32 [num_seqs + 1] on the device -> (o, lse [H, total_q])."""
    _want(q, torch.bfloat16, 3, "q")
    _want(k, torch.bfloat16, 3, "k")
    _want(v, torch.bfloat16, 3, "v")
    _want(cu_seqlens_q, torch.int32, 1, "cu_seqlens_q")
    _want(cu_seqlens_k, torch.int32, 1, "cu_seqlens_k")
    total_q, H, d = q.shape
    dev = q.device
    total_k = k.shape[0]
    nseq = cu_seqlens_q.numel() - 1
    _want(k, torch.bfloat16, 3, "k", shape=(total_k, H, d), device=dev)
    _want(v, torch.bfloat16, 3, "v", shape=(total_k, H, d), device=dev)
    _want(cu_seqlens_q, torch.int32, 1, "cu_seqlens_q", device=dev)
    _want(cu_seqlens_k, torch.int32, 1, "cu_seqlens_k", shape=(nseq + 1,), device=dev)
    _want_counter(counter, dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.bfloat16, 3, "o", shape=(total_q, H, d), device=dev)
    if lse is None:
        lse = torch.empty((H, total_q), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 2, "lse", shape=(H, total_q), device=dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), nseq, H, total_q,
            total_k, int(max_seqlen_q), d, scale, int(bool(causal)), int(window_left), int(window_right))
    if counter is None:
        _check(lib.attn_fwd_varlen(*args, _stream()), "attn_fwd_varlen")
    else:
        _check(lib.attn_fwd_varlen_counted(*args, _ptr(counter), _stream()), "attn_fwd_varlen_counted")
    return o, lse


def attn_fwd_f32(q, k, v, o=None, lse=None, scale=None, causal=False, window_left=-1, window_right=-1):
    """fp32 prefill forward on the CUDA cores.  Same arguments as attn_fwd."""
    _want(q, torch.float32, 4, "q")
    _want(k, torch.float32, 4, "k")
    _want(v, torch.float32, 4, "v")
    B, H, Lq, d = q.shape
    dev = q.device
    Lk = k.shape[2]
    _want(k, torch.float32, 4, "k", shape=(B, H, Lk, d), device=dev)
    _want(v, torch.float32, 4, "v", shape=(B, H, Lk, d), device=dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.float32, 4, "o", shape=(B, H, Lq, d), device=dev)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 3, "lse", shape=(B, H, Lq), device=dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    _check(lib.attn_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, Lq, Lk, d, scale,
                            int(bool(causal)), int(window_left), int(window_right), _stream()), "attn_fwd_f32")
    return o, lse


def attn_decode_auto_splits(B, H, Lk, d) -> int:
    return lib.attn_decode_auto_splits(B, H, Lk, d)


def attn_decode_workspace_bytes(B, H, Lk, d, num_splits=0) -> int:
    return lib.attn_decode_workspace_bytes(B, H, Lk, d, num_splits)


def attn_decode_splitkv(q, k_cache, v_cache, o=None, lse=None, seqlens_k=None, scale=None,
                        num_splits=0, workspace=None):
    """Split-KV decode.  q: [B,H,1,d], caches [B,H,Lk,d] -> (o [B,H,1,d], lse [B,H])."""
    _want(q, torch.bfloat16, 4, "q")
    _want(k_cache, torch.bfloat16, 4, "k_cache")
    _want(v_cache, torch.bfloat16, 4, "v_cache")
    B, H, Lq, d = q.shape
    dev = q.device
    if Lq != 1:
        raise ValueError(f"q: decode takes one query per head, got Lq={Lq}")
    Lk = k_cache.shape[2]
    _want(k_cache, torch.bfloat16, 4, "k_cache", shape=(B, H, Lk, d), device=dev)
    _want(v_cache, torch.bfloat16, 4, "v_cache", shape=(B, H, Lk, d), device=dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.bfloat16, 4, "o", shape=(B, H, 1, d), device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 2, "lse", shape=(B, H), device=dev)
    if seqlens_k is not None:
        _want(seqlens_k, torch.int32, 1, "seqlens_k", shape=(B,), device=dev)
    S = num_splits if num_splits > 0 else attn_decode_auto_splits(B, H, Lk, d)
    need = attn_decode_workspace_bytes(B, H, Lk, d, S)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _want_workspace(workspace, dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    _check(lib.attn_decode_splitkv(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                                   _ptr(seqlens_k), B, H, Lk, d, scale, S, _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream()),
           "attn_decode_splitkv")
    return o, lse


def attn_decode_splitkv_noalloc(q, k_cache, v_cache, o=None, lse=None, seqlens_k=None, scale=None,
                                num_splits=0):
    """Split-KV decode whose split partials live in the library's own static
    scratch (for callers that cannot allocate device memory); o and lse are
    still the caller's.  Same results as attn_decode_splitkv."""
    _want(q, torch.bfloat16, 4, "q")
    _want(k_cache, torch.bfloat16, 4, "k_cache")
    _want(v_cache, torch.bfloat16, 4, "v_cache")
    B, H, Lq, d = q.shape
    dev = q.device
    if Lq != 1:
        raise ValueError(f"q: decode takes one query per head, got Lq={Lq}")
    Lk = k_cache.shape[2]
    _want(k_cache, torch.bfloat16, 4, "k_cache", shape=(B, H, Lk, d), device=dev)
    _want(v_cache, torch.bfloat16, 4, "v_cache", shape=(B, H, Lk, d), device=dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.bfloat16, 4, "o", shape=(B, H, 1, d), device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 2, "lse", shape=(B, H), device=dev)
    if seqlens_k is not None:
        _want(seqlens_k, torch.int32, 1, "seqlens_k", shape=(B,), device=dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    _check(lib.attn_decode_splitkv_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(o), _ptr(lse),
                                           _ptr(seqlens_k), B, H, Lk, d, scale, int(num_splits), _stream()),
           "attn_decode_splitkv_noalloc")
    return o, lse


def attn_decode_paged(q, k_pages, v_pages, block_table, seqlens_k, o=None, lse=None, scale=None, num_splits=0,
                      workspace=None):
    """Split-KV decode over a paged cache.  q: [B,H,1,d]; k_pages, v_pages:
    [num_pages, page_size, H, d] bf16; block_table: int32 [B, max_pages];
    seqlens_k: int32 [B] -> (o [B,H,1,d], lse [B,H])."""
    _want(q, torch.bfloat16, 4, "q")
    _want(k_pages, torch.bfloat16, 4, "k_pages")
    _want(v_pages, torch.bfloat16, 4, "v_pages")
    _want(block_table, torch.int32, 2, "block_table")
    _want(seqlens_k, torch.int32, 1, "seqlens_k")
    B, H, Lq, d = q.shape
    dev = q.device
    if Lq != 1:
        raise ValueError(f"q: decode takes one query per head, got Lq={Lq}")
    num_pages, page_size = k_pages.shape[0], k_pages.shape[1]
    max_pages = block_table.shape[1]
    Lk = max_pages * page_size
    _want(k_pages, torch.bfloat16, 4, "k_pages", shape=(num_pages, page_size, H, d), device=dev)
    _want(v_pages, torch.bfloat16, 4, "v_pages", shape=(num_pages, page_size, H, d), device=dev)
    _want(block_table, torch.int32, 2, "block_table", shape=(B, max_pages), device=dev)
    _want(seqlens_k, torch.int32, 1, "seqlens_k", shape=(B,), device=dev)
    if o is None:
        o = torch.empty_like(q)
    _want(o, torch.bfloat16, 4, "o", shape=(B, H, 1, d), device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 2, "lse", shape=(B, H), device=dev)
    S = num_splits if num_splits > 0 else attn_decode_auto_splits(B, H, Lk, d)
    if workspace is None:
        workspace = torch.empty(attn_decode_workspace_bytes(B, H, Lk, d, S), dtype=torch.uint8, device=dev)
    _want_workspace(workspace, dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    _check(lib.attn_decode_paged(_ptr(q), _ptr(k_pages), _ptr(v_pages), _ptr(block_table), max_pages, page_size,
                                 num_pages, _ptr(o), _ptr(lse), _ptr(seqlens_k), B, H, d, scale, S, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream()), "attn_decode_paged")
    return o, lse


# The calls of a serving step are short (a few us on the GPU).  Their ordinary
# case runs in native code (csrc/binding.cpp: the same checks and allocations,
# then the same library call); it answers None to anything else, which then goes
# through the checks below and gets their messages.  The module is built against
# one torch and loaded with that one only; without it every call takes the checks
# below, with the same results some 10 us later.
def _load_calls(path):
    """The native module at ``path``, bound to the library's functions, or None where there is none that loads."""
    if not os.path.exists(path):
        return None
    spec = importlib.util.spec_from_file_location("io_aware_exact_34_b200._fattn_calls", path)
    try:
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except ImportError as e:
        warnings.warn(f"{path} does not load ({e}); the paged-cache calls go without it")
        return None
    for name in ("attn_paged_plan", "attn_append_paged_fp8", "attn_decode_paged_fp8", "attn_decode_paged_fp8_auto_splits",
                 "attn_fwd_paged_fp8", "attn_fwd_paged_fp8_workspace_bytes"):
        module.bind(name, ctypes.cast(getattr(lib, name), ctypes.c_void_p).value)
    return module


_calls = _load_calls(calls_path(torch.__version__))
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _need(t, dtype, shape, index, name):
    """_want for a tensor of one exact shape (a tuple) on CUDA device `index`."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _want(t, dtype, len(shape), name, shape=shape, device=torch.device("cuda", index))


def _first(t, dtype, ndim, name):
    """The first tensor of a call -> its device index, which has to be the
    current device's: the library launches there."""
    _want(t, dtype, ndim, name)
    index = t.get_device()
    if index != torch.cuda.current_device():
        raise ValueError(f"{name}: on cuda:{index}, but the current device is cuda:{torch.cuda.current_device()}")
    return index


_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # device index -> cudaStream_t (torch without CUDA: none)


def _int32(x, name):
    """An integer that the C ABI takes in 32 bits: ctypes would drop its upper ones."""
    x = operator.index(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name}: {x} is beyond 32 bits")
    return x


def _window(x):
    """A window's length for the C ABI: negative is unlimited, and 2^31 - 1 is wider than any sequence."""
    return max(-1, min(operator.index(x), 2 ** 31 - 1))


def attn_paged_plan(seqlens_k, seqlens_new, free_pages, block_table, page_size, max_tokens, slot_map=None,
                    cu_seqlens=None, seqlens_out=None, counts=None):
    """Where the new tokens of a batch go in a paged cache.  seqlens_k,
    seqlens_new: int32 [B], tokens held and tokens arriving; free_pages: int32
    [num_free] physical pages not in use; block_table: int32 [B, max_pages],
    updated in place with the pages taken -> (slot_map int64 [max_tokens],
    cu_seqlens int32 [B + 1], seqlens_out int32 [B], counts int32 [2]: tokens,
    pages needed).  Tokens without a page and places behind the last token have
    slot -1.  cu_seqlens, seqlens_out and counts may be parts of one allocation,
    which lives as long as any of them."""
    if _calls is not None and slot_map is None and cu_seqlens is None and seqlens_out is None and counts is None:
        got = _calls.plan(seqlens_k, seqlens_new, free_pages, block_table, page_size, max_tokens)
        if got is not None:
            return got
    page_size, max_tokens = _int32(page_size, "page_size"), _int32(max_tokens, "max_tokens")
    dev = _first(seqlens_k, _I32, 1, "seqlens_k")
    B = seqlens_k.shape[0]
    _need(seqlens_new, _I32, (B,), dev, "seqlens_new")
    _want(free_pages, _I32, 1, "free_pages")
    _need(free_pages, _I32, free_pages.shape, dev, "free_pages")
    max_pages = _table_width(block_table, B, dev)
    if slot_map is None:
        slot_map = seqlens_k.new_empty(max_tokens, dtype=_I64)
    else:
        _need(slot_map, _I64, (max_tokens,), dev, "slot_map")
    if cu_seqlens is None:
        cu_seqlens = seqlens_k.new_empty(B + 1)
    else:
        _need(cu_seqlens, _I32, (B + 1,), dev, "cu_seqlens")
    if seqlens_out is None:
        seqlens_out = torch.empty_like(seqlens_k)
    else:
        _need(seqlens_out, _I32, (B,), dev, "seqlens_out")
    if counts is None:
        counts = seqlens_k.new_empty(2)
    else:
        _need(counts, _I32, (2,), dev, "counts")
    st = lib.attn_paged_plan(seqlens_k.data_ptr(), seqlens_new.data_ptr(), B, free_pages.data_ptr(), free_pages.shape[0],
                             block_table.data_ptr(), max_pages, page_size, slot_map.data_ptr(), max_tokens,
                             cu_seqlens.data_ptr(), seqlens_out.data_ptr(), counts.data_ptr(), _stream_of(dev))
    _check(st, "attn_paged_plan")
    return slot_map, cu_seqlens, seqlens_out, counts


def _table_width(block_table, B, dev):
    """The int32 [B, max_pages] table's max_pages."""
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        _want(block_table, _I32, 2, "block_table")
    max_pages = block_table.shape[1]
    _need(block_table, _I32, (B, max_pages), dev, "block_table")
    return max_pages


def _cache_shape(k_pages, v_pages, k_scales, v_scales, dev):
    """The four tensors of a paged 8-bit cache -> (num_pages, page_size, Hkv, d)."""
    _want(k_pages, _U8, 4, "k_pages")
    shape = k_pages.shape
    scales = (shape[0], shape[2])
    _need(k_pages, _U8, shape, dev, "k_pages")
    _need(v_pages, _U8, shape, dev, "v_pages")
    _need(k_scales, _F32, scales, dev, "k_scales")
    _need(v_scales, _F32, scales, dev, "v_scales")
    return shape


def _want_rows(t, name, shape, dev):
    """bf16 rows [tokens, H, d] whose tokens may be apart (a view of a fused
    projection); the heads of a token are contiguous -> the token stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    tokens, H, d = shape
    st = t.stride()
    if t.dtype != _BF16 or t.get_device() != dev or t.shape != shape or st[2] != 1 or (H > 1 and st[1] != d) \
            or (tokens > 1 and st[0] < H * d):
        raise ValueError(f"{name}: expected bf16 rows {tuple(shape)} on cuda:{dev} with contiguous heads, got "
                         f"{t.dtype} {tuple(t.shape)}, strides {st}, on {t.device}")
    return st[0] if tokens > 1 else H * d


def attn_append_paged_fp8(k, v, slot_map, k_pages, v_pages, k_scales, v_scales):
    """Quantize new rows into a paged 8-bit cache, in place.  k, v: bf16
    [tokens, Hkv, d] (token stride free); slot_map: int64 [tokens] (the first
    tokens of a longer map are taken as a slice); k_pages, v_pages: uint8 e4m3
    codes [num_pages, page_size, Hkv, d]; k_scales, v_scales: fp32
    [num_pages, Hkv]."""
    if _calls is not None and _calls.append(k, v, slot_map, k_pages, v_pages, k_scales, v_scales):
        return
    dev = _first(slot_map, _I64, 1, "slot_map")
    num_pages, page_size, H, d = _cache_shape(k_pages, v_pages, k_scales, v_scales, dev)
    tokens = slot_map.shape[0]
    rows = (tokens, H, d)
    ks, vs = _want_rows(k, "k", rows, dev), _want_rows(v, "v", rows, dev)
    st = lib.attn_append_paged_fp8(k.data_ptr(), v.data_ptr(), ks, vs, slot_map.data_ptr(), tokens, k_pages.data_ptr(),
                                   v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), num_pages, page_size,
                                   H, d, _stream_of(dev))
    _check(st, "attn_append_paged_fp8")


def attn_decode_paged_fp8_auto_splits(B, Hq, Hkv, Lk, d) -> int:
    return lib.attn_decode_paged_fp8_auto_splits(B, Hq, Hkv, _int32(Lk, "Lk"), d)


def _want_heads(Hq, d, Hkv, dk):
    if dk != d or Hkv == 0 or Hq % Hkv:
        raise ValueError(f"k_pages: heads of {dk} elements, {Hkv} of them, do not serve {Hq} query heads of {d}")


def attn_decode_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, o=None, lse=None, scale=None,
                          window_left=-1, num_splits=0, workspace=None):
    """Split-KV decode over a paged 8-bit cache.  q: bf16 [B,Hq,1,d]; cache as
    attn_append_paged_fp8; block_table: int32 [B, max_pages]; seqlens_k: int32
    [B], the new token included -> (o [B,Hq,1,d], lse [B,Hq])."""
    if _calls is not None and o is None and lse is None and workspace is None:
        got = _calls.decode(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, scale, window_left, num_splits)
        if got is not None:
            return got
    window_left, num_splits = _window(window_left), _int32(num_splits, "num_splits")
    dev = _first(q, _BF16, 4, "q")
    B, Hq, Lq, d = q.shape
    if Lq != 1:
        raise ValueError(f"q: decode takes one query per head, got Lq={Lq}")
    num_pages, page_size, Hkv, dk = _cache_shape(k_pages, v_pages, k_scales, v_scales, dev)
    _want_heads(Hq, d, Hkv, dk)
    max_pages = _table_width(block_table, B, dev)
    _need(seqlens_k, _I32, (B,), dev, "seqlens_k")
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, _BF16, (B, Hq, 1, d), dev, "o")
    if lse is None:
        lse = k_scales.new_empty((B, Hq))
    else:
        _need(lse, _F32, (B, Hq), dev, "lse")
    if workspace is None:
        Lk = max_pages * page_size
        S = num_splits if num_splits != 0 else lib.attn_decode_paged_fp8_auto_splits(B, Hq, Hkv, Lk, d)
        need = 4 * B * Hq * S * (d + 1) if S > 1 else 0  # attn_decode_workspace_bytes
        workspace = k_pages.new_empty(need) if need > 0 else None
    else:
        _want_workspace(workspace, q.device)
        need = workspace.numel() * workspace.element_size()
    st = lib.attn_decode_paged_fp8(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                                   v_scales.data_ptr(), block_table.data_ptr(), max_pages, page_size, num_pages,
                                   o.data_ptr(), lse.data_ptr(), seqlens_k.data_ptr(), B, Hq, Hkv, d,
                                   d ** -0.5 if scale is None else scale, window_left, num_splits,
                                   None if workspace is None else workspace.data_ptr(), need, _stream_of(dev))
    _check(st, "attn_decode_paged_fp8")
    return o, lse


def attn_fwd_paged_fp8_workspace_bytes(B, total_q, max_seqlen_q, Hq, Hkv, Lk, d) -> int:
    return lib.attn_fwd_paged_fp8_workspace_bytes(B, _int32(total_q, "total_q"), _int32(max_seqlen_q, "max_seqlen_q"), Hq, Hkv,
                                                  _int32(Lk, "Lk"), d)


def attn_fwd_paged_fp8(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q,
                       o=None, lse=None, scale=None, causal=False, window_left=-1, window_right=-1, workspace=None):
    """Packed prefill over a paged 8-bit cache.  q: bf16 [total_q, Hq, d], the
    new tokens of all sequences; cu_seqlens_q: int32 [B + 1]; seqlens_k: int32
    [B], the new tokens included; cache and block_table as
    attn_decode_paged_fp8 -> (o [total_q, Hq, d], lse [Hq, total_q])."""
    if _calls is not None and o is None and lse is None and workspace is None:
        got = _calls.fwd(q, k_pages, v_pages, k_scales, v_scales, block_table, seqlens_k, cu_seqlens_q, max_seqlen_q, scale,
                         causal, window_left, window_right)
        if got is not None:
            return got
    max_seqlen_q = _int32(max_seqlen_q, "max_seqlen_q")
    window_left, window_right = _window(window_left), _window(window_right)
    dev = _first(q, _BF16, 3, "q")
    total_q, Hq, d = q.shape
    num_pages, page_size, Hkv, dk = _cache_shape(k_pages, v_pages, k_scales, v_scales, dev)
    _want_heads(Hq, d, Hkv, dk)
    _want(seqlens_k, _I32, 1, "seqlens_k")
    B = seqlens_k.shape[0]
    _need(seqlens_k, _I32, (B,), dev, "seqlens_k")
    max_pages = _table_width(block_table, B, dev)
    _need(cu_seqlens_q, _I32, (B + 1,), dev, "cu_seqlens_q")
    if o is None:
        o = torch.empty_like(q)
    else:
        _need(o, _BF16, (total_q, Hq, d), dev, "o")
    if lse is None:
        lse = k_scales.new_empty((Hq, total_q))
    else:
        _need(lse, _F32, (Hq, total_q), dev, "lse")
    if workspace is None:
        need = lib.attn_fwd_paged_fp8_workspace_bytes(B, total_q, max_seqlen_q, Hq, Hkv, max_pages * page_size, d)
        workspace = k_pages.new_empty(need) if need > 0 else None
    else:
        _want_workspace(workspace, q.device)
        need = workspace.numel() * workspace.element_size()
    st = lib.attn_fwd_paged_fp8(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                                v_scales.data_ptr(), block_table.data_ptr(), max_pages, page_size, num_pages,
                                o.data_ptr(), lse.data_ptr(), seqlens_k.data_ptr(), cu_seqlens_q.data_ptr(), B, total_q,
                                max_seqlen_q, Hq, Hkv, d, d ** -0.5 if scale is None else scale, int(bool(causal)),
                                window_left, window_right, None if workspace is None else workspace.data_ptr(), need,
                                _stream_of(dev))
    _check(st, "attn_fwd_paged_fp8")
    return o, lse


def attn_fp8_ld(Lk) -> int:
    return lib.attn_fp8_ld(Lk)


def attn_quantize_fp8(x, transpose=False, codes=None, descale=None):
    """bf16 [B,H,L,d] -> (e4m3 codes as uint8 [B,H,L,d], or [B,H,d,ld] when
    transposed; fp32 descale [B,H])."""
    _want(x, torch.bfloat16, 4, "x")
    B, H, L, d = x.shape
    dev = x.device
    shape = (B, H, d, attn_fp8_ld(L)) if transpose else (B, H, L, d)
    if codes is None:
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
    _want(codes, torch.uint8, 4, "codes", shape=shape, device=dev)
    if descale is None:
        descale = torch.empty((B, H), dtype=torch.float32, device=dev)
    _want(descale, torch.float32, 2, "descale", shape=(B, H), device=dev)
    _check(lib.attn_quantize_fp8(_ptr(x), _ptr(codes), _ptr(descale), B, H, L, d, int(bool(transpose)), _stream()),
           "attn_quantize_fp8")
    return codes, descale


def attn_fwd_fp8(q8, k8, vt8, q_descale, k_descale, v_descale, o=None, lse=None, scale=None, causal=False,
                 window_left=-1, window_right=-1, counter=None):
    """FP8 prefill forward.  q8: [B,H,Lq,128], k8: [B,H,Lk,128] and vt8:
    [B,H,128,ld] uint8 e4m3 codes; descales fp32 [B,H] -> (o bf16, lse fp32)."""
    for t, name in ((q8, "q8"), (k8, "k8"), (vt8, "vt8")):
        _want(t, torch.uint8, 4, name)
    for t, name in ((q_descale, "q_descale"), (k_descale, "k_descale"), (v_descale, "v_descale")):
        _want(t, torch.float32, 2, name)
    B, H, Lq, d = q8.shape
    dev = q8.device
    Lk = k8.shape[2]
    _want(k8, torch.uint8, 4, "k8", shape=(B, H, Lk, d), device=dev)
    _want(vt8, torch.uint8, 4, "vt8", shape=(B, H, d, attn_fp8_ld(Lk)), device=dev)
    for t, name in ((q_descale, "q_descale"), (k_descale, "k_descale"), (v_descale, "v_descale")):
        _want(t, torch.float32, 2, name, shape=(B, H), device=dev)
    _want_counter(counter, dev)
    if o is None:
        o = torch.empty((B, H, Lq, d), dtype=torch.bfloat16, device=dev)
    _want(o, torch.bfloat16, 4, "o", shape=(B, H, Lq, d), device=dev)
    if lse is None:
        lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev)
    _want(lse, torch.float32, 3, "lse", shape=(B, H, Lq), device=dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    args = (_ptr(q8), _ptr(k8), _ptr(vt8), _ptr(q_descale), _ptr(k_descale), _ptr(v_descale), _ptr(o), _ptr(lse),
            B, H, Lq, Lk, d, scale, int(bool(causal)), int(window_left), int(window_right))
    if counter is None:
        _check(lib.attn_fwd_fp8(*args, _stream()), "attn_fwd_fp8")
    else:
        _check(lib.attn_fwd_fp8_counted(*args, _ptr(counter), _stream()), "attn_fwd_fp8_counted")
    return o, lse


def attn_bwd_workspace_bytes(B, H, Lq, d) -> int:
    return lib.attn_bwd_workspace_bytes(B, H, Lq, d)


def attn_bwd(q, k, v, o, dout, lse, scale=None, causal=False, window_left=-1, window_right=-1, dq=None, dk=None,
             dv=None, workspace=None, counter=None):
    """Attention backward with recomputation.  q, o, dout: [B,H,Lq,d], k, v:
    [B,H,Lk,d] bf16; lse: fp32 [B,H,Lq] from attn_fwd -> (dq, dk, dv) bf16.
    ``counter`` (optional, a zeroed one-element int64 CUDA tensor) receives the
    number of (key tile, query tile) pairs computed."""
    for t, name in ((q, "q"), (k, "k"), (v, "v"), (o, "o"), (dout, "dout")):
        _want(t, torch.bfloat16, 4, name)
    _want(lse, torch.float32, 3, "lse")
    B, H, Lq, d = q.shape
    dev = q.device
    Lk = k.shape[2]
    for t, name, shp in ((k, "k", (B, H, Lk, d)), (v, "v", (B, H, Lk, d)), (o, "o", (B, H, Lq, d)),
                         (dout, "dout", (B, H, Lq, d))):
        _want(t, torch.bfloat16, 4, name, shape=shp, device=dev)
    _want(lse, torch.float32, 3, "lse", shape=(B, H, Lq), device=dev)
    _want_counter(counter, dev)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    for t, name, shp in ((dq, "dq", (B, H, Lq, d)), (dk, "dk", (B, H, Lk, d)), (dv, "dv", (B, H, Lk, d))):
        _want(t, torch.bfloat16, 4, name, shape=shp, device=dev)
    if workspace is None:
        workspace = torch.empty(attn_bwd_workspace_bytes(B, H, Lq, d), dtype=torch.uint8, device=dev)
    _want_workspace(workspace, dev)
    scale = (1.0 / d ** 0.5) if scale is None else scale
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv), B, H, Lq, Lk, d,
            scale, int(bool(causal)), int(window_left), int(window_right), _ptr(workspace),
            workspace.numel() * workspace.element_size())
    if counter is None:
        _check(lib.attn_bwd(*args, _stream()), "attn_bwd")
    else:
        _check(lib.attn_bwd_counted(*args, _ptr(counter), _stream()), "attn_bwd_counted")
    return dq, dk, dv


def attn_bwd_count_blocks(Lq, Lk, causal=False, window_left=-1, window_right=-1, block_q=128, block_k=128) -> int:
    """Host-side: (query tile, key tile) pairs the backward visits per head."""
    out = ctypes.c_longlong(0)
    _check(lib.attn_bwd_count_blocks(Lq, Lk, int(bool(causal)), window_left, window_right, block_q, block_k,
                                     ctypes.byref(out)), "attn_bwd_count_blocks")
    return out.value


def attn_count_blocks(Lq, Lk, causal=False, window_left=-1, window_right=-1, block_q=128, block_k=128):
    """Host-side block accounting -> dict(visited, total, partial, pairs)."""
    out = [ctypes.c_longlong(0) for _ in range(4)]
    _check(lib.attn_count_blocks(Lq, Lk, int(bool(causal)), window_left, window_right, block_q, block_k,
                                 *[ctypes.byref(x) for x in out]), "attn_count_blocks")
    return dict(visited=out[0].value, total=out[1].value, partial=out[2].value, pairs=out[3].value)


def fattn_device_status() -> int:
    return lib.fattn_device_status(_stream())


def fattn_debug_inject_stall(on: bool = True) -> None:
    """Test hook: the next prefill launch lets its bounded waits run out."""
    _check(lib.fattn_debug_inject_stall(int(bool(on))), "fattn_debug_inject_stall")


def status_string(status: int) -> str:
    return lib.fattn_status_string(status).decode()
