"""Thin Python binding of libfa.so (exact attention on GB300).

The functions carry the C entry points' names and only marshal arguments: torch tensors give device
pointers and the current CUDA stream; every step of the computation runs in the library's kernels.
There is no fallback: if ``libfa.so`` is missing or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")

FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_TIMEOUT = range(5)
STATUS_NAMES = {0: "FA_OK", 1: "FA_ERR_INVALID_ARG", 2: "FA_ERR_UNSUPPORTED", 3: "FA_ERR_CUDA", 4: "FA_ERR_TIMEOUT"}

# Every symbol include/fa.h declares.
EXPORTS = ("fa_fwd", "fa_fwd_stepnorm", "fa_fwd_f32", "fa_bwd_workspace_size", "fa_bwd", "fa_bwd_noalloc",
           "fa_last_error_string", "fa_check_status", "fa_kernel_launches", "fa_test_force_wait_timeout",
           "fa_debug_time_bwd_main", "fa_cross_fwd_workspace_size", "fa_cross_fwd", "fa_cross_bwd_workspace_size",
           "fa_cross_bwd", "fa_cache_plan", "fa_cache_append", "fa_cache_fwd_workspace_size", "fa_cache_fwd")

# Bytes of the static scratch that fa_bwd_noalloc uses (FA_BWD_NOALLOC_MAX_SCRATCH_BYTES).
NOALLOC_MAX_SCRATCH_BYTES = 32 << 20

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Loads libfa.so and declares the C signatures; raises if the library is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m exact_io_aware_17_gb300.build`")
    lib = ctypes.CDLL(path)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    lib.fa_fwd.argtypes = [P, P, P, P, P, I, I, I, I, F, P]
    lib.fa_fwd.restype = I
    lib.fa_fwd_stepnorm.argtypes = [P, P, P, P, P, I, I, I, I, F, P]
    lib.fa_fwd_stepnorm.restype = I
    lib.fa_fwd_f32.argtypes = [P, P, P, P, P, I, I, I, I, F, P]
    lib.fa_fwd_f32.restype = I
    lib.fa_bwd_workspace_size.argtypes = [I, I, I, I]
    lib.fa_bwd_workspace_size.restype = Z
    lib.fa_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, P, Z, P]
    lib.fa_bwd.restype = I
    lib.fa_bwd_noalloc.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, F, P]
    lib.fa_bwd_noalloc.restype = I
    lib.fa_last_error_string.argtypes = []
    lib.fa_last_error_string.restype = ctypes.c_char_p
    lib.fa_check_status.argtypes = [P]
    lib.fa_check_status.restype = I
    lib.fa_kernel_launches.argtypes = []
    lib.fa_kernel_launches.restype = ctypes.c_ulonglong
    lib.fa_debug_time_bwd_main.argtypes = [P, P]
    lib.fa_debug_time_bwd_main.restype = None
    lib.fa_test_force_wait_timeout.argtypes = [I]
    lib.fa_test_force_wait_timeout.restype = None
    L = ctypes.c_longlong
    lib.fa_cross_fwd_workspace_size.argtypes = [I] * 6
    lib.fa_cross_fwd_workspace_size.restype = Z
    lib.fa_cross_fwd.argtypes = [P] * 6 + [I] * 6 + [F, P, Z, P]
    lib.fa_cross_fwd.restype = I
    lib.fa_cross_bwd_workspace_size.argtypes = [I] * 6
    lib.fa_cross_bwd_workspace_size.restype = Z
    lib.fa_cross_bwd.argtypes = [P] * 10 + [I] * 6 + [F, P, Z, P]
    lib.fa_cross_bwd.restype = I
    lib.fa_cache_plan.argtypes = [P] * 9 + [I] * 5 + [P]
    lib.fa_cache_plan.restype = I
    lib.fa_cache_append.argtypes = [P] * 7 + [I] * 3 + [L] * 4 + [I] * 2 + [P]
    lib.fa_cache_append.restype = I
    lib.fa_cache_fwd_workspace_size.argtypes = [I] * 7
    lib.fa_cache_fwd_workspace_size.restype = Z
    lib.fa_cache_fwd.argtypes = [P] * 9 + [I] * 8 + [F, P, Z, P]
    lib.fa_cache_fwd.restype = I
    _lib = lib
    return lib


def _check(status: int):
    if status != FA_OK:
        msg = load_library().fa_last_error_string().decode(errors="replace")
        raise FAError(status, msg)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, device=None):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _shape(q):
    if q.dim() != 4:
        raise ValueError("expected [B, H, N, d] tensors")
    return tuple(int(x) for x in q.shape)


def _default_scale(d, scale):
    return 1.0 / math.sqrt(d) if scale is None else float(scale)


def _check_tensor(name, t, shape, dtype, device=None):
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor of shape {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device} (every tensor of a call on one GPU)")


def _scratch(shape, dtype, device, stream):
    """Memory that the call allocates: on a given stream, of that stream's pool, where nothing that the caller's stream
    still has queued can be using it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _new(shape, dtype, device, stream):
    """An output that the call allocates: torch hands its memory on only when the caller's stream is done with it too."""
    t = _scratch(shape, dtype, device, stream)
    if stream is not None:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def fa_fwd(q, k, v, scale=None, o=None, lse=None, stream=None, _entry="fa_fwd"):
    """bf16 forward: returns (o bf16 [B,H,N,d], lse fp32 [B,H,N])."""
    B, H, N, d = _shape(q)
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, (B, H, N, d), torch.bfloat16, dev)
    o = _new((B, H, N, d), torch.bfloat16, dev, stream) if o is None else o
    lse = _new((B, H, N), torch.float32, dev, stream) if lse is None else lse
    _check_tensor("o", o, (B, H, N, d), torch.bfloat16, dev)
    _check_tensor("lse", lse, (B, H, N), torch.float32, dev)
    with torch.cuda.device(dev):
        _check(getattr(load_library(), _entry)(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                               _default_scale(d, scale), _stream(stream, dev)))
    return o, lse


def fa_fwd_stepnorm(q, k, v, scale=None, o=None, lse=None, stream=None):
    """bf16 forward with the per-step normalised accumulator (ablation of fa_fwd's update rule)."""
    return fa_fwd(q, k, v, scale, o, lse, stream, _entry="fa_fwd_stepnorm")


def fa_fwd_f32(q, k, v, scale=None, o=None, lse=None, stream=None):
    """fp32 forward: returns (o fp32 [B,H,N,d], lse fp32 [B,H,N])."""
    B, H, N, d = _shape(q)
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, (B, H, N, d), torch.float32, dev)
    o = _new((B, H, N, d), torch.float32, dev, stream) if o is None else o
    lse = _new((B, H, N), torch.float32, dev, stream) if lse is None else lse
    _check_tensor("o", o, (B, H, N, d), torch.float32, dev)
    _check_tensor("lse", lse, (B, H, N), torch.float32, dev)
    with torch.cuda.device(dev):
        _check(load_library().fa_fwd_f32(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), B, H, N, d,
                                         _default_scale(d, scale), _stream(stream, dev)))
    return o, lse


def fa_bwd_workspace_size(B, H, N, d) -> int:
    return int(load_library().fa_bwd_workspace_size(B, H, N, d))


def fa_bwd(q, k, v, o, do, lse, scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """bf16 backward: returns (dq, dk, dv), bf16 [B,H,N,d].  ``workspace`` is a uint8 CUDA tensor of at
    least fa_bwd_workspace_size(B,H,N,d) bytes; one is allocated by torch if not given."""
    B, H, N, d = _shape(q)
    dev = q.device
    dq, dk, dv = _bwd_outputs(q, k, v, o, do, lse, dq, dk, dv, stream)
    if workspace is None:
        workspace = _scratch((fa_bwd_workspace_size(B, H, N, d),), torch.uint8, dev, stream)
    if not workspace.is_cuda or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {dev}")
    with torch.cuda.device(dev):
        _check(load_library().fa_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq), _ptr(dk),
                                     _ptr(dv), B, H, N, d, _default_scale(d, scale), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream, dev)))
    return dq, dk, dv


def _bwd_outputs(q, k, v, o, do, lse, dq, dk, dv, stream):
    """Checks the backward's inputs and caller-given outputs (dtype, shape, contiguity, one device) and
    allocates the outputs not given."""
    B, H, N, d = _shape(q)
    dev = q.device
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("do", do)):
        _check_tensor(name, t, (B, H, N, d), torch.bfloat16, dev)
    _check_tensor("lse", lse, (B, H, N), torch.float32, dev)
    dq = _new((B, H, N, d), torch.bfloat16, dev, stream) if dq is None else dq
    dk = _new((B, H, N, d), torch.bfloat16, dev, stream) if dk is None else dk
    dv = _new((B, H, N, d), torch.bfloat16, dev, stream) if dv is None else dv
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        _check_tensor(name, t, (B, H, N, d), torch.bfloat16, dev)
    return dq, dk, dv


def fa_bwd_noalloc(q, k, v, o, do, lse, scale=None, dq=None, dk=None, dv=None, stream=None):
    """bf16 backward that allocates no scratch: the library's static scratch array stands in for the
    workspace (for callers that cannot allocate device memory).  Pass preallocated dq, dk, dv to make
    the call allocate nothing at all; shapes needing more than NOALLOC_MAX_SCRATCH_BYTES of scratch
    raise FAError (FA_ERR_INVALID_ARG)."""
    B, H, N, d = _shape(q)
    dev = q.device
    dq, dk, dv = _bwd_outputs(q, k, v, o, do, lse, dq, dk, dv, stream)
    with torch.cuda.device(dev):
        _check(load_library().fa_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(do), _ptr(lse), _ptr(dq),
                                             _ptr(dk), _ptr(dv), B, H, N, d, _default_scale(d, scale),
                                             _stream(stream, dev)))
    return dq, dk, dv


def _call(entry, device, *args):
    """Calls a C entry point with the tensors' GPU as the current one (which costs nothing where it already is)."""
    if torch._C._cuda_getDevice() == device.index:
        status = entry(*args)
    else:
        with torch.cuda.device(device):
            status = entry(*args)
    if status:
        _check(status)


def _raw_stream(stream, device):
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


def _need(name, t, shape, dtype, device):
    """_check_tensor for the calls of a decoding step, which are short: no temporaries where the tensor is right."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != device or not t.is_cuda:
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on one CUDA device (that of "
                         f"the call's first tensor), got {t.dtype} {tuple(t.shape)} on {t.device}")


def _output(name, t, shape, dtype, device, stream):
    """The caller's output tensor, checked, or a new one."""
    if t is None:
        return _new(shape, dtype, device, stream)
    _need(name, t, shape, dtype, device)
    return t


def _check_workspace(workspace, need, device, stream):
    """The caller's workspace, or one of the call's stream that torch allocates; (None, 0) where the call needs none."""
    if workspace is None:
        if not need:
            return None, 0
        workspace = _scratch((need,), torch.uint8, device, stream)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace: expected a contiguous tensor on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _cross_shape(q, k):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("expected q [B, Hq, Nq, d] and k [B, Hk, Nk, d]")
    (B, Hq, Nq, d), (Bk, Hk, Nk, dk) = q.shape, k.shape
    if Bk != B or dk != d:
        raise ValueError(f"k: expected [{B}, Hk, Nk, {d}], got {tuple(k.shape)}")
    return B, Hq, Hk, Nq, Nk, d


@functools.lru_cache(maxsize=1024)
def fa_cross_fwd_workspace_size(B, Hq, Hk, Nq, Nk, d) -> int:
    return int(load_library().fa_cross_fwd_workspace_size(B, Hq, Hk, Nq, Nk, d))


def fa_cross_fwd(q, k, v, key_lens=None, scale=None, o=None, lse=None, workspace=None, stream=None):
    """bf16 forward over keys of another length: q [B,Hq,Nq,d], k and v [B,Hk,Nk,d] (Hq a multiple of Hk), key_lens
    int32 [B] or None.  Returns (o bf16 [B,Hq,Nq,d], lse fp32 [B,Hq,Nq]).  ``workspace``: a uint8 CUDA tensor of at
    least fa_cross_fwd_workspace_size bytes; torch allocates one if the call needs it and none is given."""
    B, Hq, Hk, Nq, Nk, d = _cross_shape(q, k)
    dev, bf16 = q.device, torch.bfloat16
    _need("q", q, (B, Hq, Nq, d), bf16, dev)
    _need("k", k, (B, Hk, Nk, d), bf16, dev)
    _need("v", v, (B, Hk, Nk, d), bf16, dev)
    if key_lens is not None:
        _need("key_lens", key_lens, (B,), torch.int32, dev)
    o = _output("o", o, (B, Hq, Nq, d), bf16, dev, stream)
    lse = _output("lse", lse, (B, Hq, Nq), torch.float32, dev, stream)
    lib = load_library()
    ws, ws_bytes = _check_workspace(workspace, fa_cross_fwd_workspace_size(B, Hq, Hk, Nq, Nk, d), dev, stream)
    _call(lib.fa_cross_fwd, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          None if key_lens is None else key_lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hk, Nq, Nk, d,
          _default_scale(d, scale), None if ws is None else ws.data_ptr(), ws_bytes, _raw_stream(stream, dev))
    return o, lse


@functools.lru_cache(maxsize=1024)
def fa_cross_bwd_workspace_size(B, Hq, Hk, Nq, Nk, d) -> int:
    return int(load_library().fa_cross_bwd_workspace_size(B, Hq, Hk, Nq, Nk, d))


def fa_cross_bwd(q, k, v, o, do, lse, key_lens=None, scale=None, dq=None, dk=None, dv=None, workspace=None, stream=None):
    """bf16 backward of fa_cross_fwd: returns (dq bf16 [B,Hq,Nq,d], dk, dv bf16 [B,Hk,Nk,d]).  ``workspace``: a uint8
    CUDA tensor of at least fa_cross_bwd_workspace_size bytes; torch allocates one if not given."""
    B, Hq, Hk, Nq, Nk, d = _cross_shape(q, k)
    dev, bf16 = q.device, torch.bfloat16
    _need("q", q, (B, Hq, Nq, d), bf16, dev)
    for name, t in (("k", k), ("v", v)):
        _need(name, t, (B, Hk, Nk, d), bf16, dev)
    for name, t in (("o", o), ("do", do)):
        _need(name, t, (B, Hq, Nq, d), bf16, dev)
    _need("lse", lse, (B, Hq, Nq), torch.float32, dev)
    if key_lens is not None:
        _need("key_lens", key_lens, (B,), torch.int32, dev)
    dq = _output("dq", dq, (B, Hq, Nq, d), bf16, dev, stream)
    dk = _output("dk", dk, (B, Hk, Nk, d), bf16, dev, stream)
    dv = _output("dv", dv, (B, Hk, Nk, d), bf16, dev, stream)
    lib = load_library()
    ws, ws_bytes = _check_workspace(workspace, fa_cross_bwd_workspace_size(B, Hq, Hk, Nq, Nk, d), dev, stream)
    _call(lib.fa_cross_bwd, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
          None if key_lens is None else key_lens.data_ptr(), o.data_ptr(), do.data_ptr(), lse.data_ptr(),
          dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hk, Nq, Nk, d, _default_scale(d, scale),
          None if ws is None else ws.data_ptr(), ws_bytes, _raw_stream(stream, dev))
    return dq, dk, dv


def fa_cache_plan(lens, new_lens, block_table, free_blocks, block_size, max_tokens, used=None, slots=None, starts=None,
                  total_lens=None, used_out=None, stream=None):
    """Block table and slots of a step from the requests' lengths: lens and new_lens int32 [B], block_table int32
    [B, max_blocks] (updated in place), free_blocks int32 [n_free], used int32 [1] or None.  Returns (slots int64
    [max_tokens], starts int32 [B+1], total_lens int32 [B], used_out int32 [1]); see include/fa.h."""
    i32 = torch.int32
    dev = lens.device
    if lens.dim() != 1 or block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("expected lens [B], block_table [B, max_blocks], free_blocks [n_free]")
    B, max_blocks, n_free = int(lens.shape[0]), int(block_table.shape[1]), int(free_blocks.shape[0])
    _need("lens", lens, (B,), i32, dev)
    _need("new_lens", new_lens, (B,), i32, dev)
    _need("block_table", block_table, (B, max_blocks), i32, dev)
    _need("free_blocks", free_blocks, (n_free,), i32, dev)
    if used is not None:
        _need("used", used, (1,), i32, dev)
    slots = _output("slots", slots, (max_tokens,), torch.int64, dev, stream)
    starts = _output("starts", starts, (B + 1,), i32, dev, stream)
    total_lens = _output("total_lens", total_lens, (B,), i32, dev, stream)
    used_out = _output("used_out", used_out, (1,), i32, dev, stream)
    _call(load_library().fa_cache_plan, dev, lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
          free_blocks.data_ptr(), None if used is None else used.data_ptr(), slots.data_ptr(), starts.data_ptr(),
          total_lens.data_ptr(), used_out.data_ptr(), B, max_blocks, n_free, max_tokens, block_size, _raw_stream(stream,
          dev))
    return slots, starts, total_lens, used_out


def _check_cache(k_cache, v_cache, k_scale, v_scale, dev):
    """The shape [n_blocks, Hk, block_size, d] of a cache, its tensors checked."""
    if k_cache.dim() != 4:
        raise ValueError("k_cache: expected [n_blocks, Hk, block_size, d]")
    shape = k_cache.shape
    _need("k_cache", k_cache, shape, torch.float8_e4m3fn, dev)
    _need("v_cache", v_cache, shape, torch.float8_e4m3fn, dev)
    _need("k_scale", k_scale, shape[:2], torch.float32, dev)
    _need("v_scale", v_scale, shape[:2], torch.float32, dev)
    return shape


def fa_cache_append(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """Puts the new tokens' keys and values (bf16 [T, Hk, d]; any token and head strides that are multiples of 8
    elements, those of a single token or head whatever they are, the last dimension contiguous) into their slots (int64
    [T]) of the cache: k_cache, v_cache float8_e4m3fn [n_blocks, Hk, block_size, d] and k_scale, v_scale fp32 [n_blocks,
    Hk], all in place."""
    dev = k.device
    n_blocks, H, bs, d = _check_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if slots.dim() != 1:
        raise ValueError("expected slots [T]")
    T = int(slots.shape[0])
    _need("slots", slots, (T,), torch.int64, dev)
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or tuple(t.shape) != (T, H, d) or not t.is_cuda or t.device != dev or \
                (T and t.stride(2) != 1):
            raise ValueError(f"{name}: expected a CUDA bfloat16 tensor of shape {(T, H, d)} on {dev}, contiguous in its last "
                             "dimension")
    _call(load_library().fa_cache_append, dev, k.data_ptr(), v.data_ptr(), slots.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), T, H, d, k.stride(0), k.stride(1), v.stride(0),
          v.stride(1), n_blocks, bs, _raw_stream(stream, dev))


@functools.lru_cache(maxsize=1024)
def fa_cache_fwd_workspace_size(B, Hq, Hk, N, d, block_size, max_blocks) -> int:
    return int(load_library().fa_cache_fwd_workspace_size(B, Hq, Hk, N, d, block_size, max_blocks))


def fa_cache_fwd(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, scale=None, o=None, lse=None, workspace=None,
                 stream=None):
    """Attention of each request's last N tokens, q bf16 [B,Hq,N,d], over its cached tokens: block_table int32
    [B, max_blocks], lens int32 [B] (the N tokens among them).  Returns (o bf16 [B,Hq,N,d], lse fp32 [B,Hq,N])."""
    if q.dim() != 4:
        raise ValueError("expected q [B, Hq, N, d]")
    B, Hq, N, d = q.shape
    dev = q.device
    _need("q", q, (B, Hq, N, d), torch.bfloat16, dev)
    n_blocks, Hk, bs, dc = _check_cache(k_cache, v_cache, k_scale, v_scale, dev)
    if dc != d or block_table.dim() != 2:
        raise ValueError(f"expected a cache of head size {d} and block_table [{B}, max_blocks]")
    max_blocks = int(block_table.shape[1])
    _need("block_table", block_table, (B, max_blocks), torch.int32, dev)
    _need("lens", lens, (B,), torch.int32, dev)
    o = _output("o", o, (B, Hq, N, d), torch.bfloat16, dev, stream)
    lse = _output("lse", lse, (B, Hq, N), torch.float32, dev, stream)
    lib = load_library()
    ws, ws_bytes = _check_workspace(workspace, fa_cache_fwd_workspace_size(B, Hq, Hk, N, d, bs, max_blocks), dev, stream)
    _call(lib.fa_cache_fwd, dev, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
          v_scale.data_ptr(), block_table.data_ptr(), lens.data_ptr(), o.data_ptr(), lse.data_ptr(), B, Hq, Hk, N, d,
          n_blocks, bs, max_blocks, _default_scale(d, scale), None if ws is None else ws.data_ptr(), ws_bytes,
          _raw_stream(stream, dev))
    return o, lse


def fa_check_status(stream=None):
    _check(load_library().fa_check_status(_stream(stream)))


def fa_kernel_launches() -> int:
    """Kernels libfa.so has launched in this process so far (a diagnostic; see include/fa.h)."""
    return int(load_library().fa_kernel_launches())


def fa_debug_time_bwd_main(start, stop) -> None:
    """Timing diagnostic: the next fa_bwd / fa_bwd_noalloc on this thread records the torch.cuda.Events
    `start` and `stop` (already recorded once, so that they exist) around its main kernel only."""
    load_library().fa_debug_time_bwd_main(ctypes.c_void_p(start.cuda_event), ctypes.c_void_p(stop.cuda_event))


def fa_test_force_wait_timeout(enable: bool) -> None:
    """Test switch of the failure path: while enabled, the tensor-core kernels withhold their Q loads and
    their bounded waits run out after ~10 ms (fa_check_status then raises FA_ERR_TIMEOUT).  Tests only."""
    load_library().fa_test_force_wait_timeout(1 if enable else 0)


def fa_last_error_string() -> str:
    return load_library().fa_last_error_string().decode(errors="replace")


__all__ = ["fa_fwd", "fa_fwd_stepnorm", "fa_fwd_f32", "fa_bwd", "fa_bwd_workspace_size", "fa_bwd_noalloc",
           "fa_cross_fwd", "fa_cross_fwd_workspace_size", "fa_cross_bwd", "fa_cross_bwd_workspace_size", "fa_cache_plan",
           "fa_cache_append", "fa_cache_fwd", "fa_cache_fwd_workspace_size", "fa_check_status", "fa_last_error_string",
           "fa_kernel_launches", "fa_test_force_wait_timeout", "fa_debug_time_bwd_main", "load_library", "FAError", "EXPORTS",
           "LIB_PATH"]
