"""Python binding of libattn (masked attention with LSE, LSE merge, paged KV
append, paged GQA decode) for one GB300 GPU.

This module only marshals arguments: it turns torch tensors into the C ABI's
pointer/shape/stride descriptors (``include/libattn.h``) and calls the shared
library through ctypes on the current CUDA stream.  Every step of the
computation runs in the library's CUDA kernels; torch supplies device memory
(outputs and workspaces the caller did not pass are allocated with it) and
the stream.  There is no CPU fallback: if the library is missing or a call
fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import math
import os
import struct
import threading
from typing import Optional, Sequence

import torch

from . import build as _build

__all__ = [
    "load", "LibAttnError", "Workspace",
    "attn_fwd", "attn_lse_merge", "kv_append", "paged_decode_attn", "paged_kv_gather",
    "attn_fwd_workspace_size", "paged_decode_workspace_size", "check_device_status",
    "rope_frequencies", "rope_apply", "rope_kv_append", "rope_kv_append_q8",
    "paged_tree_workspace_size", "paged_tree_attn", "kv_tree_accept",
    "paged_attn_weights_workspace_size", "paged_attn_weights", "kv_evict",
]

ATTN_F32, ATTN_BF16 = 0, 1
_STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA",
           4: "ATTN_ERR_TIMEOUT", 5: "ATTN_ERR_DEVICE_BOUNDS", 6: "ATTN_ERR_WORKSPACE"}


class LibAttnError(RuntimeError):
    def __init__(self, call: str, status: int):
        self.status = status
        super().__init__(f"{call}: {_STATUS.get(status, status)}")


class AttnTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


class AttnKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("block_size", ctypes.c_int32), ("num_blocks", ctypes.c_int64),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]


class AttnKVCacheQ8(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def _signatures() -> dict:
    """ctypes result and argument types of every libattn entry point."""
    P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    T = ctypes.POINTER(AttnTensor)
    C = ctypes.POINTER(AttnKVCache)
    CQ = ctypes.POINTER(AttnKVCacheQ8)
    return {
        "attn_version": (I32, []),
        "attn_status_string": (ctypes.c_char_p, [I32]),
        "attn_fwd_workspace_size": (SZ, []),
        "attn_fwd_workspace_size_for": (SZ, [I32, I32, I64, I32]),
        "kv_append_workspace_size": (SZ, []),
        "paged_decode_workspace_size": (SZ, [I32, I32, I32, I32, I32]),
        "attn_fwd": (I32, [T, T, T, P, I64, F, T, P, P, SZ, P]),
        "attn_fwd_varlen": (I32, [T, T, T, P, F, T, P, P, SZ, P]),
        "attn_key_padding_to_additive": (I32, [P, I64, I32, I64, P, I64, P]),
        "attn_lse_merge": (I32, [I32, T, ctypes.POINTER(P), T, P, P]),
        "kv_append": (I32, [C, P, I64, I32, P, T, T, P, SZ, P]),
        "paged_decode_attn": (I32, [T, C, P, I64, I32, P, F, T, P, P, SZ, P]),
        "paged_decode_attn_append": (I32, [T, T, T, C, P, I64, I32, P, F, T, P, P, SZ, P]),
        "paged_prefill_attn": (I32, [T, T, T, C, P, I64, I32, P, I32, F, T, P, P, SZ, P]),
        "kv_append_q8": (I32, [CQ, P, I64, I32, P, T, T, P, SZ, P]),
        "paged_decode_attn_q8": (I32, [T, CQ, P, I64, I32, P, F, T, P, P, SZ, P]),
        "paged_decode_attn_append_q8": (I32, [T, T, T, CQ, P, I64, I32, P, F, T, P, P, SZ, P]),
        "paged_kv_gather": (I32, [C, I32, P, I64, I32, P, I32, I64, P, P, SZ, P]),
        "paged_decode_attn_noalloc": (I32, [T, C, P, I64, I32, P, F, T, P, P, P]),
        "attn_rope_frequencies": (I32, [I32, ctypes.c_double, I32, ctypes.c_double, I64, ctypes.c_double,
                                        ctypes.c_double, P, ctypes.POINTER(F)]),
        "rope_apply": (I32, [P, P, I64, P, I32, I32, I32, F, P, P]),
        "rope_kv_append": (I32, [P, P, P, P, I64, P, I32, I32, F, P, P, P, I64, I32, P, P, SZ, P]),
        "rope_kv_append_q8": (I32, [P, P, P, P, I64, P, I32, I32, F, P, P, P, I64, I32, P, P, SZ, P]),
        "paged_tree_workspace_size": (SZ, [I32, I32, I32, I32, I32, I32, I32]),
        "paged_tree_attn": (I32, [P, P, P, P, P, I64, I32, P, P, I64, F, P, P, P, SZ, P]),
        "kv_tree_accept": (I32, [P, P, I64, I32, P, P, I64, I32, P, I32, P, SZ, P]),
        "paged_attn_weights_workspace_size": (SZ, [I32, I32, I32, I32]),
        "paged_attn_weights": (I32, [P, P, P, P, I64, I32, P, P, I32, F, P, P, SZ, P]),
        "kv_evict": (I32, [P, P, P, I64, I32, P, P, I64, I32, I32, I32, I32, I32, P, P, P, SZ, P]),
        "attn_check_device_status": (I32, [P, ctypes.POINTER(ctypes.c_uint32), P]),
        "attn_reset_device_status": (I32, [P, P]),
        "attn_selftest_wait_timeout": (I32, [P, SZ, ctypes.c_uint32, P]),
    }


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = False):
    """Load libattn.so (built in-tree by ``__graft_entry__.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"libattn is not built ({path} missing); run "
                                   "`python -c 'import __graft_entry__ as g; g.build()'`")
            _build.build()
        lib = ctypes.CDLL(path)
        sig = _signatures()
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def exported_symbols() -> list[str]:
    return ["attn_fwd", "attn_lse_merge", "kv_append", "paged_decode_attn", "paged_kv_gather",
            "attn_fwd_workspace_size", "kv_append_workspace_size", "paged_decode_workspace_size",
            "attn_check_device_status", "attn_reset_device_status", "attn_status_string", "attn_version",
            "paged_decode_attn_noalloc", "attn_selftest_wait_timeout", "attn_fwd_varlen",
            "attn_key_padding_to_additive", "paged_decode_attn_append", "paged_prefill_attn",
            "attn_fwd_workspace_size_for", "kv_append_q8", "paged_decode_attn_q8", "paged_decode_attn_append_q8",
            "attn_rope_frequencies", "rope_apply", "rope_kv_append", "rope_kv_append_q8",
            "paged_tree_workspace_size", "paged_tree_attn", "kv_tree_accept",
            "paged_attn_weights_workspace_size", "paged_attn_weights", "kv_evict"]


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------
_DTYPE_CODES = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}


def _dtype_code(t: torch.Tensor) -> int:
    code = _DTYPE_CODES.get(t.dtype)
    if code is None:
        raise TypeError(f"libattn takes bfloat16 or float32 tensors, got {t.dtype}")
    return code


# An AttnTensor's bytes in one step: a call of a few microseconds on the GPU is
# bound by the host, and setting the structure's fields one by one costs about
# as much as the launch.
_pack_tensor = struct.Struct("@Pii8q").pack
_pack_by_dim = tuple(struct.Struct(f"@Pii{n}q{32 - 8 * n}x{n}q{32 - 8 * n}x").pack for n in range(5))
_pack_cache = struct.Struct("@PPiiqii").pack  # an AttnKVCache
_NO_DIMS = ((0, 0, 0, 0), (0, 0, 0), (0, 0), (0,), ())  # by number of dimensions used


def _desc(t: torch.Tensor) -> AttnTensor:
    if not _on_device(t):
        raise ValueError("libattn tensors must be on a CUDA device")
    n = t.dim()
    if n > 4:
        raise ValueError(f"libattn tensors have up to 4 dimensions, got {n}")
    rest = _NO_DIMS[n]
    return AttnTensor.from_buffer_copy(_pack_tensor(t.data_ptr(), _dtype_code(t), n, *t.shape, *rest, *t.stride(),
                                                    *rest))


# The current stream's handle without a Stream object around it (which costs ten
# times as much), where torch has the call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _tensor_bytes(t: torch.Tensor) -> bytes:
    """An AttnTensor as bytes, for entry points declared with a plain pointer."""
    if not _on_device(t):
        raise ValueError("libattn tensors must be on a CUDA device")
    n = t.dim()
    if n > 4:
        raise ValueError(f"libattn tensors have up to 4 dimensions, got {n}")
    return _pack_by_dim[n](t.data_ptr(), _dtype_code(t), n, *t.shape, *t.stride())


def _cache_bytes(k_cache: torch.Tensor, v_cache: torch.Tensor) -> bytes:
    """The AttnKVCache of two cache tensors, as bytes."""
    if not (k_cache.dim() == 4 and k_cache.shape == v_cache.shape and k_cache.dtype == v_cache.dtype):
        raise ValueError("K and V caches must be [num_blocks, Hkv, block_size, D] of one dtype")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError("K and V caches must be contiguous")
    if not (_on_device(k_cache) and _on_device(v_cache)):
        raise ValueError("K and V caches must be on a CUDA device")
    nb, heads, bs, D = k_cache.shape
    return _pack_cache(k_cache.data_ptr(), v_cache.data_ptr(), _dtype_code(k_cache), bs, nb, heads, D)


_marshal = None      # the compiled caller (marshal.cpp), or None
_marshal_tried = False
_entries: dict = {}  # C entry points' addresses


def _call(name: str, fmt: str, *args) -> bool:
    """The C entry point, its arguments checked and converted in one step; False
    (and nothing called) where they are not plainly as documented: the caller
    then takes them one by one, with every check worded."""
    global _marshal, _marshal_tried
    if not _marshal_tried:
        _marshal_tried = True
        path = _build.marshal_path()
        if os.path.exists(path):
            loader = importlib.machinery.ExtensionFileLoader("_marshal", path)
            try:
                _marshal = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
            except ImportError:  # a library that it was linked to is not there: the checks serve
                pass
    if _marshal is None:
        return False
    entry = _entries.get(name)
    if entry is None:
        entry = _entries[name] = ctypes.cast(getattr(load(), name), ctypes.c_void_p).value
    st = _marshal.call(entry, name, fmt, *args)
    if st is None:
        return False
    if st != 0:
        raise LibAttnError(name, st)
    return True


def _handle(stream):
    """A stream argument as a raw handle; None stays None."""
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _fresh(make, stream, device):
    """make(), its memory of the stream that the call runs on: what a call
    allocates must neither wait for nor be reused on the current stream when
    another one was passed."""
    if stream is None or device.type != "cuda":
        return make()
    if not isinstance(stream, torch.cuda.Stream):
        # (of the handle 0, the default stream, an ExternalStream would be a new one)
        stream = int(stream)
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return make()


def _check(name: str, st: int):
    if st != 0:
        raise LibAttnError(name, st)


# Arguments that reach the library as bare pointers (LSE buffers, masks,
# block tables, per-sequence positions and lengths) carry no shape the C side
# could check, so their dtype, layout and size are checked here, with real
# exceptions rather than asserts (which `python -O` would drop, leaving a
# kernel to read or write past a short buffer), and their device when the
# pointer is taken.
def _require(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _on_device(t: torch.Tensor) -> bool:
    """Whether t lives where the library's kernels can read it."""
    return t.is_cuda


def _ptr(t: Optional[torch.Tensor], name: str = "tensor"):
    """Device pointer of t (None passes through as NULL)."""
    if t is None:
        return None
    if not _on_device(t):
        raise ValueError(f"{name} must be on a CUDA device")
    return t.data_ptr()


# The checks of every call test their conditions first and word the refusal
# after: the wording costs more than the check.
def _check_f32_buffer(t: torch.Tensor, numel: int, name: str):
    """float32, contiguous, exactly `numel` elements."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float32 and t.is_contiguous() and t.numel() == numel:
        return
    _require(isinstance(t, torch.Tensor), f"{name} must be a torch tensor")
    _require(t.dtype == torch.float32, f"{name} must be float32, got {t.dtype}")
    _require(t.is_contiguous(), f"{name} must be contiguous")
    _require(t.numel() == numel, f"{name} must hold {numel} elements, got {t.numel()}")


def _check_int32_vec(t: torch.Tensor, n: int, name: str):
    """int32 [n], contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.shape == (n,) and t.is_contiguous():
        return
    _require(isinstance(t, torch.Tensor), f"{name} must be a torch tensor")
    _require(t.dtype == torch.int32, f"{name} must be int32, got {t.dtype}")
    _require(t.dim() == 1 and t.shape[0] == n and t.is_contiguous(), f"{name} must be contiguous [{n}], got "
             f"{tuple(t.shape)}")


def _check_block_table(t: torch.Tensor, batch: int):
    """int32 [>= batch, max_blocks] with unit stride along a row."""
    if (isinstance(t, torch.Tensor) and t.dtype == torch.int32 and t.dim() == 2 and t.shape[0] >= batch
            and t.stride(1) == 1 and t.stride(0) >= t.shape[1]):
        return
    _require(isinstance(t, torch.Tensor), "block_table must be a torch tensor")
    _require(t.dtype == torch.int32, f"block_table must be int32, got {t.dtype}")
    _require(t.dim() == 2 and t.shape[0] >= batch and t.stride(1) == 1 and t.stride(0) >= t.shape[1],
             f"block_table must be [>= {batch}, max_blocks] with contiguous rows, got {tuple(t.shape)} "
             f"strides {tuple(t.stride())}")


class Workspace:
    """A zero-initialised device buffer for the library's workspace argument
    (its first word is the sticky device status)."""

    def __init__(self, nbytes: int, device=None):
        nbytes = max(256, (int(nbytes) + 255) // 256 * 256)
        self.tensor = torch.zeros(nbytes, dtype=torch.uint8, device=device or "cuda")
        self.nbytes = nbytes

    @property
    def ptr(self) -> int:
        return self.tensor.data_ptr()

    def status(self, stream=None) -> int:
        return check_device_status(self, stream)

    def reset(self, stream=None):
        _check("attn_reset_device_status", load().attn_reset_device_status(self.ptr, _stream(stream)))


_default_ws: dict = {}


def _default(key, nbytes: int, device, stream) -> Workspace:
    """A workspace for the calls on a device that pass none, made at the first of
    them and kept under `key`.  Its zeroes are in place before any call uses it,
    on whichever stream.  A call that is captured into a graph before there is
    one gets a workspace of its own, which is not kept: its clearing is part of
    the graph, and each replay would wipe the status of every other call."""
    device = torch.device(device)

    def make():
        ws = Workspace(nbytes, device=device)
        if device.type == "cuda":
            if torch.cuda.is_current_stream_capturing():
                return ws
            torch.cuda.current_stream(device).synchronize()
        with _lock:  # of two threads that come here at once, one's is kept and both use it
            kept = _default_ws.get(key)
            if kept is None or kept.nbytes < nbytes:
                kept = _default_ws[key] = ws
        return kept

    return _fresh(make, stream, device)


def _small_ws(device, stream=None) -> Workspace:
    """The default workspace of the calls that need the status word alone."""
    key = torch.device(device).index
    ws = _default_ws.get(key)
    return _default(key, 256, device, stream) if ws is None else ws


def _attn_ws(q: torch.Tensor, k: torch.Tensor, stream=None) -> Workspace:
    """Default attn_fwd workspace: the status word plus room for the per-tile
    key bounds and the last-wave partials of this shape (kept per device,
    grown when a call needs more).  It is shared by every call on the device
    that passes no workspace, so calls that may run concurrently (on
    different streams) must each pass their own."""
    need = attn_fwd_workspace_size_for(k.shape[0], k.shape[1], k.shape[2], k.shape[3])
    key = ("attn", torch.device(q.device).index)
    ws = _default_ws.get(key)
    if ws is None or ws.nbytes < need:
        ws = _default(key, max(need, 256), q.device, stream)
    return ws


def _ws_ptr(ws: Workspace):
    return _ptr(ws.tensor, "workspace")


def _ws_tensor(workspace: Optional[Workspace]):
    return workspace.tensor if workspace is not None else None


def check_device_status(ws: Workspace, stream=None) -> int:
    raw = ctypes.c_uint32(0)
    st = load().attn_check_device_status(ws.ptr, ctypes.byref(raw), _stream(stream))
    return int(st)


def attn_fwd_workspace_size() -> int:
    return int(load().attn_fwd_workspace_size())


def attn_fwd_workspace_size_for(batch: int, kv_heads: int, num_keys: int, head_dim: int) -> int:
    return int(load().attn_fwd_workspace_size_for(batch, kv_heads, num_keys, head_dim))


def paged_decode_workspace_size(batch: int, num_q_heads: int, max_blocks: int, block_size: int = 16,
                                head_dim: int = 128) -> int:
    return int(load().paged_decode_workspace_size(batch, num_q_heads, max_blocks, block_size, head_dim))


# --------------------------------------------------------------------------
# the four calls
# --------------------------------------------------------------------------
def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, key_pad_mask: Optional[torch.Tensor] = None,
             scale: Optional[float] = None, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
             return_lse: bool = True, workspace: Optional[Workspace] = None, stream=None):
    """Masked exact attention; q [B, Hq, Pq, D], k/v [B, Hkv, Pk, D] (any
    strides with a contiguous last dim, e.g. packed [T, H, D] permuted to
    [1, H, T, D]).  key_pad_mask: float32 [B, Pk] additive (0 / -inf).
    Returns (out, lse) with lse float32 [B, Hq, Pq] (or out alone)."""
    lib = load()
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty(q.shape[:3], dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, q.shape[0] * q.shape[1] * q.shape[2], "lse")
    mptr, mstride = None, 0
    if key_pad_mask is not None:
        m = key_pad_mask
        _require(m.dtype == torch.float32, f"key_pad_mask must be float32 (additive), got {m.dtype}")
        _require(m.dim() == 2 and tuple(m.shape) == (q.shape[0], k.shape[2]) and m.stride(1) == 1,
                 f"key_pad_mask must be [{q.shape[0]}, {k.shape[2]}] with contiguous rows, got {tuple(m.shape)}")
        mptr, mstride = _ptr(m, "key_pad_mask"), m.stride(0)
    ws = workspace or _attn_ws(q, k, stream)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    st = lib.attn_fwd(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), mptr, mstride, float(scale),
                      ctypes.byref(do), _ptr(lse, "lse"), _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("attn_fwd", st)
    return (out, lse) if return_lse else out


def attn_fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, key_lens: torch.Tensor,
                    scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None, return_lse: bool = True,
                    workspace: Optional[Workspace] = None, stream=None):
    """attn_fwd where batch row b attends to its first key_lens[b] keys (int32
    [B] on the device); KV tiles past the length are skipped."""
    lib = load()
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    _check_int32_vec(key_lens, q.shape[0], "key_lens")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty(q.shape[:3], dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, q.shape[0] * q.shape[1] * q.shape[2], "lse")
    ws = workspace or _attn_ws(q, k, stream)
    dq, dk, dv, do = _desc(q), _desc(k), _desc(v), _desc(out)
    st = lib.attn_fwd_varlen(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), _ptr(key_lens, "key_lens"),
                             float(scale), ctypes.byref(do), _ptr(lse, "lse"), _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("attn_fwd_varlen", st)
    return (out, lse) if return_lse else out


def key_padding_to_additive(key_padding_mask: torch.Tensor, out: Optional[torch.Tensor] = None,
                            stream=None) -> torch.Tensor:
    """Boolean [B, Pk] key_padding_mask (True = padded key, the
    nn.MultiheadAttention convention) -> float32 additive mask (-inf / 0)."""
    lib = load()
    kpm = key_padding_mask
    _require(kpm.dim() == 2 and kpm.stride(1) == 1, "key_padding_mask must be [B, Pk] with contiguous rows")
    if kpm.dtype == torch.bool:
        kpm = kpm.view(torch.uint8)
    _require(kpm.dtype == torch.uint8, f"key_padding_mask must be bool or uint8, got {kpm.dtype}")
    B, Pk = kpm.shape
    if out is None:
        out = _fresh(lambda: torch.empty(B, Pk, dtype=torch.float32, device=kpm.device), stream, kpm.device)
    _require(out.dtype == torch.float32 and out.dim() == 2 and tuple(out.shape) == (B, Pk) and out.stride(1) == 1,
             f"out must be float32 [{B}, {Pk}] with contiguous rows")
    st = lib.attn_key_padding_to_additive(_ptr(kpm, "key_padding_mask"), kpm.stride(0), B, Pk, _ptr(out, "out"),
                                          out.stride(0), _stream(stream))
    _check("attn_key_padding_to_additive", st)
    return out


def attn_lse_merge(outs: Sequence[torch.Tensor], lses: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, stream=None):
    """Merge chunk results: lse = log sum_i exp(lse_i), out = sum_i exp(lse_i - lse) out_i."""
    lib = load()
    n = len(outs)
    _require(n >= 1 and len(lses) == n, f"attn_lse_merge takes n >= 1 outputs and as many LSEs ({n}, {len(lses)})")
    if out is None:
        out = _fresh(lambda: torch.empty(outs[0].shape, dtype=outs[0].dtype, device=outs[0].device),
                     stream, outs[0].device)
    rows = outs[0].shape[0] * outs[0].shape[1] * outs[0].shape[2]  # B * H * P
    if lse is None:
        lse = _fresh(lambda: torch.empty(lses[0].shape, dtype=torch.float32, device=outs[0].device),
                     stream, outs[0].device)
    _check_f32_buffer(lse, rows, "lse")
    for i, l in enumerate(lses):
        _check_f32_buffer(l, rows, f"lses[{i}]")
    arr = (AttnTensor * n)(*[_desc(o) for o in outs])
    lptrs = (ctypes.c_void_p * n)(*[_ptr(l, f"lses[{i}]") for i, l in enumerate(lses)])
    do = _desc(out)
    st = lib.attn_lse_merge(n, arr, lptrs, ctypes.byref(do), _ptr(lse, "lse"), _stream(stream))
    _check("attn_lse_merge", st)
    return out, lse


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor) -> AttnKVCache:
    return AttnKVCache.from_buffer_copy(_cache_bytes(k_cache, v_cache))


def kv_append(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, pos: torch.Tensor,
              k_new: torch.Tensor, v_new: torch.Tensor, workspace: Optional[Workspace] = None, stream=None):
    """Write k_new/v_new [B, Hkv, D] at token position pos[b] of each
    sequence's paged cache (caches [num_blocks, Hkv, block_size, D])."""
    lib = load()
    _check_block_table(block_table, k_new.shape[0])
    _check_int32_vec(pos, k_new.shape[0], "pos")
    ws = workspace or _small_ws(k_cache.device, stream)
    c = _cache(k_cache, v_cache)
    dk, dv = _desc(k_new), _desc(v_new)
    st = lib.kv_append(ctypes.byref(c), _ptr(block_table, "block_table"), block_table.stride(0),
                       block_table.shape[1], _ptr(pos, "pos"), ctypes.byref(dk), ctypes.byref(dv), _ws_ptr(ws),
                       ws.nbytes, _stream(stream))
    _check("kv_append", st)


def paged_decode_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                      ctx_lens: torch.Tensor, scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                      lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                      workspace: Optional[Workspace] = None, stream=None):
    """One query token per sequence, q [B, Hq, D], over the paged cache;
    ctx_lens int32 [B] counts the attended tokens (the appended one included)."""
    lib = load()
    B, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq), dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, B * Hq, "lse")
    max_blocks = block_table.shape[1]
    need = paged_decode_workspace_size(B, Hq, max_blocks, k_cache.shape[2], D)
    ws = workspace
    if ws is None or ws.nbytes < need:
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    c = _cache(k_cache, v_cache)
    dq, do = _desc(q), _desc(out)
    st = lib.paged_decode_attn(ctypes.byref(dq), ctypes.byref(c), _ptr(block_table, "block_table"),
                               block_table.stride(0), max_blocks, _ptr(ctx_lens, "ctx_lens"), float(scale),
                               ctypes.byref(do), _ptr(lse, "lse"),
                               _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("paged_decode_attn", st)
    return (out, lse) if return_lse else out


def paged_decode_attn_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor,
                             v_cache: torch.Tensor, block_table: torch.Tensor, pos: torch.Tensor,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                             workspace: Optional[Workspace] = None, stream=None):
    """kv_append(pos, k_new, v_new) and the decode over tokens [0, pos[b]] in
    one launch; k_new, v_new [B, Hkv, D], pos int32 [B]."""
    lib = load()
    B, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_block_table(block_table, B)
    _check_int32_vec(pos, B, "pos")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq), dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, B * Hq, "lse")
    max_blocks = block_table.shape[1]
    need = paged_decode_workspace_size(B, Hq, max_blocks, k_cache.shape[2], D)
    ws = workspace
    if ws is None or ws.nbytes < need:
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    c = _cache(k_cache, v_cache)
    dq, dk, dv, do = _desc(q), _desc(k_new), _desc(v_new), _desc(out)
    st = lib.paged_decode_attn_append(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), ctypes.byref(c),
                                      _ptr(block_table, "block_table"), block_table.stride(0), max_blocks,
                                      _ptr(pos, "pos"), float(scale), ctypes.byref(do), _ptr(lse, "lse"), _ws_ptr(ws),
                                      ws.nbytes,
                                      _stream(stream))
    _check("paged_decode_attn_append", st)
    return (out, lse) if return_lse else out


def paged_prefill_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                       start_pos: torch.Tensor, k_new: Optional[torch.Tensor] = None,
                       v_new: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       return_lse: bool = False, workspace: Optional[Workspace] = None, stream=None):
    """A chunk of T tokens per sequence: q [B, Hq, T, D] at positions
    start_pos[b] + i.  With k_new / v_new ([B, Hkv, T, D]) their K/V are
    first written to the cache; queries then attend over the cache through
    the block table (causal: up to their own position)."""
    lib = load()
    B, Hq, T, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_block_table(block_table, B)
    _check_int32_vec(start_pos, B, "start_pos")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq, T), dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, B * Hq * T, "lse")
    ws = workspace or _small_ws(q.device, stream)
    c = _cache(k_cache, v_cache)
    dq, do = _desc(q), _desc(out)
    dk = ctypes.byref(_desc(k_new)) if k_new is not None else None
    dv = ctypes.byref(_desc(v_new)) if v_new is not None else None
    st = lib.paged_prefill_attn(ctypes.byref(dq), dk, dv, ctypes.byref(c), _ptr(block_table, "block_table"),
                                block_table.stride(0), block_table.shape[1], _ptr(start_pos, "start_pos"),
                                int(bool(causal)), float(scale), ctypes.byref(do), _ptr(lse, "lse"), _ws_ptr(ws),
                                ws.nbytes, _stream(stream))
    _check("paged_prefill_attn", st)
    return (out, lse) if return_lse else out


def _cache_q8(kq: torch.Tensor, vq: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> AttnKVCacheQ8:
    _require(kq.dtype == torch.int8 and vq.dtype == torch.int8, "INT8 caches must be int8")
    _require(kq.dim() == 4 and kq.shape == vq.shape, "INT8 caches must be [num_blocks, Hkv, block_size, D], "
             "K and V alike")
    _require(k_scale.dtype == torch.float32 and v_scale.dtype == torch.float32, "INT8 row scales must be float32")
    _require(tuple(k_scale.shape) == tuple(kq.shape[:3]) and tuple(v_scale.shape) == tuple(kq.shape[:3]),
             f"INT8 row scales must be {tuple(kq.shape[:3])}")
    for t in (kq, vq, k_scale, v_scale):
        _require(t.is_contiguous() and _on_device(t), "INT8 caches and scales must be contiguous CUDA tensors")
    c = AttnKVCacheQ8()
    c.k, c.v, c.k_scale, c.v_scale = kq.data_ptr(), vq.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr()
    c.num_blocks, c.num_kv_heads, c.block_size, c.head_dim = kq.shape
    c.reserved = 0
    return c


def kv_append_q8(kq_cache: torch.Tensor, vq_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                 block_table: torch.Tensor, pos: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                 workspace: Optional[Workspace] = None, stream=None):
    """Quantise each sequence's new K/V rows (bf16 [B, Hkv, D]) to INT8 codes
    with one float32 scale per row and write them at pos[b]."""
    lib = load()
    _check_block_table(block_table, k_new.shape[0])
    _check_int32_vec(pos, k_new.shape[0], "pos")
    ws = workspace or _small_ws(kq_cache.device, stream)
    c = _cache_q8(kq_cache, vq_cache, k_scale, v_scale)
    dk, dv = _desc(k_new), _desc(v_new)
    st = lib.kv_append_q8(ctypes.byref(c), _ptr(block_table, "block_table"), block_table.stride(0),
                          block_table.shape[1], _ptr(pos, "pos"), ctypes.byref(dk), ctypes.byref(dv), _ws_ptr(ws),
                          ws.nbytes, _stream(stream))
    _check("kv_append_q8", st)


def paged_decode_attn_q8(q: torch.Tensor, kq_cache: torch.Tensor, vq_cache: torch.Tensor, k_scale: torch.Tensor,
                         v_scale: torch.Tensor, block_table: torch.Tensor, ctx_lens: torch.Tensor,
                         scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                         workspace: Optional[Workspace] = None, stream=None):
    """paged_decode_attn over an INT8 cache (codes int8 [N, Hkv, 16, D],
    scales float32 [N, Hkv, 16])."""
    lib = load()
    B, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq), dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, B * Hq, "lse")
    max_blocks = block_table.shape[1]
    need = paged_decode_workspace_size(B, Hq, max_blocks, kq_cache.shape[2], D)
    ws = workspace
    if ws is None or ws.nbytes < need:
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    c = _cache_q8(kq_cache, vq_cache, k_scale, v_scale)
    dq, do = _desc(q), _desc(out)
    st = lib.paged_decode_attn_q8(ctypes.byref(dq), ctypes.byref(c), _ptr(block_table, "block_table"),
                                  block_table.stride(0), max_blocks, _ptr(ctx_lens, "ctx_lens"), float(scale),
                                  ctypes.byref(do), _ptr(lse, "lse"),
                                  _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("paged_decode_attn_q8", st)
    return (out, lse) if return_lse else out


def paged_decode_attn_append_q8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, kq_cache: torch.Tensor,
                                vq_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor,
                                block_table: torch.Tensor, pos: torch.Tensor, scale: Optional[float] = None,
                                out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                                return_lse: bool = False, workspace: Optional[Workspace] = None, stream=None):
    """kv_append_q8(pos, k_new, v_new) and paged_decode_attn_q8 over tokens
    [0, pos[b]] in one call; k_new, v_new bf16 [B, Hkv, D], pos int32 [B]."""
    lib = load()
    B, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_block_table(block_table, B)
    _check_int32_vec(pos, B, "pos")
    if out is None:
        out = _fresh(lambda: torch.empty(q.shape, dtype=q.dtype, device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq), dtype=torch.float32, device=q.device), stream, q.device)
    if lse is not None:
        _check_f32_buffer(lse, B * Hq, "lse")
    max_blocks = block_table.shape[1]
    need = paged_decode_workspace_size(B, Hq, max_blocks, kq_cache.shape[2], D)
    ws = workspace
    if ws is None or ws.nbytes < need:
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    c = _cache_q8(kq_cache, vq_cache, k_scale, v_scale)
    dq, dk, dv, do = _desc(q), _desc(k_new), _desc(v_new), _desc(out)
    st = lib.paged_decode_attn_append_q8(ctypes.byref(dq), ctypes.byref(dk), ctypes.byref(dv), ctypes.byref(c),
                                         _ptr(block_table, "block_table"), block_table.stride(0), max_blocks,
                                         _ptr(pos, "pos"), float(scale), ctypes.byref(do), _ptr(lse, "lse"),
                                         _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("paged_decode_attn_append_q8", st)
    return (out, lse) if return_lse else out


def paged_kv_gather(cache: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor, max_len: int,
                    out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None,
                    stream=None) -> torch.Tensor:
    """Contiguous copy [B, Hkv, max_len, D] of the first lens[b] tokens of each
    sequence in one paged cache tensor (K or V); rows past lens[b] untouched."""
    lib = load()
    B = lens.shape[0]
    nb, Hkv, bs, D = cache.shape
    _check_int32_vec(lens, B, "lens")
    _check_block_table(block_table, B)
    if out is None:
        out = _fresh(lambda: torch.zeros((B, Hkv, max_len, D), dtype=cache.dtype, device=cache.device),
                     stream, cache.device)
    _require(out.dtype == cache.dtype and tuple(out.shape) == (B, Hkv, max_len, D) and out.is_contiguous(),
             f"out must be contiguous {cache.dtype} [{B}, {Hkv}, {max_len}, {D}]")
    c = _cache(cache, cache)
    ws = workspace or _small_ws(cache.device, stream)
    st = lib.paged_kv_gather(ctypes.byref(c), 0, _ptr(block_table, "block_table"), block_table.stride(0),
                             block_table.shape[1], _ptr(lens, "lens"), B, max_len, _ptr(out, "out"), _ws_ptr(ws),
                             ws.nbytes, _stream(stream))
    _check("paged_kv_gather", st)
    return out


def paged_decode_attn_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                              block_table: torch.Tensor, ctx_lens: torch.Tensor, scale: Optional[float] = None,
                              out: torch.Tensor = None, lse: Optional[torch.Tensor] = None,
                              device_status: Optional[torch.Tensor] = None, stream=None):
    """paged_decode_attn for callers that cannot allocate device memory: the
    split-K scratch is the library's built-in 20 MiB array, so `out` (and
    `lse`, `device_status` if wanted) must be passed in.  Calls that overlap on
    the GPU race on the shared scratch."""
    lib = load()
    B, Hq, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _require(out is not None, "the no-alloc call writes into a caller buffer: pass out")
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    if lse is not None:
        _check_f32_buffer(lse, B * Hq, "lse")
    if device_status is not None:
        _require(device_status.dtype in (torch.int32, torch.uint32) and device_status.numel() >= 1,
                 "device_status must be a 32-bit word")
    c = _cache(k_cache, v_cache)
    dq, do = _desc(q), _desc(out)
    st = lib.paged_decode_attn_noalloc(ctypes.byref(dq), ctypes.byref(c), _ptr(block_table, "block_table"),
                                       block_table.stride(0), block_table.shape[1], _ptr(ctx_lens, "ctx_lens"),
                                       float(scale), ctypes.byref(do), _ptr(lse, "lse"),
                                       _ptr(device_status, "device_status"),
                                       _stream(stream))
    _check("paged_decode_attn_noalloc", st)
    return out


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
_ROPE_SCALING = {"plain": 0, "linear": 1, "base": 2, "banded": 3, "ramp": 4}


def rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0,
                     original_len: int = 0, low: float = 1.0, high: Optional[float] = None, device=None):
    """Frequencies for the rope calls: (freqs, magnitude) with freqs int64
    [rotary_dim / 2] on the device, each pair's turns a token as a 64-bit
    fraction.  scaling: "plain", "linear" (positions / factor), "base" (a larger
    base), "banded" or "ramp" (slow pairs interpolated, fast ones kept; low and
    high in turns over original_len tokens; high is 4 for "banded" and 32 for
    "ramp" unless given, the values that models of either kind are trained with)."""
    _require(scaling in _ROPE_SCALING, f"scaling must be one of {sorted(_ROPE_SCALING)}, got {scaling!r}")
    if high is None:
        high = 32.0 if scaling == "ramp" else 4.0
    turns = torch.empty(max(0, int(rotary_dim) // 2), dtype=torch.int64)
    magnitude = ctypes.c_float(1.0)
    st = load().attn_rope_frequencies(int(rotary_dim), float(base), _ROPE_SCALING[scaling], float(factor),
                                      int(original_len), float(low), float(high), turns.data_ptr() or None,
                                      ctypes.byref(magnitude))
    _check("attn_rope_frequencies", st)
    return turns.to(device or "cuda"), float(magnitude.value)


def _check_devices(name: str, *tensors: Optional[torch.Tensor]):
    """The kernels run on the current device: a tensor of another one is refused."""
    current = -1
    for t in tensors:
        if t is not None:
            device = t.get_device()  # -1 on the CPU: refused where its pointer is taken
            if device != current and device >= 0:
                if current < 0:
                    current = torch.cuda.current_device()
                if device != current:
                    raise ValueError(f"{name} runs on the current device cuda:{current}, got a tensor on {t.device}")


def _check_rope(positions: torch.Tensor, freqs: torch.Tensor, B: int, T: int, D: int):
    if not (isinstance(positions, torch.Tensor) and positions.dtype == torch.int32):
        raise ValueError("positions must be int32")
    if positions.shape != (B, T) or not (T <= 1 or positions.stride(1) == 1):
        raise ValueError(f"positions must be [{B}, {T}] with contiguous rows, got {tuple(positions.shape)}")
    if not (isinstance(freqs, torch.Tensor) and freqs.dtype == torch.int64 and freqs.dim() == 1
            and freqs.is_contiguous()):
        raise ValueError("freqs must be contiguous int64 [rotary_dim / 2]")
    if not 1 <= freqs.shape[0] <= D // 2:
        raise ValueError(f"freqs must hold 1 to {D // 2} pairs, got {freqs.shape[0]}")


def _one_token(*tensors: torch.Tensor):
    """[B, H, D] rows as [B, H, 1, D] views."""
    _require(all(t.dim() == 3 for t in tensors), "rows without a token dimension must all be [B, H, D]")
    return tuple(t.unsqueeze(2) for t in tensors)


def rope_apply(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, interleaved: bool = False,
               inverse: bool = False, magnitude: float = 1.0, out: Optional[torch.Tensor] = None, stream=None):
    """Rotate x [B, H, T, D] (bf16 or f32, any strides with a contiguous last
    dim) by its tokens' positions (int32 [B, T]), the first 2 * len(freqs) dims
    of each row in neighbouring pairs (interleaved) or pairs half the rotated
    dims apart.  x [B, H, D] with positions [B] is one token a row.  inverse:
    the transposed rotation, which is its gradient.  out may be x."""
    lib = load()
    if out is None:
        out = _fresh(lambda: torch.empty_like(x), stream, x.device)
    elif not (out.dtype == x.dtype and out.shape == x.shape):
        raise ValueError(f"out must be {x.dtype} {tuple(x.shape)}")
    if x.is_cuda:
        if _call("rope_apply", "yRf===YS", x, positions, freqs, int(bool(interleaved)), int(bool(inverse)),
                 float(magnitude), out, _handle(stream)):
            return out
    full = out
    if x.dim() == 3:
        x, full = _one_token(x, out)
        positions = positions.unsqueeze(-1)
    if x.dim() != 4:
        raise ValueError(f"x must be [B, H, T, D] or [B, H, D], got {tuple(x.shape)}")
    B, H, T, D = x.shape
    _check_rope(positions, freqs, B, T, D)
    _check_devices("rope_apply", x, positions, freqs, out)
    st = lib.rope_apply(_tensor_bytes(x), _ptr(positions, "positions"), positions.stride(0), _ptr(freqs, "freqs"),
                        2 * freqs.shape[0], int(bool(interleaved)), int(bool(inverse)), float(magnitude),
                        _tensor_bytes(full), _stream(stream))
    _check("rope_apply", st)
    return out


def _rope_append(name, cache, caches, q, k_new, v_new, positions, freqs, block_table, start_pos, interleaved, magnitude,
                 q_out, workspace, stream):
    lib = load()
    if q_out is None:
        q_out = _fresh(lambda: torch.empty_like(q), stream, q.device)
    elif not (q_out.dtype == q.dtype and q_out.shape == q.shape):
        raise ValueError(f"q_out must be {q.dtype} {tuple(q.shape)}")
    full = q_out
    if q.dim() == 3:
        q, k_new, v_new, full = _one_token(q, k_new, v_new, q_out)
        positions = positions.unsqueeze(-1)
    if q.dim() != 4:
        raise ValueError(f"q must be [B, Hq, T, D] or [B, Hq, D], got {tuple(q.shape)}")
    B, Hq, T, D = q.shape
    _check_rope(positions, freqs, B, T, D)
    _check_block_table(block_table, B)
    _check_int32_vec(start_pos, B, "start_pos")
    _check_devices(name, q, k_new, v_new, positions, freqs, block_table, start_pos, q_out, *caches,
                   _ws_tensor(workspace))
    ws = workspace or _small_ws(caches[0].device, stream)
    _require(k_new.dim() == 4 and v_new.dim() == 4, "k_new and v_new must have q's number of dimensions")
    st = getattr(lib, name)(_tensor_bytes(q), _tensor_bytes(k_new), _tensor_bytes(v_new), _ptr(positions, "positions"),
                            positions.stride(0), _ptr(freqs, "freqs"), 2 * freqs.shape[0], int(bool(interleaved)),
                            float(magnitude), _tensor_bytes(full), cache, _ptr(block_table, "block_table"),
                            block_table.stride(0), block_table.shape[1], _ptr(start_pos, "start_pos"), _ws_ptr(ws),
                            ws.nbytes, _stream(stream))
    _check(name, st)
    return q_out


def rope_kv_append(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                   freqs: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   start_pos: torch.Tensor, interleaved: bool = False, magnitude: float = 1.0,
                   q_out: Optional[torch.Tensor] = None, workspace: Optional[Workspace] = None, stream=None):
    """Rotate q [B, Hq, T, D] and k_new [B, Hkv, T, D] by positions (int32
    [B, T]), and write the rotated keys and v_new to cache slots start_pos[b] +
    i.  Without the T dimension (and positions [B]): one token a sequence.
    Returns the rotated q (q_out may be q)."""
    if q_out is None:
        q_out = _fresh(lambda: torch.empty_like(q), stream, q.device)
    if k_cache.is_cuda:
        ws = workspace or _small_ws(k_cache.device, stream)
        if _call("rope_kv_append", "yyyRf==YcbvWS", q, k_new, v_new, positions, freqs, int(bool(interleaved)),
                 float(magnitude), q_out, k_cache, v_cache, block_table, start_pos, ws.tensor, _handle(stream)):
            return q_out
    return _rope_append("rope_kv_append", _cache_bytes(k_cache, v_cache), (k_cache, v_cache), q, k_new, v_new,
                        positions, freqs, block_table, start_pos, interleaved, magnitude, q_out, workspace, stream)


def rope_kv_append_q8(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, positions: torch.Tensor,
                      freqs: torch.Tensor, kq_cache: torch.Tensor, vq_cache: torch.Tensor, k_scale: torch.Tensor,
                      v_scale: torch.Tensor, block_table: torch.Tensor, start_pos: torch.Tensor,
                      interleaved: bool = False, magnitude: float = 1.0, q_out: Optional[torch.Tensor] = None,
                      workspace: Optional[Workspace] = None, stream=None):
    """rope_kv_append into an INT8 cache (codes int8 [N, Hkv, 16, D], scales
    float32 [N, Hkv, 16])."""
    return _rope_append("rope_kv_append_q8", bytes(_cache_q8(kq_cache, vq_cache, k_scale, v_scale)),
                        (kq_cache, vq_cache, k_scale, v_scale), q, k_new, v_new, positions, freqs, block_table,
                        start_pos, interleaved, magnitude, q_out, workspace, stream)


# --------------------------------------------------------------------------
# trees of drafted tokens
# --------------------------------------------------------------------------
def _check_int32_rows(t: torch.Tensor, batch: int, name: str):
    """int32 [batch, n] with contiguous rows."""
    if not (isinstance(t, torch.Tensor) and t.dtype == torch.int32):
        raise ValueError(f"{name} must be int32")
    if not (t.dim() == 2 and t.shape[0] == batch and (t.shape[1] <= 1 or t.stride(1) == 1)):
        raise ValueError(f"{name} must be [{batch}, n] with contiguous rows, got {tuple(t.shape)}")


def paged_tree_workspace_size(batch: int, num_q_heads: int, num_kv_heads: int, num_drafts: int, max_blocks: int,
                              block_size: int = 16, head_dim: int = 128) -> int:
    return int(load().paged_tree_workspace_size(batch, num_q_heads, num_kv_heads, num_drafts, max_blocks, block_size,
                                                head_dim))


def paged_tree_attn(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                    ctx_lens: torch.Tensor, parents: torch.Tensor, k_new: Optional[torch.Tensor] = None,
                    v_new: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, return_lse: bool = False,
                    workspace: Optional[Workspace] = None, stream=None):
    """A tree of T drafted tokens per sequence over its paged cache: q [B, Hq,
    T, D]; parents int32 [B, T] (-1: follows the context, below: no token);
    ctx_lens int32 [B] counts the tokens before the drafts.  With k_new / v_new
    ([B, Hkv, T, D]) draft t's K/V go to slot ctx_lens[b] + t; each draft
    attends to the context, itself and its ancestors."""
    lib = load()
    B, Hq, T, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    if out is None:
        out = _fresh(lambda: torch.empty_strided((B, Hq, T, D), (T * Hq * D, D, Hq * D, 1), dtype=q.dtype,
                                                 device=q.device), stream, q.device)
    if lse is None and return_lse:
        lse = _fresh(lambda: torch.empty((B, Hq, T), dtype=torch.float32, device=q.device), stream, q.device)
    if workspace is not None and q.is_cuda:
        if _call("paged_tree_attn", "xoocbvq=XlWS", q, k_new, v_new, k_cache, v_cache, block_table, ctx_lens, parents,
                 float(scale), out, lse, workspace.tensor, _handle(stream)):
            return (out, lse) if return_lse else out
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    _check_int32_rows(parents, B, "parents")
    if parents.shape[1] != T:
        raise ValueError(f"parents must be [{B}, {T}], got {tuple(parents.shape)}")
    if lse is not None:
        _check_f32_buffer(lse, B * Hq * T, "lse")
    _check_devices("paged_tree_attn", q, k_cache, v_cache, block_table, ctx_lens, parents, k_new, v_new, out, lse,
                   _ws_tensor(workspace))
    c = _cache_bytes(k_cache, v_cache)
    max_blocks = block_table.shape[1]
    ws = workspace
    if ws is None:
        need = paged_tree_workspace_size(B, Hq, k_cache.shape[1], T, max_blocks, k_cache.shape[2], D)
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    dk = _tensor_bytes(k_new) if k_new is not None else None
    dv = _tensor_bytes(v_new) if v_new is not None else None
    st = lib.paged_tree_attn(_tensor_bytes(q), dk, dv, c, _ptr(block_table, "block_table"),
                             block_table.stride(0), max_blocks, _ptr(ctx_lens, "ctx_lens"), _ptr(parents, "parents"),
                             parents.stride(0), float(scale), _tensor_bytes(out), _ptr(lse, "lse"), _ws_ptr(ws),
                             ws.nbytes, _stream(stream))
    _check("paged_tree_attn", st)
    return (out, lse) if return_lse else out


def kv_tree_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, ctx_lens: torch.Tensor,
                   path: torch.Tensor, n_accept: torch.Tensor, workspace: Optional[Workspace] = None, stream=None):
    """Move the cache rows of the accepted drafts path[b, :n_accept[b]] (int32
    [B, n], strictly increasing draft indices) to the slots behind the context,
    ctx_lens[b] + i."""
    lib = load()
    B = ctx_lens.shape[0]
    if k_cache.is_cuda:
        ws = workspace or _small_ws(k_cache.device, stream)
        if _call("kv_tree_accept", "cbVrv=WS", k_cache, v_cache, block_table, ctx_lens, path, n_accept, B, ws.tensor,
                 _handle(stream)):
            return
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    _check_int32_rows(path, B, "path")
    _check_int32_vec(n_accept, B, "n_accept")
    _check_devices("kv_tree_accept", k_cache, v_cache, block_table, ctx_lens, path, n_accept, _ws_tensor(workspace))
    ws = workspace or _small_ws(k_cache.device, stream)
    c = _cache_bytes(k_cache, v_cache)
    st = lib.kv_tree_accept(c, _ptr(block_table, "block_table"), block_table.stride(0),
                            block_table.shape[1], _ptr(ctx_lens, "ctx_lens"), _ptr(path, "path"), path.stride(0),
                            path.shape[1], _ptr(n_accept, "n_accept"), B, _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("kv_tree_accept", st)


# --------------------------------------------------------------------------
# eviction by accumulated attention weight
# --------------------------------------------------------------------------
def _check_acc(acc: torch.Tensor, cache: torch.Tensor):
    if not (isinstance(acc, torch.Tensor) and acc.dtype == torch.float32 and acc.is_contiguous()
            and acc.shape == cache.shape[:3]):
        raise ValueError(f"acc must be contiguous float32 {tuple(cache.shape[:3])}")


def paged_attn_weights_workspace_size(batch: int, num_kv_heads: int, max_blocks: int, block_size: int = 16) -> int:
    return int(load().paged_attn_weights_workspace_size(batch, num_kv_heads, max_blocks, block_size))


def paged_attn_weights(q: torch.Tensor, lse: torch.Tensor, k_cache: torch.Tensor, block_table: torch.Tensor,
                       start_pos: torch.Tensor, acc: torch.Tensor, q_lens: Optional[torch.Tensor] = None,
                       causal: bool = True, scale: Optional[float] = None, workspace: Optional[Workspace] = None,
                       stream=None) -> torch.Tensor:
    """Add the attention weight each cached token received from a chunk of
    queries to acc (float32 [num_blocks, Hkv, 16], in place; the chunk's own
    tokens start from zero).  q [B, Hq, T, D] at positions start_pos[b] + i with
    lse float32 [B, Hq, T] as an attention call returned it; [B, Hq, D] and [B,
    Hq] for one token a sequence.  q_lens int32 [B]: queries of each sequence."""
    lib = load()
    if workspace is not None and q.is_cuda:
        if _call("paged_attn_weights", "ylcbvn==AWS", q, lse, k_cache, k_cache, block_table, start_pos, q_lens,
                 int(bool(causal)), float(1.0 / math.sqrt(q.shape[-1]) if scale is None else scale), acc, workspace.tensor,
                 _handle(stream)):
            return acc
    if q.dim() == 3:
        q, lse = q.unsqueeze(2), lse.unsqueeze(2)
    B, Hq, T, D = q.shape
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _check_f32_buffer(lse, B * Hq * T, "lse")
    _check_block_table(block_table, B)
    _check_int32_vec(start_pos, B, "start_pos")
    if q_lens is not None:
        _check_int32_vec(q_lens, B, "q_lens")
    c = _cache_bytes(k_cache, k_cache)
    _check_acc(acc, k_cache)
    _check_devices("paged_attn_weights", q, lse, k_cache, block_table, start_pos, acc, q_lens, _ws_tensor(workspace))
    max_blocks = block_table.shape[1]
    ws = workspace
    if ws is None:
        need = paged_attn_weights_workspace_size(B, k_cache.shape[1], max_blocks, k_cache.shape[2])
        ws = _fresh(lambda: Workspace(need, device=q.device), stream, q.device)
    st = lib.paged_attn_weights(_tensor_bytes(q), _ptr(lse, "lse"), c, _ptr(block_table, "block_table"),
                                block_table.stride(0), max_blocks, _ptr(start_pos, "start_pos"),
                                _ptr(q_lens, "q_lens"), int(bool(causal)), float(scale), _ptr(acc, "acc"), _ws_ptr(ws),
                                ws.nbytes, _stream(stream))
    _check("paged_attn_weights", st)
    return acc


def kv_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, acc: torch.Tensor, block_table: torch.Tensor,
             ctx_lens: torch.Tensor, dst_block_table: torch.Tensor, keep: int, sink: int = 0, recent: int = 0,
             new_lens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
             workspace: Optional[Workspace] = None, stream=None):
    """Keep `keep` tokens of each sequence and KV head (the first `sink`, the
    last `recent`, and the largest acc of the others) and copy their K, V and
    acc, in order, to the blocks of dst_block_table.  Returns (new_lens int32
    [B], kept int32 [B, Hkv, keep]: the source slots, -1 past them); new_lens may
    be ctx_lens, which is then updated in place."""
    lib = load()
    B, Hkv = ctx_lens.shape[0], k_cache.shape[1]
    keep, sink, recent = int(keep), int(sink), int(recent)
    if max(keep, sink, recent) >= 1 << 31 or min(keep, sink, recent) < -1 << 31:  # C would see their low 32 bits
        raise ValueError(f"keep, sink and recent must be 32-bit integers, got {keep}, {sink} and {recent}")
    if new_lens is None:
        new_lens = _fresh(lambda: torch.empty(B, dtype=torch.int32, device=k_cache.device), stream, k_cache.device)
    if kept is None:
        kept = _fresh(lambda: torch.empty((B, Hkv, max(keep, 0)), dtype=torch.int32, device=k_cache.device), stream,
                      k_cache.device)
    if k_cache.is_cuda and kept.shape == (B, Hkv, keep):
        ws = workspace or _small_ws(k_cache.device, stream)
        if _call("kv_evict", "cAbVb====vKWS", k_cache, v_cache, acc, block_table, ctx_lens, dst_block_table, B, keep,
                 sink, recent, new_lens, kept, ws.tensor, _handle(stream)):
            return new_lens, kept
    _check_block_table(block_table, B)
    _check_int32_vec(ctx_lens, B, "ctx_lens")
    if not (isinstance(dst_block_table, torch.Tensor) and dst_block_table.dtype == torch.int32
            and dst_block_table.dim() == 2 and dst_block_table.shape[0] >= B and dst_block_table.stride(1) == 1
            and dst_block_table.stride(0) >= dst_block_table.shape[1]):
        raise ValueError(f"dst_block_table must be int32 [>= {B}, blocks] with contiguous rows")
    c = _cache_bytes(k_cache, v_cache)
    _check_acc(acc, k_cache)
    _check_int32_vec(new_lens, B, "new_lens")
    if not (kept.dtype == torch.int32 and kept.is_contiguous() and kept.shape == (B, Hkv, keep)):
        raise ValueError(f"kept must be contiguous int32 {(B, Hkv, keep)}, got {tuple(kept.shape)}")
    _check_devices("kv_evict", k_cache, v_cache, acc, block_table, ctx_lens, dst_block_table, new_lens, kept,
                   _ws_tensor(workspace))
    ws = workspace or _small_ws(k_cache.device, stream)
    st = lib.kv_evict(c, _ptr(acc, "acc"), _ptr(block_table, "block_table"), block_table.stride(0),
                      block_table.shape[1], _ptr(ctx_lens, "ctx_lens"), _ptr(dst_block_table, "dst_block_table"),
                      dst_block_table.stride(0), dst_block_table.shape[1], B, keep, sink, recent,
                      _ptr(new_lens, "new_lens"), _ptr(kept, "kept"), _ws_ptr(ws), ws.nbytes, _stream(stream))
    _check("kv_evict", st)
    return new_lens, kept
