"""ctypes binding of libhs2 (argument marshalling only; every step runs in the CUDA
library).  PyTorch provides device memory and the current stream.

    cache = Cache(k, v, lens)                        # FP8: Cache(k, v, lens, k_scale, v_scale)
    ws = alloc_workspace(cache, n_q, h_q)
    kv_append(k_new, v_new, cache, ws)               # the new tokens' K/V rows; lens grows
    out, idx, lse = full_attn_select(q, cache, workspace=ws)    # full layer + selection
    out_l = sparse_attn(q_layer, cache, idx, ws)     # one reusing sparse layer
    # comparators and neighbours of the step:
    out, idx, lse = full_attn_select_blocks(q, cache, block=64, workspace=ws)
    out, lse = prefill_attn(q_chunk, cache)          # full layer over a chunk of new tokens

Serving many sequences (grouped K/V heads, a cache in pages, prompts packed together):

    cache = PagedCache(k_pages, v_pages, pages, lens)     # FP8: with k_scale, v_scale
    ws = paged_workspace(cache, h_q)
    out, lse = packed_attn(q, k, v, cu_q)                 # causal, prompts of any lengths
    paged_kv_write(k, v, cache, ws, cu_new=cu_q)          # their rows into the pages
    paged_kv_write(k_new, v_new, cache, ws)               # one new token per sequence ...
    out, lse = paged_attn(q_new, cache, ws)               # ... and its attention
    k, v = paged_kv_read(cache, cu, ws)                   # cached rows back, packed

The library is loaded from ``long_context_token_b200/_lib/libhs2.so``.  There is no
fallback: if the library is missing or no CUDA device is present, calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
from typing import Optional, Tuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libhs2.so")

HS2_KV_BF16 = 0
HS2_KV_FP8_E4M3 = 1
HS2_KV_F16 = 2

STATUS = {
    0: "HS2_OK", 1: "HS2_ERR_INVALID_ARGUMENT", 2: "HS2_ERR_UNSUPPORTED",
    3: "HS2_ERR_WORKSPACE_TOO_SMALL", 4: "HS2_ERR_CUDA", 5: "HS2_ERR_DEVICE_TIMEOUT",
    6: "HS2_ERR_INDEX_OUT_OF_RANGE", 7: "HS2_ERR_BAD_LENGTH",
}

EXPORTS = ("hs2_workspace_bytes", "hs2_full_attn_select", "hs2_full_attn", "hs2_select",
           "hs2_sparse_attn", "hs2_check_device_status", "hs2_status_string",
           "hs2_last_cuda_error", "hs2_abi_version", "hs2_sparse_attn_noalloc", "hs2_kv_append",
           "hs2_full_attn_select_blocks", "hs2_select_blocks", "hs2_prefill_workspace_bytes",
           "hs2_prefill_attn", "hs2_select_fused", "hs2_workspace_lse64_offset",
           "hs2_debug_stall_waits", "hs2_set_deterministic", "hs2_paged_workspace_bytes",
           "hs2_paged_kv_write", "hs2_paged_kv_read", "hs2_paged_attn",
           "hs2_packed_workspace_bytes", "hs2_packed_attn")


class Hs2Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        self.name = STATUS.get(code, str(code))
        detail = lib().hs2_status_string(code).decode()
        cuda = lib().hs2_last_cuda_error().decode() if code == 4 else ""
        super().__init__(f"{what}: {self.name} ({detail}){' - ' + cuda if cuda else ''}")


class KV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("lens", ctypes.c_void_p), ("batch", ctypes.c_int32),
                ("max_len", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class PagedKV(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("pages", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("scale_page_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64), ("scale_row_stride", ctypes.c_int64),
                ("batch", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32)]


class Packed(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("cu_q", ctypes.c_void_p), ("cu_k", ctypes.c_void_p),
                ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("kv_token_stride", ctypes.c_int64), ("kv_head_stride", ctypes.c_int64),
                ("n_q", ctypes.c_int32), ("n_k", ctypes.c_int32), ("batch", ctypes.c_int32),
                ("h_q", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


_lib = None


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load libhs2 (once).  Raises if the shared library has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"libhs2 is not built ({_LIB_PATH} missing); run "
                           "`python -m long_context_token_b200.build`")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    kvp = ctypes.POINTER(KV)
    L.hs2_workspace_bytes.argtypes = [i32] * 7
    L.hs2_workspace_bytes.restype = sz
    L.hs2_full_attn_select.argtypes = [vp, i32, i32, kvp, i32, i32, f32, vp, vp, vp, vp, sz, vp]
    L.hs2_full_attn_select.restype = i32
    L.hs2_full_attn.argtypes = [vp, i32, i32, kvp, i32, i32, f32, vp, vp, vp, sz, vp]
    L.hs2_full_attn.restype = i32
    L.hs2_select.argtypes = [vp, i32, i32, kvp, i32, i32, f32, vp, vp, sz, vp]
    L.hs2_select.restype = i32
    L.hs2_sparse_attn.argtypes = [vp, i32, i32, kvp, vp, i32, f32, vp, vp, sz, vp]
    L.hs2_sparse_attn.restype = i32
    L.hs2_sparse_attn_noalloc.argtypes = [vp, i32, i32, kvp, vp, i32, f32, vp, vp, vp]
    L.hs2_sparse_attn_noalloc.restype = i32
    L.hs2_full_attn_select_blocks.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, vp, vp, vp,
                                              vp, sz, vp]
    L.hs2_full_attn_select_blocks.restype = i32
    L.hs2_select_blocks.argtypes = [vp, i32, i32, kvp, i32, i32, i32, f32, vp, vp, sz, vp]
    L.hs2_select_blocks.restype = i32
    L.hs2_prefill_workspace_bytes.argtypes = [i32] * 5
    L.hs2_prefill_workspace_bytes.restype = sz
    L.hs2_prefill_attn.argtypes = [vp, i32, i32, kvp, f32, vp, vp, vp, sz, vp]
    L.hs2_prefill_attn.restype = i32
    L.hs2_kv_append.argtypes = [vp, vp, i32, kvp, vp, vp, sz, vp]
    L.hs2_kv_append.restype = i32
    L.hs2_check_device_status.argtypes = [vp, vp]
    L.hs2_check_device_status.restype = i32
    L.hs2_status_string.argtypes = [i32]
    L.hs2_status_string.restype = ctypes.c_char_p
    L.hs2_last_cuda_error.argtypes = []
    L.hs2_last_cuda_error.restype = ctypes.c_char_p
    L.hs2_abi_version.argtypes = []
    L.hs2_abi_version.restype = i32
    L.hs2_select_fused.argtypes = [i32, i32, i32]
    L.hs2_select_fused.restype = i32
    L.hs2_workspace_lse64_offset.argtypes = [i32] * 7
    L.hs2_workspace_lse64_offset.restype = sz
    L.hs2_debug_stall_waits.argtypes = [i32]
    L.hs2_debug_stall_waits.restype = None
    L.hs2_set_deterministic.argtypes = [i32]
    L.hs2_set_deterministic.restype = None
    i64, pgp = ctypes.c_int64, ctypes.POINTER(PagedKV)
    L.hs2_paged_workspace_bytes.argtypes = [pgp, i32]
    L.hs2_paged_workspace_bytes.restype = sz
    L.hs2_paged_kv_write.argtypes = [vp, vp, i32, i64, i64, i32, vp, pgp, vp, sz, vp]
    L.hs2_paged_kv_write.restype = i32
    L.hs2_paged_kv_read.argtypes = [pgp, vp, vp, i32, vp, vp, i32, i64, i64, vp, sz, vp]
    L.hs2_paged_kv_read.restype = i32
    L.hs2_paged_attn.argtypes = [vp, i32, i32, i64, i64, pgp, f32, vp, vp, vp, sz, vp]
    L.hs2_paged_attn.restype = i32
    L.hs2_packed_workspace_bytes.argtypes = []
    L.hs2_packed_workspace_bytes.restype = sz
    L.hs2_packed_attn.argtypes = [ctypes.POINTER(Packed), f32, vp, vp, vp, sz, vp]
    L.hs2_packed_attn.restype = i32
    _lib = L
    return L


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _check(code: int, what: str):
    if code != 0:
        raise Hs2Error(code, what)


class Cache:
    """The shared KV cache of one hybrid block, resident on the device.

    k, v: [B, max_len, 128] bf16, or uint8 / float8_e4m3fn E4M3 codes with
    k_scale / v_scale float32 [B, max_len]; lens int32 [B]."""

    def __init__(self, k, v, lens, k_scale=None, v_scale=None):
        if k.dtype == torch.float8_e4m3fn:
            k, v = k.view(torch.uint8), v.view(torch.uint8)
        fp8 = k.dtype == torch.uint8
        for name, t in (("k", k), ("v", v), ("lens", lens)):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous CUDA tensor")
        if k.shape != v.shape or k.dim() != 3 or k.shape[2] != 128:
            raise ValueError("k and v must be [B, max_len, 128]")
        if not fp8 and k.dtype != torch.bfloat16:
            raise ValueError("k/v must be bfloat16 or E4M3 codes")
        if lens.dtype != torch.int32 or lens.shape != (k.shape[0],):
            raise ValueError("lens must be int32 [B]")
        if fp8:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is None or t.dtype != torch.float32 or not t.is_cuda or \
                        t.shape != k.shape[:2] or not t.is_contiguous():
                    raise ValueError(f"{name} must be float32 [B, max_len] on the device")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("bf16 caches take no scales")
        self.k, self.v, self.lens, self.k_scale, self.v_scale = k, v, lens, k_scale, v_scale
        self.dtype = HS2_KV_FP8_E4M3 if fp8 else HS2_KV_BF16
        self._struct = KV(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                          lens.data_ptr(), k.shape[0], k.shape[1], 128, self.dtype)

    @property
    def batch(self) -> int:
        return self.k.shape[0]

    @property
    def max_len(self) -> int:
        return self.k.shape[1]

    def ref(self):
        return ctypes.byref(self._struct)


def workspace_bytes(batch: int, n_q: int, h_q: int, max_len: int, window: int = 128,
                    k_sel: int = 1024, fp8: bool = False) -> int:
    n = lib().hs2_workspace_bytes(batch, n_q, h_q, max_len, window, k_sel,
                                  HS2_KV_FP8_E4M3 if fp8 else HS2_KV_BF16)
    if n == 0:
        raise Hs2Error(2, "hs2_workspace_bytes")
    return n


def alloc_workspace(cache: Cache, n_q: int, h_q: int, window: int = 128, k_sel: int = 1024,
                    device=None) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for these sizes."""
    n = workspace_bytes(cache.batch, n_q, h_q, cache.max_len, window, k_sel,
                        cache.dtype == HS2_KV_FP8_E4M3)
    return torch.zeros(n, dtype=torch.uint8, device=device or cache.k.device)


def _check_q(q: torch.Tensor, cache: Cache) -> Tuple[int, int]:
    if q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous() or q.dim() != 4 \
            or q.shape[0] != cache.batch or q.shape[3] != 128:
        raise ValueError("queries must be contiguous bf16 [B, n_q, h_q, 128] on the device")
    return q.shape[1], q.shape[2]


def default_scale() -> float:
    return float(torch.tensor(1.0 / math.sqrt(128.0), dtype=torch.float32))


def select_fused(cache: "Cache", n_q: int, h_q: int) -> bool:
    """True if full_attn_select runs as one kernel for these sizes (hs2_select_fused)."""
    return bool(lib().hs2_select_fused(n_q, h_q, cache.dtype))


def set_deterministic(on: bool) -> None:
    """Static key chunks in the full layer: bitwise-reproducible runs (hs2_set_deterministic)."""
    lib().hs2_set_deterministic(1 if on else 0)


def workspace_lse64(workspace: torch.Tensor, cache: "Cache", n_q: int, h_q: int,
                    window: int = 128, k_sel: int = 1024) -> torch.Tensor:
    """The float64 lse [batch, n_q, h_q] that the last full layer left in `workspace`
    (a view, not a copy; hs2_workspace_lse64_offset)."""
    off = lib().hs2_workspace_lse64_offset(cache.batch, n_q, h_q, cache.max_len, window,
                                           k_sel, cache.dtype)
    if off == (1 << 64) - 1:
        raise Hs2Error(2, "hs2_workspace_lse64_offset")
    n = cache.batch * n_q * h_q * 8
    return workspace[off:off + n].view(torch.float64).view(cache.batch, n_q, h_q)


def full_attn_select(q: torch.Tensor, cache: Cache, window: int = 128, k_sel: int = 1024,
                     sm_scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Full-attention layer + token selection.  Returns (out, idx, lse)."""
    n_q, h = _check_q(q, cache)
    B = cache.batch
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if workspace is None:
        workspace = alloc_workspace(cache, n_q, h, window, k_sel)
    if out is None:
        out = torch.empty(B, n_q, h, 128, dtype=torch.float32, device=q.device)
    if idx is None:
        idx = torch.empty(B, n_q, window + k_sel, dtype=torch.int32, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, n_q, h, dtype=torch.float32, device=q.device)
    code = lib().hs2_full_attn_select(q.data_ptr(), n_q, h, cache.ref(), window, k_sel,
                                      sm_scale, out.data_ptr(), idx.data_ptr(), _ptr(lse),
                                      workspace.data_ptr(), workspace.numel(), _stream(stream))
    _check(code, "hs2_full_attn_select")
    return out, idx, lse


def full_attn_select_blocks(q: torch.Tensor, cache: Cache, window: int = 128, k_sel: int = 1024,
                            block: int = 64, sm_scale: Optional[float] = None,
                            workspace: Optional[torch.Tensor] = None,
                            out: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                            lse: Optional[torch.Tensor] = None, want_lse: bool = True,
                            stream=None):
    """Full-attention layer + block-level selection (whole blocks of ``block``
    positions, the first-generation comparator).  Returns (out, idx, lse)."""
    n_q, h = _check_q(q, cache)
    B = cache.batch
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if workspace is None:
        workspace = alloc_workspace(cache, n_q, h, window, k_sel)
    if out is None:
        out = torch.empty(B, n_q, h, 128, dtype=torch.float32, device=q.device)
    if idx is None:
        idx = torch.empty(B, n_q, window + k_sel, dtype=torch.int32, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(B, n_q, h, dtype=torch.float32, device=q.device)
    code = lib().hs2_full_attn_select_blocks(q.data_ptr(), n_q, h, cache.ref(), window, k_sel,
                                             block, sm_scale, out.data_ptr(), idx.data_ptr(),
                                             _ptr(lse), workspace.data_ptr(), workspace.numel(),
                                             _stream(stream))
    _check(code, "hs2_full_attn_select_blocks")
    return out, idx, lse


def select_blocks(q, cache: Cache, workspace: torch.Tensor, window=128, k_sel=1024, block=64,
                  sm_scale=None, idx=None, stream=None):
    """Block-level selection alone; must follow full_attn on the same workspace."""
    n_q, h = _check_q(q, cache)
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if idx is None:
        idx = torch.empty(cache.batch, n_q, window + k_sel, dtype=torch.int32, device=q.device)
    code = lib().hs2_select_blocks(q.data_ptr(), n_q, h, cache.ref(), window, k_sel, block,
                                   sm_scale, idx.data_ptr(), workspace.data_ptr(),
                                   workspace.numel(), _stream(stream))
    _check(code, "hs2_select_blocks")
    return idx


def prefill_workspace(cache: Cache, n_q: int, h_q: int, device=None) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for prefill_attn at these sizes."""
    n = lib().hs2_prefill_workspace_bytes(cache.batch, n_q, h_q, cache.max_len, cache.dtype)
    if n == 0:
        raise Hs2Error(2, "hs2_prefill_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device or cache.k.device)


def prefill_attn(q: torch.Tensor, cache: Cache, sm_scale: Optional[float] = None,
                 workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Full-attention layer over a chunk of n_q new tokens per sequence (chunked
    prefill; no selection).  Returns (out, lse)."""
    n_q, h = _check_q(q, cache)
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if workspace is None:
        workspace = prefill_workspace(cache, n_q, h)
    if out is None:
        out = torch.empty(cache.batch, n_q, h, 128, dtype=torch.float32, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty(cache.batch, n_q, h, dtype=torch.float32, device=q.device)
    code = lib().hs2_prefill_attn(q.data_ptr(), n_q, h, cache.ref(), sm_scale, out.data_ptr(),
                                  _ptr(lse), workspace.data_ptr(), workspace.numel(),
                                  _stream(stream))
    _check(code, "hs2_prefill_attn")
    return out, lse


def full_attn(q, cache: Cache, window=128, k_sel=1024, sm_scale=None, workspace=None,
              out=None, lse=None, stream=None):
    """Full-attention layer alone (leaves the per-head lse in the workspace)."""
    n_q, h = _check_q(q, cache)
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if workspace is None:
        workspace = alloc_workspace(cache, n_q, h, window, k_sel)
    if out is None:
        out = torch.empty(cache.batch, n_q, h, 128, dtype=torch.float32, device=q.device)
    code = lib().hs2_full_attn(q.data_ptr(), n_q, h, cache.ref(), window, k_sel, sm_scale,
                               out.data_ptr(), _ptr(lse), workspace.data_ptr(),
                               workspace.numel(), _stream(stream))
    _check(code, "hs2_full_attn")
    return out


def select(q, cache: Cache, workspace: torch.Tensor, window=128, k_sel=1024, sm_scale=None,
           idx=None, stream=None):
    """Token selection alone; must follow full_attn on the same workspace."""
    n_q, h = _check_q(q, cache)
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if idx is None:
        idx = torch.empty(cache.batch, n_q, window + k_sel, dtype=torch.int32, device=q.device)
    code = lib().hs2_select(q.data_ptr(), n_q, h, cache.ref(), window, k_sel, sm_scale,
                            idx.data_ptr(), workspace.data_ptr(), workspace.numel(),
                            _stream(stream))
    _check(code, "hs2_select")
    return idx


def sparse_attn(q_layer: torch.Tensor, cache: Cache, idx: torch.Tensor,
                workspace: torch.Tensor, sm_scale: Optional[float] = None,
                out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """One reusing sparse-attention layer over the rows named by ``idx``."""
    n_q, h = _check_q(q_layer, cache)
    if idx.dtype != torch.int32 or not idx.is_contiguous() or idx.dim() != 3 \
            or idx.shape[:2] != (cache.batch, n_q):
        raise ValueError("idx must be contiguous int32 [B, n_q, width]")
    sm_scale = default_scale() if sm_scale is None else sm_scale
    if out is None:
        out = torch.empty(cache.batch, n_q, h, 128, dtype=torch.float32, device=q_layer.device)
    code = lib().hs2_sparse_attn(q_layer.data_ptr(), n_q, h, cache.ref(), idx.data_ptr(),
                                 idx.shape[2], sm_scale, out.data_ptr(), workspace.data_ptr(),
                                 workspace.numel(), _stream(stream))
    _check(code, "hs2_sparse_attn")
    return out


def kv_append(k_new: torch.Tensor, v_new: torch.Tensor, cache: Cache, workspace: torch.Tensor,
              stream=None) -> None:
    """Appends n_new tokens per sequence to ``cache`` (bf16 [B, n_new, 128] keys and
    values; FP8 caches quantise each new row with its own scale) and grows
    ``cache.lens`` in place."""
    for name, t in (("k_new", k_new), ("v_new", v_new)):
        if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 3 \
                or t.shape[0] != cache.batch or t.shape[2] != 128:
            raise ValueError(f"{name} must be contiguous bf16 [B, n_new, 128] on the device")
    if k_new.shape != v_new.shape:
        raise ValueError("k_new and v_new must have the same shape")
    code = lib().hs2_kv_append(k_new.data_ptr(), v_new.data_ptr(), k_new.shape[1], cache.ref(),
                               cache.lens.data_ptr(), workspace.data_ptr(), workspace.numel(),
                               _stream(stream))
    _check(code, "hs2_kv_append")


def check_device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise, return (and clear) the first device-side error code (0 = none)."""
    return lib().hs2_check_device_status(workspace.data_ptr(), _stream(stream))


# ---------------------------------------------------------------- paged caches, packed prompts
_FLOAT16S = {torch.bfloat16: HS2_KV_BF16, torch.float16: HS2_KV_F16}


def _launch(what: str, index: int, stream, *args) -> None:
    """Calls a library function on device ``index`` (the tensors' own, which need not be the
    current one) and on ``stream`` (default: that device's current stream)."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)  # (no Stream object: these calls are short)
    elif stream.device_index != index:
        raise ValueError("stream and tensors must be on the same device")
    else:
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        code = getattr(lib(), what)(*args, raw)
    else:
        with torch.cuda.device(index):
            code = getattr(lib(), what)(*args, raw)
    if code:
        raise Hs2Error(code, what)


def _new(stream, make, *shape, **kw) -> torch.Tensor:
    """A tensor made (torch.empty, torch.zeros) on the stream that uses it."""
    if stream is None:
        return make(*shape, **kw)
    with torch.cuda.stream(stream):
        return make(*shape, **kw)


def _check_on(index: int, *tensors: Optional[torch.Tensor]) -> None:
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"every tensor of a call must be on the same device (cuda:{index})")


def _check_int32(name: str, t: torch.Tensor, shape: Tuple[int, ...]) -> None:
    if t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {list(shape)}")


def _check_ws(ws: torch.Tensor) -> None:
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous uint8 tensor")


def _row_strides(name: str, t: torch.Tensor) -> Tuple[int, ...]:
    """Strides of all axes but the last, which must be contiguous.  Axes of one element get
    the dense stride: theirs is never used and may be anything."""
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name} must be contiguous along its last axis")
    strides = strides[:-1]
    if 1 in shape:
        strides = list(strides)
        dense = shape[-1]
        for i in range(len(strides) - 1, -1, -1):
            if shape[i] <= 1:
                strides[i] = dense
            dense *= shape[i]
        strides = tuple(strides)
    return strides


class PagedCache:
    """A KV cache in pages with grouped K/V heads, resident on the device.

    k, v: [num_pages, h_kv, page_size, d] (d 64 or 128, page_size a power of two in
    [8, 256]), bfloat16, float16, or uint8 / float8_e4m3fn E4M3 codes with k_scale / v_scale
    float32 [num_pages, h_kv, page_size].  Any strides with a contiguous last axis will do (a
    cache held as [num_pages, page_size, h_kv, d] is passed as ``cache.transpose(1, 2)``), the
    same for k and v.  pages int32 [B, max_pages]: the pages of each sequence in order; lens
    int32 [B]: its length.  Both are read on the device at every call and may change between
    calls."""

    def __init__(self, k, v, pages, lens, k_scale=None, v_scale=None):
        if k.dtype == torch.float8_e4m3fn:
            k, v = k.view(torch.uint8), v.view(torch.uint8)
        fp8 = k.dtype == torch.uint8
        if not k.is_cuda:
            raise ValueError("k must be a CUDA tensor")
        self.index = k.get_device()
        _check_on(self.index, v, pages, lens, k_scale, v_scale)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be [num_pages, h_kv, page_size, d] of one type")
        if not fp8 and k.dtype not in _FLOAT16S:
            raise ValueError("k/v must be bfloat16, float16 or E4M3 codes")
        strides = _row_strides("k", k)
        if strides != _row_strides("v", v):
            raise ValueError("k and v must have the same strides")
        if pages.dim() != 2:
            raise ValueError("pages must be int32 [B, max_pages]")
        _check_int32("pages", pages, pages.shape)
        _check_int32("lens", lens, pages.shape[:1])
        scale_strides = (0, 0, 0)
        if fp8:
            for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
                if t is None or t.dtype != torch.float32 or t.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be float32 [num_pages, h_kv, page_size]")
            # (a last axis of one, so that every stride counts as a row's)
            scale_strides = _row_strides("k_scale", k_scale.unsqueeze(3))
            if scale_strides != _row_strides("v_scale", v_scale.unsqueeze(3)):
                raise ValueError("k_scale and v_scale must have the same strides")
        elif k_scale is not None or v_scale is not None:
            raise ValueError("16-bit caches take no scales")
        self.k, self.v, self.pages, self.lens = k, v, pages, lens
        self.k_scale, self.v_scale = k_scale, v_scale
        self.dtype = HS2_KV_FP8_E4M3 if fp8 else _FLOAT16S[k.dtype]
        self._struct = PagedKV(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale),
                               pages.data_ptr(), lens.data_ptr(), *strides, *scale_strides,
                               pages.shape[0], pages.shape[1], k.shape[0], k.shape[2], k.shape[1],
                               k.shape[3], self.dtype)
        self._ref = ctypes.byref(self._struct)
        self.batch, self.h_kv, self.head_dim = pages.shape[0], k.shape[1], k.shape[3]
        #: types of the rows and queries that go with this cache
        self.row_dtypes = tuple(_FLOAT16S) if fp8 else (k.dtype,)

    def ref(self):
        return self._ref


def paged_workspace(cache: PagedCache, h_q: int = 0) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for the paged calls with h_q query heads (0:
    paged_kv_write and paged_kv_read only)."""
    n = lib().hs2_paged_workspace_bytes(cache.ref(), h_q)
    if n == 0:
        raise Hs2Error(2, "hs2_paged_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def _check_rows(k_name: str, v_name: str, k: torch.Tensor, v: torch.Tensor, cache: PagedCache,
                ws: torch.Tensor):
    """Packed rows of a paged cache (and the workspace): their type code and strides."""
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or shape[1] != cache.h_kv or shape[2] != cache.head_dim \
            or v.shape != shape or v.dtype != dtype or dtype not in cache.row_dtypes:
        raise ValueError(f"{k_name} and {v_name} must be [T, {cache.h_kv}, {cache.head_dim}] of "
                         f"one type of {cache.row_dtypes}")
    strides = _row_strides(k_name, k)
    if v.stride() != k.stride() and _row_strides(v_name, v) != strides:
        raise ValueError(f"{k_name} and {v_name} must have the same strides")
    if not k.get_device() == v.get_device() == ws.get_device() == cache.index:
        raise ValueError(f"{k_name}, {v_name} and the workspace must be on the cache's device")
    _check_ws(ws)
    return _FLOAT16S[dtype], strides


def paged_kv_write(k_new: torch.Tensor, v_new: torch.Tensor, cache: PagedCache,
                   workspace: torch.Tensor, cu_new: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Writes new tokens' rows [T, h_kv, d] into the pages (quantised, each row with its own
    scale, when the cache is FP8).  ``cache.lens`` counts them already: token i of the n_b of
    sequence b goes to position lens[b] - n_b + i.  cu_new int32 [B + 1]: the sequences'
    ranges of tokens; None: T / B tokens each."""
    dtype, strides = _check_rows("k_new", "v_new", k_new, v_new, cache, workspace)
    if cu_new is not None:
        _check_int32("cu_new", cu_new, (cache.batch + 1,))
        _check_on(cache.index, cu_new)
    _launch("hs2_paged_kv_write", cache.index, stream, k_new.data_ptr(), v_new.data_ptr(),
            dtype, *strides, k_new.shape[0], _ptr(cu_new), cache.ref(), workspace.data_ptr(),
            workspace.numel())


def paged_kv_read(cache: PagedCache, cu: torch.Tensor, workspace: torch.Tensor,
                  start: Optional[torch.Tensor] = None, n_tokens: Optional[int] = None,
                  dtype: Optional[torch.dtype] = None, k_out: Optional[torch.Tensor] = None,
                  v_out: Optional[torch.Tensor] = None, stream=None):
    """Reads cached rows back (dequantised when FP8): packed token i of sequence b, tokens
    [cu[b], cu[b + 1]), is position start[b] + i (start None: i).  Returns (k, v), both
    [n_tokens, h_kv, d]: ``k_out`` and ``v_out``, or new tensors of ``n_tokens`` rows (None:
    cu[-1], which waits for the device) of ``dtype`` (None: the cache's type, bfloat16 when
    FP8), zero where no row is read."""
    _check_int32("cu", cu, (cache.batch + 1,))
    if start is not None:
        _check_int32("start", start, (cache.batch,))
    _check_on(cache.index, cu, start)
    if (k_out is None) != (v_out is None):
        raise ValueError("k_out and v_out go together")
    if k_out is None:
        if n_tokens is None:
            with torch.cuda.stream(stream):  # (cu may have been written on it; None: the current one)
                n_tokens = int(cu[-1])
        if dtype is None:
            dtype = torch.bfloat16 if cache.dtype == HS2_KV_FP8_E4M3 else cache.k.dtype
        k_out, v_out = (_new(stream, torch.zeros, n_tokens, cache.h_kv, cache.head_dim,
                             dtype=dtype, device=cache.k.device) for _ in range(2))
    code, strides = _check_rows("k_out", "v_out", k_out, v_out, cache, workspace)
    _launch("hs2_paged_kv_read", cache.index, stream, cache.ref(), cu.data_ptr(), _ptr(start),
            k_out.shape[0], k_out.data_ptr(), v_out.data_ptr(), code, *strides,
            workspace.data_ptr(), workspace.numel())
    return k_out, v_out


def _check_out(name: str, t: Optional[torch.Tensor], dtype: torch.dtype, shape) -> None:
    if t is not None and (t.dtype != dtype or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)}")


def paged_attn(q: torch.Tensor, cache: PagedCache, workspace: Optional[torch.Tensor] = None,
               sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
               lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Attention of one new token per sequence over its pages.  q [B, h_q, d] in the cache's
    type (bfloat16 or float16 when FP8), h_q a multiple of h_kv (query head h reads K/V head
    h // (h_q // h_kv)), any strides with a contiguous last axis.  Returns (out, lse): out
    like q and dense, lse float32 [B, h_q]; 0 and -inf for an empty sequence."""
    if q.dim() != 3 or q.shape[0] != cache.batch or q.shape[2] != cache.head_dim \
            or q.dtype not in cache.row_dtypes:
        raise ValueError("queries must be [B, h_q, d] of the cache's type (bfloat16 or float16 "
                         "for FP8)")
    shape = q.shape
    B, h_q, d = shape
    strides = _row_strides("q", q)
    _check_out("out", out, q.dtype, shape)
    _check_out("lse", lse, torch.float32, shape[:2])
    _check_on(cache.index, q, out, lse, workspace)
    if workspace is None:
        n = lib().hs2_paged_workspace_bytes(cache.ref(), h_q)
        if n == 0:
            raise Hs2Error(2, "hs2_paged_workspace_bytes")
        workspace = _new(stream, torch.zeros, n, dtype=torch.uint8, device=q.device)
    _check_ws(workspace)
    if out is None:
        out = _new(stream, torch.empty, B, h_q, d, dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = _new(stream, torch.empty, B, h_q, dtype=torch.float32, device=q.device)
    sm_scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    _launch("hs2_paged_attn", cache.index, stream, q.data_ptr(), _FLOAT16S[q.dtype], h_q, *strides,
            cache.ref(), sm_scale, out.data_ptr(), _ptr(lse), workspace.data_ptr(),
            workspace.numel())
    return out, lse


def packed_workspace(device) -> torch.Tensor:
    """A zero-filled workspace (uint8 tensor) for packed_attn, of any sizes."""
    return torch.zeros(lib().hs2_packed_workspace_bytes(), dtype=torch.uint8, device=device)


def packed_attn(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                cu_k: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                sm_scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                lse: Optional[torch.Tensor] = None, want_lse: bool = True, stream=None):
    """Causal attention over packed prompts of different lengths.  q [Tq, h_q, d], k and v
    [Tk, h_kv, d], bfloat16 or float16, d 64 or 128, any strides with a contiguous last axis
    (the same for k and v; slices of one fused projection will do).  Sequence b has queries
    [cu_q[b], cu_q[b + 1]) and keys [cu_k[b], cu_k[b + 1]) (cu_k None: cu_q), int32 [B + 1];
    its last query sees its last key.  Returns (out, lse): out [Tq, h_q, d] like q and dense,
    lse float32 [Tq, h_q]; 0 and -inf for a query that sees nothing.  Rows behind cu_q[B] are
    left as they were (zeros, lse -inf, in tensors made here)."""
    cu_k = cu_q if cu_k is None else cu_k
    if not q.is_cuda or q.dtype not in _FLOAT16S or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k and v must be bfloat16 or float16 CUDA tensors of one type")
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [Tq, h_q, d], k and v [Tk, h_kv, d]")
    if cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError("cu_q must be int32 [B + 1]")
    B = cu_q.shape[0] - 1
    _check_int32("cu_q", cu_q, (B + 1,))
    if cu_k is not cu_q:
        _check_int32("cu_k", cu_k, (B + 1,))
    shape, index = q.shape, q.get_device()
    tq, h_q, d = shape
    q_strides, kv_strides = _row_strides("q", q), _row_strides("k", k)
    if v.stride() != k.stride() and _row_strides("v", v) != kv_strides:
        raise ValueError("k and v must have the same strides")
    _check_out("out", out, q.dtype, shape)
    _check_out("lse", lse, torch.float32, shape[:2])
    _check_on(index, k, v, cu_q, cu_k, out, lse, workspace)
    if workspace is None:
        workspace = _new(stream, packed_workspace, q.device)
    _check_ws(workspace)
    if out is None:
        out = _new(stream, torch.zeros, tq, h_q, d, dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = _new(stream, torch.full, (tq, h_q), -math.inf, dtype=torch.float32, device=q.device)
    sm_scale = 1.0 / math.sqrt(d) if sm_scale is None else sm_scale
    args = Packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), cu_k.data_ptr(),
                  *q_strides, *kv_strides, tq, k.shape[0], B, h_q, k.shape[1], d,
                  _FLOAT16S[q.dtype])
    _launch("hs2_packed_attn", index, stream, ctypes.byref(args), sm_scale, out.data_ptr(),
            _ptr(lse), workspace.data_ptr(), workspace.numel())
    return out, lse
