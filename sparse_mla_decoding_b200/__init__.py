"""B200-native token-level sparse MLA decoding over a paged FP8 KV cache.

Thin Python binding of ``libsmla.so`` (C ABI in ``include/smla.h``): it only
checks shapes, allocates outputs with torch and passes raw device pointers and
the current CUDA stream through ctypes.  Every step of the computation runs in
the library's sm_100a kernels; there is no CPU or PyTorch fallback, and a
missing or unbuildable library raises.

    sched_meta, num_splits = get_mla_metadata(cache_seqlens, topk, h_q, s_q=s_q)
    for layer in layers:                    # the schedule is reused across layers
        o, lse = flash_mla_with_kvcache(q, kvcache, block_table, cache_seqlens,
                                        indices, sched_meta, num_splits)
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Tuple

import torch

from . import build as _build

D_QK, D_V, D_ROPE, KV_ROW_BYTES, BLOCK_SIZE, INDEX_TILE = 576, 512, 64, 656, 64, 64
STATUS_NAMES = {0: "SMLA_OK", 1: "SMLA_ERR_INVALID_ARGUMENT", 2: "SMLA_ERR_UNSUPPORTED", 3: "SMLA_ERR_CUDA",
                4: "SMLA_ERR_DEVICE_TIMEOUT", 5: "SMLA_ERR_SCRATCH_LIMIT"}
# Raw flag bits of the device status word (kernel side, sticky until reset).
STATUS_FLAGS = {1: "a bounded device wait gave up", 2: "a valid index mapped outside the block table or the cache",
                4: "scheduler metadata inconsistent with the call's shapes"}

_lib = None
_lib_lock = threading.Lock()


class SmlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class _Q8Cache(ctypes.Structure):
    """smla_q8_cache."""
    _fields_ = [("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_blocks", ctypes.c_int64), ("k_block_stride", ctypes.c_int64),
                ("v_block_stride", ctypes.c_int64), ("k_scale_stride", ctypes.c_int64),
                ("v_scale_stride", ctypes.c_int64), ("h_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("format", ctypes.c_int)]


def lib() -> ctypes.CDLL:
    """Load libsmla.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    with _lib_lock:
        if _lib is None:
            path = _build.build()
            L = ctypes.CDLL(path)
            vp, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
            L.smla_status_string.argtypes = [i32]
            L.smla_status_string.restype = ctypes.c_char_p
            L.smla_version.argtypes = []
            L.smla_version.restype = i32
            L.smla_last_cuda_error.argtypes = []
            L.smla_last_cuda_error.restype = i32
            L.smla_last_cuda_error_string.argtypes = []
            L.smla_last_cuda_error_string.restype = ctypes.c_char_p
            L.smla_set_head_pair_form.argtypes = [i32]
            L.smla_set_head_pair_form.restype = i32
            L.smla_default_num_sm_parts.argtypes = [i32, i32]
            L.smla_default_num_sm_parts.restype = i32
            L.smla_workspace_bytes.argtypes = [i32, i32, i32, i32, i32]
            L.smla_workspace_bytes.restype = sz
            L.smla_get_mla_metadata.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp]
            L.smla_get_mla_metadata.restype = i32
            L.smla_flash_mla_with_kvcache.argtypes = [vp, vp, i64, vp, i32, vp, vp, vp, vp, i32, f32, i32, i32, i32,
                                                      i32, vp, vp, vp, sz, vp]
            L.smla_flash_mla_with_kvcache.restype = i32
            L.smla_get_mla_metadata_dense.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp]
            L.smla_get_mla_metadata_dense.restype = i32
            L.smla_flash_mla_dense_with_kvcache.argtypes = [vp, vp, i32, i64, vp, i32, vp, vp, vp, vp, i32, f32, i32,
                                                            i32, i32, i32, vp, vp, vp, sz, vp]
            L.smla_flash_mla_dense_with_kvcache.restype = i32
            L.smla_flash_mla_sparse_fwd.argtypes = [vp, vp, i64, vp, i32, i32, i32, i32, f32, vp, vp, vp, sz, vp]
            L.smla_flash_mla_sparse_fwd.restype = i32
            L.smla_sparse_fwd_workspace_bytes.argtypes = [i32, i32, i64, i32, i32]
            L.smla_sparse_fwd_workspace_bytes.restype = sz
            L.smla_quantize_kv.argtypes = [vp, vp, i64, vp, vp, i64, vp]
            L.smla_quantize_kv.restype = i32
            L.smla_extend_block_table.argtypes = [vp, i32, vp, vp, i32, vp, i64, vp, i64, vp, vp, vp, vp, vp]
            L.smla_extend_block_table.restype = i32
            L.smla_quantize_kv_blocks.argtypes = [vp, vp, i64, i64, i64, i64, i64, ctypes.POINTER(_Q8Cache), vp, i32,
                                                  i32, vp, vp, vp, vp, vp]
            L.smla_quantize_kv_blocks.restype = i32
            L.smla_gqa_workspace_bytes.argtypes = [i32, i32]
            L.smla_gqa_workspace_bytes.restype = sz
            L.smla_gqa_attention_with_kvcache.argtypes = [vp, i64, i64, i64, i32, ctypes.POINTER(_Q8Cache), vp, i32,
                                                          i32, vp, vp, i32, i32, i32, f32, f32, vp, vp, vp, vp, vp,
                                                          vp, sz, vp, vp]
            L.smla_gqa_attention_with_kvcache.restype = i32
            L.smla_get_device_status.argtypes = [vp, ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_uint32), vp]
            L.smla_get_device_status.restype = i32
            L.smla_reset_device_status.argtypes = [vp, vp]
            L.smla_reset_device_status.restype = i32
            L.smla_selftest_bounded_wait.argtypes = [vp, ctypes.c_uint64, vp]
            L.smla_selftest_bounded_wait.restype = i32
            _lib = L
    return _lib


def _check(rc: int, what: str) -> None:
    if rc != 0:
        if rc == 3:   # SMLA_ERR_CUDA: name the CUDA runtime error behind it
            what = f"{what} ({lib().smla_last_cuda_error_string().decode()})"
        raise SmlaError(rc, what)


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _raw_stream(index: int) -> int:
    """The current stream of device `index` as a cudaStream_t, without the Stream object."""
    return torch._C._cuda_getCurrentRawStream(index)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _require(cond: bool, msg: str) -> None:
    if not cond:
        raise ValueError(msg)


def set_head_pair_form(enable: bool) -> bool:
    """Run 128-head decodes as two-CTA clusters that share dequantised tiles
    (True) or as independent CTAs (False, the default); returns the previous
    setting.  Process-wide; results are bitwise identical either way."""
    return bool(lib().smla_set_head_pair_form(1 if enable else 0))


def default_num_sm_parts(h_q: int, device: Optional[torch.device] = None) -> int:
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    n = lib().smla_default_num_sm_parts(h_q, dev.index if dev.index is not None else torch.cuda.current_device())
    if n < 1:
        raise SmlaError(3, "smla_default_num_sm_parts")
    return n


def workspace_bytes(batch: int, s_q: int, h_q: int, topk: int, num_sm_parts: int) -> int:
    n = lib().smla_workspace_bytes(batch, s_q, h_q, topk, num_sm_parts)
    if n == 0:
        raise SmlaError(1, "smla_workspace_bytes")
    return int(n)


def new_workspace(batch: int, s_q: int, h_q: int, topk: int, num_sm_parts: int,
                  device: Optional[torch.device] = None) -> torch.Tensor:
    """A zeroed workspace buffer (the zeroed header is the device status word)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.zeros(workspace_bytes(batch, s_q, h_q, topk, num_sm_parts), dtype=torch.uint8, device=dev)


_ws_cache: dict = {}
_ws_lock = threading.Lock()


def _ws_key(device: torch.device):
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    return idx, torch.cuda.current_stream(idx).cuda_stream


def _cached_workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """The workspace used when a call passes none: one per (device, current stream).

    When a call needs more room, the buffer is replaced by a larger one and the
    old status header (the sticky device status word) is carried over on the
    stream, so flags raised by earlier calls are not lost.
    """
    key = _ws_key(device)
    with _ws_lock:
        ws = _ws_cache.get(key)
        if ws is None or ws.numel() < nbytes:
            new = torch.zeros(nbytes, dtype=torch.uint8, device=device)
            if ws is not None:
                new[:256].copy_(ws[:256])
            ws = new
            _ws_cache[key] = ws
    return ws


def cached_workspace_status(device: Optional[torch.device] = None) -> Tuple[int, int]:
    """(status, raw flags) of the device status word of the workspace that calls
    without a `workspace` argument share on `device` and the current stream.

    Kernels record skipped bad block-table entries, inconsistent scheduler
    metadata and bounded waits that gave up there; the flags stay set until
    reset_cached_workspace_status.  Synchronises the current stream.
    (0, 0) if no such call has run yet.
    """
    with _ws_lock:
        ws = _ws_cache.get(_ws_key(device))
    if ws is None:
        return 0, 0
    return get_device_status(ws)


def reset_cached_workspace_status(device: Optional[torch.device] = None) -> None:
    """Clear the status word of the shared workspace on `device` and the current stream."""
    with _ws_lock:
        ws = _ws_cache.get(_ws_key(device))
    if ws is not None:
        reset_device_status(ws)


def _raise_on_flags(workspace: torch.Tensor, what: str) -> None:
    st, raw = get_device_status(workspace)
    if st != 0:
        why = "; ".join(v for k, v in STATUS_FLAGS.items() if raw & k) or f"flags {raw:#x}"
        raise SmlaError(st, f"{what} (device status: {why})")


def get_mla_metadata(cache_seqlens: torch.Tensor, topk: int, h_q: int, num_sm_parts: Optional[int] = None,
                     s_q: int = 1) -> Tuple[torch.Tensor, torch.Tensor]:
    """Tile-scheduler metadata for batch = len(cache_seqlens) requests of s_q query tokens.

    Returns (sched_meta int32 [num_sm_parts, 8], num_splits int32 [batch*s_q + 1]).
    """
    _require(cache_seqlens.is_cuda and cache_seqlens.dtype == torch.int32 and cache_seqlens.dim() == 1,
             "cache_seqlens must be a 1-D int32 CUDA tensor")
    dev = cache_seqlens.device
    if num_sm_parts is None:
        num_sm_parts = default_num_sm_parts(h_q, dev)
    batch = cache_seqlens.shape[0]
    sched_meta = torch.empty((num_sm_parts, 8), dtype=torch.int32, device=dev)
    num_splits = torch.empty((batch * s_q + 1,), dtype=torch.int32, device=dev)
    rc = lib().smla_get_mla_metadata(_ptr(cache_seqlens.contiguous()), batch, s_q, int(topk), int(h_q),
                                     int(num_sm_parts), _ptr(sched_meta), _ptr(num_splits), _stream(dev))
    _check(rc, "smla_get_mla_metadata")
    return sched_meta, num_splits


def flash_mla_with_kvcache(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor,
                           cache_seqlens: torch.Tensor, indices: torch.Tensor, sched_meta: torch.Tensor,
                           num_splits: torch.Tensor, softmax_scale: Optional[float] = None,
                           workspace: Optional[torch.Tensor] = None,
                           out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                           check_device_status: bool = False
                           ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sparse MLA decode: returns (o bf16 [b, s_q, h_q, 512], lse float32 [b, s_q, h_q]).

    q: bf16 [b, s_q, h_q, 576]; kvcache: uint8 [num_blocks, 64, (1,) 656];
    block_table: int32 [b, max_blocks]; cache_seqlens: int32 [b];
    indices: int32 [b, s_q, topk] (negative or >= seqlen = skip);
    sched_meta / num_splits from get_mla_metadata with the same shapes.
    Device-side problems (a valid index whose block lies outside the block
    table or the cache, inconsistent metadata, a wait that gave up) set flags
    in the workspace's status word: read them with get_device_status(workspace),
    or with cached_workspace_status() when no workspace was passed.
    check_device_status=True synchronises after the call and raises SmlaError
    if any flag is set.
    """
    _require(q.is_cuda and q.dtype == torch.bfloat16 and q.dim() == 4 and q.shape[-1] == D_QK,
             "q must be a bf16 CUDA tensor [b, s_q, h_q, 576]")
    b, s_q, h_q, _ = q.shape
    _require(kvcache.dtype == torch.uint8 and kvcache.shape[-1] == KV_ROW_BYTES and kvcache.shape[1] == BLOCK_SIZE,
             "kvcache must be uint8 [num_blocks, 64, (1,) 656]")
    _require(indices.dtype == torch.int32 and indices.dim() == 3 and tuple(indices.shape[:2]) == (b, s_q),
             "indices must be int32 [b, s_q, topk]")
    _require(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == b,
             "block_table must be int32 [b, max_blocks]")
    _require(cache_seqlens.dtype == torch.int32 and tuple(cache_seqlens.shape) == (b,),
             "cache_seqlens must be int32 [b]")
    _require(sched_meta.dtype == torch.int32 and sched_meta.dim() == 2 and sched_meta.shape[1] == 8,
             "sched_meta must be int32 [num_sm_parts, 8]")
    _require(num_splits.dtype == torch.int32 and tuple(num_splits.shape) == (b * s_q + 1,),
             "num_splits must be int32 [b*s_q + 1]")
    for name, t in (("kvcache", kvcache), ("block_table", block_table), ("cache_seqlens", cache_seqlens),
                    ("indices", indices), ("sched_meta", sched_meta), ("num_splits", num_splits)):
        _require(t.is_cuda and t.device == q.device, f"{name} must be on {q.device}")
        _require(t.is_contiguous(), f"{name} must be contiguous")
    q = q.contiguous()
    topk = indices.shape[2]
    num_sm_parts = sched_meta.shape[0]
    dev = q.device
    nbytes = workspace_bytes(b, s_q, h_q, topk, num_sm_parts)
    if workspace is None:
        workspace = _cached_workspace(dev, nbytes)
    _require(workspace.is_cuda and workspace.numel() * workspace.element_size() >= nbytes,
             f"workspace needs {nbytes} bytes")
    if out is None:
        o = torch.empty((b, s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    else:
        o, lse = out
    scale = -1.0 if softmax_scale is None else float(softmax_scale)
    rc = lib().smla_flash_mla_with_kvcache(
        _ptr(q), _ptr(kvcache), kvcache.shape[0], _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        _ptr(indices), _ptr(sched_meta), _ptr(num_splits), num_sm_parts, scale, b, s_q, h_q, topk, _ptr(o),
        _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "smla_flash_mla_with_kvcache")
    if check_device_status:
        _raise_on_flags(workspace, "smla_flash_mla_with_kvcache")
    return o, lse


KV_FP8, KV_BF16 = 0, 1
BF16_ROW_BYTES = 1152


def get_mla_metadata_dense(cache_seqlens: torch.Tensor, h_q: int, s_q: int = 1, causal: bool = True,
                           num_sm_parts: Optional[int] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Scheduler metadata of a dense decode, split by the requests' visible lengths.

    Returns (sched_meta int32 [num_sm_parts, 8], num_splits int32 [b*s_q + 1],
    tile_prefix int32 [b*s_q + 1]); reusable across layers while the lengths stay.
    """
    _require(cache_seqlens.is_cuda and cache_seqlens.dtype == torch.int32 and cache_seqlens.dim() == 1,
             "cache_seqlens must be a 1-D int32 CUDA tensor")
    dev = cache_seqlens.device
    if num_sm_parts is None:
        num_sm_parts = default_num_sm_parts(h_q, dev)
    R = cache_seqlens.shape[0] * s_q
    sched_meta = torch.empty((num_sm_parts, 8), dtype=torch.int32, device=dev)
    num_splits = torch.empty((R + 1,), dtype=torch.int32, device=dev)
    tile_prefix = torch.empty((R + 1,), dtype=torch.int32, device=dev)
    rc = lib().smla_get_mla_metadata_dense(_ptr(cache_seqlens.contiguous()), cache_seqlens.shape[0], int(s_q), int(h_q),
                                           1 if causal else 0, int(num_sm_parts), _ptr(sched_meta), _ptr(num_splits),
                                           _ptr(tile_prefix), _stream(dev))
    _check(rc, "smla_get_mla_metadata_dense")
    return sched_meta, num_splits, tile_prefix


def _kv_format(kvcache: torch.Tensor) -> int:
    if kvcache.dtype == torch.uint8 and kvcache.shape[-1] == KV_ROW_BYTES:
        return KV_FP8
    if kvcache.dtype == torch.uint8 and kvcache.shape[-1] == BF16_ROW_BYTES:
        return KV_BF16
    if kvcache.dtype == torch.bfloat16 and kvcache.shape[-1] == D_QK:
        return KV_BF16
    raise ValueError("kvcache must be uint8 [..., 656] (FP8 rows), or bf16 [..., 576] / uint8 [..., 1152] (BF16 rows)")


def flash_mla_dense_with_kvcache(q: torch.Tensor, kvcache: torch.Tensor, block_table: torch.Tensor,
                                 cache_seqlens: torch.Tensor, sched_meta: torch.Tensor, num_splits: torch.Tensor,
                                 tile_prefix: torch.Tensor, causal: bool = True,
                                 softmax_scale: Optional[float] = None, workspace: Optional[torch.Tensor] = None,
                                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                                 check_device_status: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Dense MLA decode: every query token attends to all its visible cache tokens.

    q: bf16 [b, s_q, h_q, 576]; kvcache: paged [num_blocks, 64, (1,) row] with FP8
    rows (uint8, 656 bytes) or BF16 rows (bf16 576 values, or uint8 1152 bytes);
    block_table: int32 [b, max_blocks]; cache_seqlens: int32 [b]; sched_meta /
    num_splits / tile_prefix from get_mla_metadata_dense with the same lengths,
    s_q and causal.  With causal=True token t of s_q sees the first
    seqlen - (s_q - 1 - t) cache positions.  Returns (o bf16 [b, s_q, h_q, 512],
    lse float32 [b, s_q, h_q]).
    """
    _require(q.is_cuda and q.dtype == torch.bfloat16 and q.dim() == 4 and q.shape[-1] == D_QK,
             "q must be a bf16 CUDA tensor [b, s_q, h_q, 576]")
    b, s_q, h_q, _ = q.shape
    fmt = _kv_format(kvcache)
    _require(kvcache.shape[1] == BLOCK_SIZE and kvcache.is_contiguous(), "kvcache must be contiguous [num_blocks, 64, ...]")
    _require(block_table.dtype == torch.int32 and block_table.dim() == 2 and block_table.shape[0] == b,
             "block_table must be int32 [b, max_blocks]")
    _require(cache_seqlens.dtype == torch.int32 and tuple(cache_seqlens.shape) == (b,),
             "cache_seqlens must be int32 [b]")
    _require(sched_meta.dtype == torch.int32 and sched_meta.dim() == 2 and sched_meta.shape[1] == 8,
             "sched_meta must be int32 [num_sm_parts, 8]")
    for name, t in (("num_splits", num_splits), ("tile_prefix", tile_prefix)):
        _require(t.dtype == torch.int32 and tuple(t.shape) == (b * s_q + 1,), f"{name} must be int32 [b*s_q + 1]")
    for name, t in (("kvcache", kvcache), ("block_table", block_table), ("cache_seqlens", cache_seqlens),
                    ("sched_meta", sched_meta), ("num_splits", num_splits), ("tile_prefix", tile_prefix)):
        _require(t.is_cuda and t.device == q.device, f"{name} must be on {q.device}")
        _require(t.is_contiguous(), f"{name} must be contiguous")
    q = q.contiguous()
    num_sm_parts = sched_meta.shape[0]
    dev = q.device
    nbytes = workspace_bytes(b, s_q, h_q, 1, num_sm_parts)
    if workspace is None:
        workspace = _cached_workspace(dev, nbytes)
    _require(workspace.is_cuda and workspace.numel() * workspace.element_size() >= nbytes,
             f"workspace needs {nbytes} bytes")
    if out is None:
        o = torch.empty((b, s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((b, s_q, h_q), dtype=torch.float32, device=dev)
    else:
        o, lse = out
    scale = -1.0 if softmax_scale is None else float(softmax_scale)
    rc = lib().smla_flash_mla_dense_with_kvcache(
        _ptr(q), _ptr(kvcache), fmt, kvcache.shape[0], _ptr(block_table), block_table.shape[1], _ptr(cache_seqlens),
        _ptr(sched_meta), _ptr(num_splits), _ptr(tile_prefix), num_sm_parts, scale, 1 if causal else 0, b, s_q, h_q,
        _ptr(o), _ptr(lse), _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "smla_flash_mla_dense_with_kvcache")
    if check_device_status:
        _raise_on_flags(workspace, "smla_flash_mla_dense_with_kvcache")
    return o, lse


def sparse_fwd_workspace_bytes(s_q: int, h_q: int, s_kv: int, topk: int, num_sm_parts: int) -> int:
    n = lib().smla_sparse_fwd_workspace_bytes(s_q, h_q, s_kv, topk, num_sm_parts)
    if n == 0:
        raise SmlaError(1, "smla_sparse_fwd_workspace_bytes")
    return int(n)


def flash_mla_sparse_fwd(q: torch.Tensor, kv: torch.Tensor, indices: torch.Tensor,
                         softmax_scale: Optional[float] = None, num_sm_parts: Optional[int] = None,
                         workspace: Optional[torch.Tensor] = None,
                         out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                         check_device_status: bool = False
                         ) -> Tuple[torch.Tensor, torch.Tensor]:
    """Sparse attention of s_q query tokens over one flat FP8 cache: (o bf16 [s_q, h_q, 512], lse [s_q, h_q]).

    q: bf16 [s_q, h_q, 576]; kv: uint8 [s_kv, (1,) 656] (656-byte rows, one KV head);
    indices: int32 [s_q, 1, topk] (or [s_q, topk]), negative or >= s_kv = skip.
    A workspace from new_sparse_fwd_workspace may be passed; its first 256 bytes are
    the device status word (get_device_status).
    """
    _require(q.is_cuda and q.dtype == torch.bfloat16 and q.dim() == 3 and q.shape[-1] == D_QK,
             "q must be a bf16 CUDA tensor [s_q, h_q, 576]")
    s_q, h_q, _ = q.shape
    _require(kv.dtype == torch.uint8 and kv.shape[-1] == KV_ROW_BYTES and kv.dim() in (2, 3) and
             (kv.dim() == 2 or kv.shape[1] == 1), "kv must be uint8 [s_kv, (1,) 656]")
    _require(indices.dtype == torch.int32 and indices.shape[0] == s_q and
             (indices.dim() == 2 or (indices.dim() == 3 and indices.shape[1] == 1)),
             "indices must be int32 [s_q, 1, topk] or [s_q, topk]")
    for name, t in (("kv", kv), ("indices", indices)):
        _require(t.is_cuda and t.device == q.device, f"{name} must be on {q.device}")
        _require(t.is_contiguous(), f"{name} must be contiguous")
    q = q.contiguous()
    s_kv = kv.shape[0]
    topk = indices.shape[-1]
    dev = q.device
    if num_sm_parts is None:
        num_sm_parts = default_num_sm_parts(h_q, dev)
    nbytes = sparse_fwd_workspace_bytes(s_q, h_q, s_kv, topk, num_sm_parts)
    if workspace is None:
        workspace = _cached_workspace(dev, nbytes)
    _require(workspace.is_cuda and workspace.numel() * workspace.element_size() >= nbytes,
             f"workspace needs {nbytes} bytes")
    if out is None:
        o = torch.empty((s_q, h_q, D_V), dtype=torch.bfloat16, device=dev)
        lse = torch.empty((s_q, h_q), dtype=torch.float32, device=dev)
    else:
        o, lse = out
    scale = -1.0 if softmax_scale is None else float(softmax_scale)
    rc = lib().smla_flash_mla_sparse_fwd(_ptr(q), _ptr(kv), s_kv, _ptr(indices), s_q, h_q, topk, int(num_sm_parts),
                                         scale, _ptr(o), _ptr(lse), _ptr(workspace),
                                         workspace.numel() * workspace.element_size(), _stream(dev))
    _check(rc, "smla_flash_mla_sparse_fwd")
    if check_device_status:
        _raise_on_flags(workspace, "smla_flash_mla_sparse_fwd")
    return o, lse


def new_sparse_fwd_workspace(s_q: int, h_q: int, s_kv: int, topk: int, num_sm_parts: int,
                             device: Optional[torch.device] = None) -> torch.Tensor:
    """A zeroed workspace for flash_mla_sparse_fwd (the zeroed header is the device status word)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    return torch.zeros(sparse_fwd_workspace_bytes(s_q, h_q, s_kv, topk, num_sm_parts), dtype=torch.uint8,
                       device=dev)


def quantize_kv(latent: torch.Tensor, rope: torch.Tensor, kvcache: torch.Tensor,
                slot_mapping: Optional[torch.Tensor] = None) -> None:
    """Write tokens (bf16 latent [n, 512] and rope [n, 64]) into 656-byte FP8 rows of kvcache."""
    _require(latent.is_cuda and latent.dtype == torch.bfloat16 and latent.dim() == 2 and latent.shape[1] == D_V,
             "latent must be bf16 [n, 512] on CUDA")
    _require(rope.dtype == torch.bfloat16 and tuple(rope.shape) == (latent.shape[0], D_ROPE),
             "rope must be bf16 [n, 64]")
    _require(kvcache.dtype == torch.uint8 and kvcache.shape[-1] == KV_ROW_BYTES and kvcache.is_contiguous(),
             "kvcache must be contiguous uint8 [..., 656]")
    if slot_mapping is not None:
        _require(slot_mapping.dtype == torch.int64 and tuple(slot_mapping.shape) == (latent.shape[0],),
                 "slot_mapping must be int64 [n]")
        slot_mapping = slot_mapping.contiguous()
    latent, rope = latent.contiguous(), rope.contiguous()
    num_rows = kvcache.numel() // KV_ROW_BYTES
    rc = lib().smla_quantize_kv(_ptr(latent), _ptr(rope), latent.shape[0], _ptr(slot_mapping), _ptr(kvcache),
                                num_rows, _stream(latent.device))
    _check(rc, "smla_quantize_kv")


# ---------------------------------------------------------------------------
# paged serving of grouped-query attention: block tables, the block-scaled 8-bit
# cache and attention over it
# ---------------------------------------------------------------------------
_paged_words: dict = {}


def _paged_word(index: int) -> Optional[torch.Tensor]:
    """The status word that the paged calls on a device share when they get no workspace.

    Made by the first such call; a graph captured before that reports nowhere
    (an allocation inside the capture would belong to the graph)."""
    w = _paged_words.get(index)
    if w is None and not _capturing(index):
        with _ws_lock:
            w = _paged_words.get(index)
            if w is None:
                dev = torch.device("cuda", index)
                w = torch.zeros(64, dtype=torch.int32, device=dev)
                torch.cuda.current_stream(dev).synchronize()    # other streams may use it next
                _paged_words[index] = w
    return w


def _capturing(index: int) -> bool:
    with torch.cuda.device(index):
        return torch.cuda.is_current_stream_capturing()


def _paged_key(device: Optional[torch.device]) -> int:
    dev = torch.device("cuda") if device is None else torch.device(device)
    return dev.index if dev.index is not None else torch.cuda.current_device()


def paged_status(device: Optional[torch.device] = None) -> Tuple[int, int]:
    """(status, raw flags) of quantize_kv_blocks and gqa_attention_with_kvcache calls on
    `device` that were given no workspace (see STATUS_FLAGS; sticky until
    reset_paged_status).  Synchronises the current stream; (0, 0) before any such call."""
    with _ws_lock:
        w = _paged_words.get(_paged_key(device))
    return (0, 0) if w is None else get_device_status(w)


def reset_paged_status(device: Optional[torch.device] = None) -> None:
    """Clear the status word that paged_status reads (on the current stream)."""
    with _ws_lock:
        w = _paged_words.get(_paged_key(device))
    if w is not None:
        reset_device_status(w)


# Single-token steps run in a few microseconds on the GPU, so these checks are
# written to cost little where they pass: messages are only put together to be raised.
def _bad(msg: str) -> None:
    raise ValueError(msg)


def _i32_vector(t: torch.Tensor, n: int, name: str, index: int) -> torch.Tensor:
    if t.dtype != torch.int32 or t.shape != (n,) or t.get_device() != index:
        _bad(f"{name} must be int32 [{n}] on cuda:{index}")
    return t if t.is_contiguous() else t.contiguous()


def _block_table(t: torch.Tensor, index: int) -> Tuple[int, int]:
    if t.dtype != torch.int32 or t.dim() != 2 or t.get_device() != index or not t.is_contiguous() or t.shape[1] < 1:
        _bad(f"block_table must be contiguous int32 [b, max_blocks] on cuda:{index}")
    return t.shape


def _on_device(index: int, call, *args) -> int:
    """call(*args) with device `index` current."""
    back = torch._C._cuda_getDevice()
    if back == index:
        return call(*args)
    torch.cuda.set_device(index)
    try:
        return call(*args)
    finally:
        torch.cuda.set_device(back)


def extend_block_table(block_table: torch.Tensor, cache_seqlens: torch.Tensor, new_lens: torch.Tensor,
                       free_blocks: torch.Tensor, num_free: torch.Tensor, max_new_tokens: int
                       ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Blocks and cache rows for the new tokens of a step, without a host copy of the lengths.

    block_table: int32 [b, max_blocks], fresh entries written in place;
    cache_seqlens, new_lens: int32 [b], tokens held and tokens to add;
    free_blocks: int32 [capacity] whose first num_free (int32 [1]) entries are free,
    taken from the end; max_new_tokens: length of the slot map.
    Returns (slot_mapping int64 [max_new_tokens], cu_new int32 [b + 1], the lengths with
    the new tokens int32 [b], entries left on the free list int32 [1]).  A request whose
    blocks or tokens do not fit is declined: it keeps its length, and its tokens get slots
    -1, which quantize_kv skips.  cu_new counts them all the same; quantize_kv_blocks leaves
    such a request alone, and what gqa_attention_with_kvcache returns for its rows means
    nothing.  Where a request ends or gets shorter (rejected draft tokens), put its table
    entries from ceil(length / 64) on behind the first num_free of free_blocks and raise
    num_free before the next call, which overwrites them: nothing else gives blocks back.
    slot_mapping goes to quantize_kv; cu_new and the lengths go to quantize_kv_blocks
    and the attention calls.
    """
    if not block_table.is_cuda:
        _bad("block_table must be int32 [b, max_blocks] on CUDA")
    index = block_table.get_device()
    b, cols = _block_table(block_table, index)
    cache_seqlens = _i32_vector(cache_seqlens, b, "cache_seqlens", index)
    new_lens = _i32_vector(new_lens, b, "new_lens", index)
    num_free = _i32_vector(num_free, 1, "num_free", index)
    if free_blocks.dim() != 1:
        _bad("free_blocks must be int32 [capacity]")
    capacity = free_blocks.shape[0]
    free_blocks = _i32_vector(free_blocks, capacity, "free_blocks", index)
    n = int(max_new_tokens)
    if not 0 <= n < 1 << 31:
        _bad("max_new_tokens must be in [0, 2^31)")
    slots = block_table.new_empty(n, dtype=torch.int64)
    cu_new, lens, left = block_table.new_empty(b + 1), block_table.new_empty(b), block_table.new_empty(1)
    rc = _on_device(index, lib().smla_extend_block_table, block_table.data_ptr(), cols, cache_seqlens.data_ptr(),
                    new_lens.data_ptr(), b, free_blocks.data_ptr(), capacity, num_free.data_ptr(), n,
                    slots.data_ptr(), cu_new.data_ptr(), lens.data_ptr(), left.data_ptr(), _raw_stream(index))
    if rc:
        _check(rc, "smla_extend_block_table")
    return slots, cu_new, lens, left


_Q8_FORMATS = {torch.float8_e4m3fn: 0, torch.int8: 1}


def _q8_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor) -> _Q8Cache:
    fmt = _Q8_FORMATS.get(k_cache.dtype)
    shape, index = k_cache.shape, k_cache.get_device()
    if fmt is None or len(shape) != 4 or index < 0 or shape[2] != BLOCK_SIZE or shape[3] not in (64, 128):
        _bad("k_cache must be e4m3 or int8 [num_blocks, h_kv, 64, 64 or 128] on CUDA")
    nb, h_kv, _, d = shape
    ks, vs, kss, vss = k_cache.stride(), v_cache.stride(), k_scale.stride(), v_scale.stride()
    if v_cache.dtype != k_cache.dtype or v_cache.shape != shape or v_cache.get_device() != index:
        _bad("v_cache must match k_cache's type, shape and device")
    inside = (BLOCK_SIZE * d, d, 1)
    if (ks[1:] != inside or vs[1:] != inside) and (h_kv > 1 or ks[2:] != inside[1:] or vs[2:] != inside[1:]):
        _bad("k_cache and v_cache must be dense within a block")
    rows = (nb, h_kv)
    for name, t, st in (("k_scale", k_scale, kss), ("v_scale", v_scale, vss)):
        if t.dtype != torch.float32 or t.shape != rows or t.get_device() != index or (st[1] != 1 and h_kv > 1):
            _bad(f"{name} must be float32 [num_blocks, h_kv] on cuda:{index}")
    if nb == 1:                      # a lone block's stride is free to say anything
        ks = vs = (h_kv * BLOCK_SIZE * d,)
        kss = vss = (h_kv,)
    return _Q8Cache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), nb, ks[0], vs[0],
                    kss[0], vss[0], h_kv, d, fmt)


def _rows16(t: torch.Tensor, n: int, h: int, d: int) -> Tuple[torch.Tensor, int, int]:
    """t [.., h, d] of n tokens with dense rows that 16-byte loads can read (a copy where it
    has none), and the strides of its tokens and heads."""
    s = t.stride()
    if len(s) == 3:
        a, b, c = s
    else:                            # [requests, tokens each, h, d]
        r, a, b, c = s
        each = t.shape[1]
        if each == 1:
            a = r
        elif r != each * a and n > each:
            c = 0                    # no one stride leads through the tokens
    if (a | b) & 7:                  # a lone token's or head's stride is free to say anything
        a, b = h * d if n == 1 else a, d if h == 1 else b
    if c == 1 and not (a | b) & 7 and not t.data_ptr() & 15:
        return t, a, b
    return t.clone(memory_format=torch.contiguous_format), h * d, d


_gqa_bytes: dict = {}                # (head_dim, device): fixed by the device


def _gqa_workspace(d: int, index: int) -> int:
    n = _gqa_bytes.get((d, index))
    if n is None:
        n = _gqa_bytes[d, index] = lib().smla_gqa_workspace_bytes(d, index)
    return n


def quantize_kv_blocks(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                       k_scale: torch.Tensor, v_scale: torch.Tensor, block_table: torch.Tensor,
                       cache_seqlens: torch.Tensor, new_seqlens: torch.Tensor, cu_new: torch.Tensor,
                       check_device_status: bool = False) -> None:
    """Write new tokens into a block-scaled 8-bit cache.

    k, v: bf16 [total, h_kv, d], the tokens cu_new[r] .. cu_new[r + 1] - 1 of request r
    (strided views of a fused projection are read in place); k_cache, v_cache: e4m3
    (torch.float8_e4m3fn) or int8 [num_blocks, h_kv, 64, d], dense within a block;
    k_scale, v_scale: float32 [num_blocks, h_kv]; block_table: int32 [b, max_blocks];
    cache_seqlens, new_seqlens: int32 [b], the lengths before and with the tokens;
    cu_new: int32 [b + 1].  A (block, head)'s scale is the smallest power of two at which
    its values fit the code range, and never shrinks while the block fills: where new
    tokens raise it, the block's older codes are rescaled.  A request whose lengths do
    not differ by its token count (extend_block_table found no room) is left alone.  No
    two requests may write to the same block.  Problems found on the device are flagged:
    paged_status(), or check_device_status=True to synchronise and raise.
    """
    cache = _q8_cache(k_cache, v_cache, k_scale, v_scale)
    index = k_cache.get_device()
    shape = (k.shape[0], cache.h_kv, cache.head_dim)
    for name, t in (("k", k), ("v", v)):
        if t.dtype != torch.bfloat16 or t.shape != shape or t.get_device() != index:
            _bad(f"{name} must be bf16 [total, {cache.h_kv}, {cache.head_dim}] on cuda:{index}")
    b, cols = _block_table(block_table, index)
    cache_seqlens = _i32_vector(cache_seqlens, b, "cache_seqlens", index)
    new_seqlens = _i32_vector(new_seqlens, b, "new_seqlens", index)
    cu_new = _i32_vector(cu_new, b + 1, "cu_new", index)
    k, kts, khs = _rows16(k, *shape)
    v, vts, vhs = _rows16(v, *shape)
    word = _paged_word(index)
    rc = _on_device(index, lib().smla_quantize_kv_blocks, k.data_ptr(), v.data_ptr(), kts, khs, vts, vhs,
                    shape[0], ctypes.byref(cache), block_table.data_ptr(), cols, b, cache_seqlens.data_ptr(),
                    new_seqlens.data_ptr(), cu_new.data_ptr(), _ptr(word), _raw_stream(index))
    if rc:
        _check(rc, "smla_quantize_kv_blocks")
    if check_device_status and word is not None:
        _raise_on_flags(word, "smla_quantize_kv_blocks")


def gqa_workspace_bytes(head_dim: int, device: Optional[torch.device] = None) -> int:
    n = lib().smla_gqa_workspace_bytes(int(head_dim), _paged_key(device))
    if n == 0:
        raise SmlaError(1, "smla_gqa_workspace_bytes")
    return int(n)


def new_gqa_workspace(head_dim: int, device: Optional[torch.device] = None) -> torch.Tensor:
    """A workspace for gqa_attention_with_kvcache: a zeroed 256-byte header (the device
    status word), then the split partials."""
    return torch.zeros(256 + gqa_workspace_bytes(head_dim, device), dtype=torch.uint8,
                       device=torch.device("cuda", _paged_key(device)))


def gqa_attention_with_kvcache(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: torch.Tensor,
                               v_scale: torch.Tensor, block_table: torch.Tensor, cache_seqlens: torch.Tensor,
                               cu_seqlens_q: Optional[torch.Tensor] = None, max_seqlen_q: Optional[int] = None,
                               causal: bool = True, softmax_scale: Optional[float] = None, softcap: float = 0.0,
                               alibi_slopes: Optional[torch.Tensor] = None,
                               prefix_lens: Optional[torch.Tensor] = None,
                               doc_bounds: Optional[torch.Tensor] = None,
                               workspace: Optional[torch.Tensor] = None,
                               out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                               check_device_status: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """Grouped-query attention over a block-scaled 8-bit cache (see quantize_kv_blocks).

    q: bf16 [b, s_q, h_q, d], or [total_q, h_q, d] with cu_seqlens_q int32 [b + 1]; a
    request's query tokens are its last positions and are already in the cache, so
    cache_seqlens (int32 [b]) counts them (throw the rows of a request away whose tokens
    extend_block_table declined: they are taken for its last positions too).  One new token
    per request, several, or whole prompts: max_seqlen_q (the most query tokens of a
    request; total_q if not given) only helps to pick the kernel (above total_q: the one
    for long prompts).
    Scores are softmax_scale * <q, k> (default 1/sqrt(d)), then softcap * tanh(x / softcap)
    with softcap > 0, then minus alibi_slopes[h] * distance (float32 [h_q]).
    A token at position p sees j <= p (causal), every j < prefix_lens[r] as well (int32
    [b]), and with doc_bounds (int32 [total_q, 2]) only first <= j < end of its own
    document.  Returns (o bf16 as q, lse float32 [b, s_q, h_q] or [total_q, h_q]); 0 and
    -inf where a token sees nothing.  Rows of q behind the last request are not read and
    their outputs not written.
    A workspace from new_gqa_workspace may be passed; its first 256 bytes are the device
    status word.  Without one, scratch comes from torch's allocator (a captured graph
    keeps its own) and flags go to paged_status().
    """
    cache = _q8_cache(k_cache, v_cache, k_scale, v_scale)
    index, d = k_cache.get_device(), cache.head_dim
    shape = q.shape
    if (q.dtype != torch.bfloat16 or q.get_device() != index or len(shape) != (4 if cu_seqlens_q is None else 3) or
            shape[-1] != d):
        _bad(f"q must be bf16 [b, s_q, h_q, {d}], or [total_q, h_q, {d}] with cu_seqlens_q, on cuda:{index}")
    b, cols = _block_table(block_table, index)
    h_q = shape[-2]
    if h_q < 1 or h_q % cache.h_kv:
        _bad("h_q must be a multiple of h_kv")
    s_q, cu, total = 0, None, shape[0]
    if cu_seqlens_q is None:
        if shape[0] != b:
            _bad(f"q must hold {b} requests")
        s_q = shape[1]
        total = b * s_q
        if max_seqlen_q is None:
            max_seqlen_q = s_q
    else:
        cu_seqlens_q = _i32_vector(cu_seqlens_q, b + 1, "cu_seqlens_q", index)
        cu = cu_seqlens_q.data_ptr()
    rows, q_tok, q_head = _rows16(q, total, h_q, d)
    cache_seqlens = _i32_vector(cache_seqlens, b, "cache_seqlens", index)
    if alibi_slopes is not None:
        if alibi_slopes.dtype != torch.float32 or alibi_slopes.shape != (h_q,) or alibi_slopes.get_device() != index:
            _bad(f"alibi_slopes must be float32 [{h_q}] on cuda:{index}")
        alibi_slopes = alibi_slopes.contiguous()
    if prefix_lens is not None:
        if not causal:
            _bad("prefix_lens needs causal=True")
        prefix_lens = _i32_vector(prefix_lens, b, "prefix_lens", index)
    if doc_bounds is not None:
        if doc_bounds.dtype != torch.int32 or doc_bounds.shape != (total, 2) or doc_bounds.get_device() != index:
            _bad(f"doc_bounds must be int32 [{total}, 2] on cuda:{index}")
        doc_bounds = doc_bounds.contiguous()
        if doc_bounds.data_ptr() % 8:
            doc_bounds = doc_bounds.clone()
    softcap = float(softcap)
    if softcap != 0.0 and not 2.0 ** -60 <= softcap <= 2.0 ** 60:
        _bad("softcap must be 0 or from 2^-60 to 2^60")
    scale = -1.0
    if softmax_scale is not None:
        scale = float(softmax_scale)
        if not 2.0 ** -126 <= scale < 2.0 ** 127:
            _bad("softmax_scale must be > 0 and finite (as a normal float32)")
    if out is None:
        o, lse = torch.empty_like(q, memory_format=torch.contiguous_format), k_scale.new_empty(*shape[:-1])
    else:
        o, lse = out
        for name, t, dt, sh in (("o", o, torch.bfloat16, shape), ("lse", lse, torch.float32, shape[:-1])):
            if t.dtype != dt or t.shape != sh or t.get_device() != index or not t.is_contiguous():
                _bad(f"out: {name} must be contiguous {dt} {list(sh)} on cuda:{index}")
        if o.data_ptr() % 16:
            _bad("out: o must be 16-byte aligned")
    nbytes = _gqa_workspace(d, index)
    if workspace is None:
        word, scratch = _paged_word(index), k_scale.new_empty(nbytes // 4)
        at, room = scratch.data_ptr(), nbytes
    else:
        if (workspace.get_device() != index or not workspace.is_contiguous() or workspace.dtype != torch.uint8 or
                workspace.numel() < 256 + nbytes):
            _bad(f"workspace needs {256 + nbytes} bytes of uint8 on cuda:{index}")
        word, at, room = workspace, workspace.data_ptr() + 256, workspace.numel() - 256
    rc = _on_device(
        index, lib().smla_gqa_attention_with_kvcache, rows.data_ptr(), q_tok, q_head, total, h_q,
        ctypes.byref(cache), block_table.data_ptr(), cols, b, cache_seqlens.data_ptr(), cu, s_q,
        total if max_seqlen_q is None else min(int(max_seqlen_q), 0x7FFFFFFF), 1 if causal else 0, scale, softcap,
        _ptr(alibi_slopes), _ptr(prefix_lens), _ptr(doc_bounds), o.data_ptr(), lse.data_ptr(), at, room, _ptr(word),
        _raw_stream(index))
    if rc:
        _check(rc, "smla_gqa_attention_with_kvcache")
    if check_device_status and word is not None:
        _raise_on_flags(word, "smla_gqa_attention_with_kvcache")
    return o, lse


def get_device_status(workspace: torch.Tensor) -> Tuple[int, int]:
    """(status, raw flags) of a workspace's sticky status word; synchronises the current stream."""
    st = ctypes.c_int(0)
    raw = ctypes.c_uint32(0)
    rc = lib().smla_get_device_status(_ptr(workspace), ctypes.byref(st), ctypes.byref(raw), _stream(workspace.device))
    _check(rc, "smla_get_device_status")
    return st.value, raw.value


def reset_device_status(workspace: torch.Tensor) -> None:
    _check(lib().smla_reset_device_status(_ptr(workspace), _stream(workspace.device)), "smla_reset_device_status")


def selftest_bounded_wait(workspace: torch.Tensor, limit_ns: int) -> None:
    _check(lib().smla_selftest_bounded_wait(_ptr(workspace), int(limit_ns), _stream(workspace.device)),
           "smla_selftest_bounded_wait")


def default_softmax_scale() -> float:
    return 1.0 / math.sqrt(D_QK)
