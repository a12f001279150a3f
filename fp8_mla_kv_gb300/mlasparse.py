"""Thin ctypes binding to libmlasparse (include/mlasparse.h), same function names.

Argument marshalling only: torch tensors supply device memory and the current
CUDA stream; every step of the computation runs in the library's kernels. The
library is loaded on first use; if it is missing or no CUDA device is present,
the call raises. There is no fallback path.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import ROW_BYTES, ROW_BYTES_NOPE

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmlasparse.so")

MLA_OK = 0
MLA_EINVAL = -1
MLA_EUNSUPPORTED = -2
MLA_ENOWORKSPACE = -3
MLA_ECUDA = -4
MLA_ERR_WRITE_SLOT_RANGE = 0x1
MLA_ERR_DECODE_INDEX_RANGE = 0x2
MLA_ERR_PIPELINE_TIMEOUT = 0x4
MLA_ERR_GATHER_INDEX_RANGE = 0x8
MLA_ERR_CHUNK_RANGE = 0x10
MLA_ERR_PAGE_RANGE = 0x20
MLA_ERR_PAGE_COUNT = 0x40
MLA_ERR_POOL_EMPTY = 0x80

SYMBOLS = ("mla_kv_write", "mla_sparse_decode", "mla_sparse_decode_workspace_bytes",
           "mla_sparse_decode_paged", "mla_sparse_prefill", "mla_sparse_prefill_paged",
           "mla_gather_upconvert", "mla_rope", "mla_rope_kv_write", "mla_chunk_attention",
           "mla_chunk_attention_workspace_bytes", "mla_block_keys", "mla_block_scores", "mla_block_select",
           "mla_block_attention", "mla_block_attention_workspace_bytes", "mla_tree_mask", "mla_tree_attention",
           "mla_tree_commit", "mla_page_copy", "mla_page_free", "mla_page_fork",
           "mla_page_compact", "mla_page_workspace_bytes", "mla_get_error", "mla_strerror")


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__(f"{what}: {strerror(code)} ({code})")
        self.code = code


class KVCache(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("num_slots", ctypes.c_int64), ("row_bytes", ctypes.c_int64)]


class RopeSpec(ctypes.Structure):
    """mla_rope_t; rope_spec() makes one."""
    _fields_ = [("inv_freq", ctypes.c_double * 32), ("scale", ctypes.c_float), ("n_axes", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32), ("axis", ctypes.c_uint8 * 32)]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library (raises OSError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise OSError(f"libmlasparse not built: {path} is missing "
                              "(run fp8_mla_kv_gb300.build.build() or __graft_entry__.build())")
            lib = ctypes.CDLL(path)
            c = ctypes
            lib.mla_kv_write.restype = c.c_int
            lib.mla_kv_write.argtypes = [KVCache, c.c_void_p, c.c_void_p, c.c_void_p, c.c_int64, c.c_int64,
                                         c.c_void_p]
            lib.mla_sparse_decode_workspace_bytes.restype = c.c_size_t
            lib.mla_sparse_decode_workspace_bytes.argtypes = [c.c_int, c.c_int, c.c_int]
            lib.mla_sparse_decode.restype = c.c_int
            lib.mla_sparse_decode.argtypes = [c.c_void_p, c.c_int, c.c_int, c.c_int, KVCache, c.c_void_p,
                                              c.c_int, c.c_float, c.c_void_p, c.c_void_p, c.c_void_p,
                                              c.c_size_t, c.c_void_p]
            lib.mla_sparse_decode_paged.restype = c.c_int
            lib.mla_sparse_decode_paged.argtypes = [c.c_void_p, c.c_int, c.c_int, c.c_int, KVCache, c.c_void_p,
                                                    c.c_int, c.c_void_p, c.c_int, c.c_int, c.c_void_p, c.c_int,
                                                    c.c_float, c.c_void_p, c.c_void_p, c.c_void_p, c.c_size_t,
                                                    c.c_void_p]
            lib.mla_sparse_prefill.restype = c.c_int
            lib.mla_sparse_prefill.argtypes = [c.c_void_p, c.c_int, c.c_int, c.c_int, KVCache, c.c_void_p,
                                               c.c_int, c.c_float, c.c_void_p, c.c_void_p, c.c_void_p]
            lib.mla_sparse_prefill_paged.restype = c.c_int
            lib.mla_sparse_prefill_paged.argtypes = [c.c_void_p, c.c_int, c.c_int, c.c_int, KVCache, c.c_void_p,
                                                     c.c_int, c.c_void_p, c.c_int, c.c_int, c.c_void_p, c.c_int,
                                                     c.c_float, c.c_void_p, c.c_void_p, c.c_void_p]
            lib.mla_gather_upconvert.restype = c.c_int
            lib.mla_gather_upconvert.argtypes = [KVCache, c.c_void_p, c.c_int64, c.c_int, c.c_void_p, c.c_void_p]
            vp, i32, i64 = c.c_void_p, c.c_int, c.c_int64
            lib.mla_rope.restype = i32
            lib.mla_rope.argtypes = [vp, i64, i64, vp, i64, i64, i64, i32, vp, i64, c.POINTER(RopeSpec), vp]
            lib.mla_rope_kv_write.restype = i32
            lib.mla_rope_kv_write.argtypes = [KVCache, vp, vp, vp, i64, i64, vp, i64, c.POINTER(RopeSpec), vp, i64, i64,
                                              vp, i64, i64, i32, vp]
            lib.mla_chunk_attention_workspace_bytes.restype = c.c_size_t
            lib.mla_chunk_attention_workspace_bytes.argtypes = [i32, i32, i32]
            lib.mla_chunk_attention.restype = i32
            lib.mla_chunk_attention.argtypes = [vp, i32, i32, i32, KVCache, vp, vp, vp, i32, i32, i32, i32, c.c_float,
                                                vp, vp, vp, c.c_size_t, vp]
            lib.mla_block_keys.restype = i32
            lib.mla_block_keys.argtypes = [KVCache, i32, vp, vp, vp, i32, i32, i32, i32, vp, i32, vp]
            lib.mla_block_scores.restype = i32
            lib.mla_block_scores.argtypes = [vp, i32, i32, i32, vp, i32, vp, vp, vp, i32, i32, i32, c.c_float, vp, vp]
            lib.mla_block_select.restype = i32
            lib.mla_block_select.argtypes = [vp, i32, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp]
            lib.mla_block_attention_workspace_bytes.restype = c.c_size_t
            lib.mla_block_attention_workspace_bytes.argtypes = [i32, i32, i32]
            lib.mla_block_attention.restype = i32
            lib.mla_block_attention.argtypes = [vp, i32, i32, i32, KVCache, vp, i32, vp, vp, vp, i32, i32, i32, c.c_float,
                                                vp, vp, vp, c.c_size_t, vp]
            lib.mla_tree_mask.restype = i32
            lib.mla_tree_mask.argtypes = [vp, i32, vp, vp, i32, vp, i32, vp, vp]
            lib.mla_tree_attention.restype = i32
            lib.mla_tree_attention.argtypes = [vp, i32, i32, i32, KVCache, vp, vp, vp, i32, i32, i32, vp, i32, c.c_float,
                                               vp, vp, vp, c.c_size_t, vp]
            lib.mla_tree_commit.restype = i32
            lib.mla_tree_commit.argtypes = [KVCache, vp, vp, vp, i32, i32, i32, vp, vp, i32, vp, vp]
            lib.mla_page_copy.restype = i32
            lib.mla_page_copy.argtypes = [KVCache, KVCache, i32, vp, vp, i64, vp]
            lib.mla_page_free.restype = i32
            lib.mla_page_free.argtypes = [vp, i32, vp, i32, i32, vp, i32, vp]
            lib.mla_page_fork.restype = i32
            lib.mla_page_fork.argtypes = [KVCache, i32, vp, i32, vp, i32, i32, vp, vp, vp, i32, vp, c.c_size_t, vp]
            lib.mla_page_compact.restype = i32
            lib.mla_page_compact.argtypes = [KVCache, i32, vp, vp, i32, vp, vp, i32, i32, vp, vp, c.c_size_t, vp]
            lib.mla_page_workspace_bytes.restype = c.c_size_t
            lib.mla_page_workspace_bytes.argtypes = [i32, i32]
            lib.mla_get_error.restype = c.c_int
            lib.mla_get_error.argtypes = [c.POINTER(c.c_int32)]
            lib.mla_strerror.restype = c.c_char_p
            lib.mla_strerror.argtypes = [c.c_int]
            _lib = lib
    return _lib


def strerror(code: int) -> str:
    try:
        return load().mla_strerror(int(code)).decode()
    except OSError:
        return f"code {code}"


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libmlasparse takes device tensors only")


# The current stream's handle by itself costs a tenth of the Stream object around it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


# The same for the current device, where CUDA is initialised.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None and torch.cuda.is_initialized():
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Where a call's own tensors are made: on its stream, so that they are ordered with its kernels and the allocator
    hands their memory to nothing else before those are done."""
    if stream is None:
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        # (an ExternalStream of 0 would be a new stream, not the default one)
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) != 0 else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


def kv_cache(cache: torch.Tensor) -> KVCache:
    """View a uint8 [num_slots, 656] (or [num_slots, 528] NoPE-only) device tensor
    as the C cache descriptor."""
    shape = cache.shape
    if (cache.dtype is not torch.uint8 or len(shape) != 2 or (shape[1] != ROW_BYTES and shape[1] != ROW_BYTES_NOPE)
            or not cache.is_contiguous()):
        raise ValueError("cache must be a contiguous uint8 tensor [num_slots, 656] or [num_slots, 528]")
    return KVCache(cache.data_ptr(), shape[0], shape[1])


def mla_kv_write(cache: torch.Tensor, slot_idx: torch.Tensor, latent: torch.Tensor,
                 rope: torch.Tensor | None, reserved_slot: int = 0, stream=None) -> None:
    _require_cuda(cache, slot_idx, latent, rope)
    n = int(slot_idx.shape[0])
    assert slot_idx.dtype == torch.int64 and slot_idx.is_contiguous()
    assert latent.dtype == torch.bfloat16 and latent.is_contiguous() and latent.numel() == n * 512
    if rope is not None:
        assert rope.dtype == torch.bfloat16 and rope.is_contiguous() and rope.numel() == n * 64
    rc = load().mla_kv_write(kv_cache(cache), slot_idx.data_ptr(), latent.data_ptr(),
                             rope.data_ptr() if rope is not None else None, n, int(reserved_slot),
                             _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_kv_write")


def mla_sparse_decode_workspace_bytes(T: int, H: int, W: int) -> int:
    return int(load().mla_sparse_decode_workspace_bytes(int(T), int(H), int(W)))


def alloc_workspace(T: int, H: int, W: int, device=None) -> torch.Tensor | None:
    n = mla_sparse_decode_workspace_bytes(T, H, W)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def mla_sparse_decode(q: torch.Tensor, cache: torch.Tensor, topk_idx: torch.Tensor, sm_scale: float,
                      out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None):
    """q bf16 [T, H, d_qk]; topk int32 [T, W]; returns (out bf16 [T, H, 512], lse fp32 [T, H])."""
    _require_cuda(q, cache, topk_idx)
    T, H, d_qk = (int(s) for s in q.shape)
    W = int(topk_idx.shape[1])
    assert q.dtype == torch.bfloat16 and q.is_contiguous()
    assert topk_idx.dtype == torch.int32 and topk_idx.is_contiguous() and topk_idx.shape[0] == T
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, W, q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_n = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().mla_sparse_decode(q.data_ptr(), T, H, d_qk, kv_cache(cache), topk_idx.data_ptr(), W,
                                  float(sm_scale), out.data_ptr(), lse.data_ptr(), ws_ptr, ws_n,
                                  _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_sparse_decode")
    return out, lse


def mla_sparse_decode_paged(q: torch.Tensor, cache: torch.Tensor, topk_pos: torch.Tensor,
                            block_table: torch.Tensor, page_size: int, sm_scale: float,
                            token_seq: torch.Tensor | None = None, out: torch.Tensor | None = None,
                            lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Decode with the top-k given as sequence positions: q bf16 [T, H, d_qk]; topk_pos
    int32 [T, W]; block_table int32 [n_seq, max_pages] (or [max_pages]); token_seq int32
    [T] or None. Returns (out bf16 [T, H, 512], lse fp32 [T, H])."""
    _require_cuda(q, cache, topk_pos, block_table, token_seq)
    T, H, d_qk = (int(s) for s in q.shape)
    W = int(topk_pos.shape[1])
    bt = block_table if block_table.dim() == 2 else block_table.view(1, -1)
    assert q.dtype == torch.bfloat16 and q.is_contiguous()
    assert topk_pos.dtype == torch.int32 and topk_pos.is_contiguous() and topk_pos.shape[0] == T
    assert bt.dtype == torch.int32 and bt.is_contiguous()
    if token_seq is not None:
        assert token_seq.dtype == torch.int32 and token_seq.is_contiguous() and token_seq.numel() == T
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = alloc_workspace(T, H, W, q.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_n = workspace.numel() * workspace.element_size() if workspace is not None else 0
    rc = load().mla_sparse_decode_paged(q.data_ptr(), T, H, d_qk, kv_cache(cache), topk_pos.data_ptr(), W,
                                        bt.data_ptr(), int(bt.shape[0]), int(bt.shape[1]),
                                        token_seq.data_ptr() if token_seq is not None else None, int(page_size),
                                        float(sm_scale), out.data_ptr(), lse.data_ptr(), ws_ptr, ws_n,
                                        _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_sparse_decode_paged")
    return out, lse


def mla_sparse_prefill(q: torch.Tensor, cache: torch.Tensor, topk_idx: torch.Tensor, sm_scale: float,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None, stream=None):
    """What mla_sparse_decode computes, by token pairs that share their rows (causal
    prefill): q bf16 [T, H, d_qk]; topk int32 [T, W] with W <= 2304; returns
    (out bf16 [T, H, 512], lse fp32 [T, H]). No workspace."""
    _require_cuda(q, cache, topk_idx)
    T, H, d_qk = (int(s) for s in q.shape)
    W = int(topk_idx.shape[1])
    assert q.dtype == torch.bfloat16 and q.is_contiguous()
    assert topk_idx.dtype == torch.int32 and topk_idx.is_contiguous() and topk_idx.shape[0] == T
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    rc = load().mla_sparse_prefill(q.data_ptr(), T, H, d_qk, kv_cache(cache), topk_idx.data_ptr(), W,
                                   float(sm_scale), out.data_ptr(), lse.data_ptr(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_sparse_prefill")
    return out, lse


def mla_sparse_prefill_paged(q: torch.Tensor, cache: torch.Tensor, topk_pos: torch.Tensor,
                             block_table: torch.Tensor, page_size: int, sm_scale: float,
                             token_seq: torch.Tensor | None = None, out: torch.Tensor | None = None,
                             lse: torch.Tensor | None = None, stream=None):
    """mla_sparse_prefill with the top-k given as sequence positions through a block
    table (arguments as mla_sparse_decode_paged, no workspace)."""
    _require_cuda(q, cache, topk_pos, block_table, token_seq)
    T, H, d_qk = (int(s) for s in q.shape)
    W = int(topk_pos.shape[1])
    bt = block_table if block_table.dim() == 2 else block_table.view(1, -1)
    assert q.dtype == torch.bfloat16 and q.is_contiguous()
    assert topk_pos.dtype == torch.int32 and topk_pos.is_contiguous() and topk_pos.shape[0] == T
    assert bt.dtype == torch.int32 and bt.is_contiguous()
    if token_seq is not None:
        assert token_seq.dtype == torch.int32 and token_seq.is_contiguous() and token_seq.numel() == T
    if out is None:
        out = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q.device)
    rc = load().mla_sparse_prefill_paged(q.data_ptr(), T, H, d_qk, kv_cache(cache), topk_pos.data_ptr(), W,
                                         bt.data_ptr(), int(bt.shape[0]), int(bt.shape[1]),
                                         token_seq.data_ptr() if token_seq is not None else None,
                                         int(page_size), float(sm_scale), out.data_ptr(), lse.data_ptr(),
                                         _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_sparse_prefill_paged")
    return out, lse


def mla_gather_upconvert(cache: torch.Tensor, slots: torch.Tensor, pe_dim: int,
                         out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Rows at slots (int32 [n]) widened to bf16 [n, 576]."""
    _require_cuda(cache, slots, out)
    n = int(slots.numel())
    assert slots.dtype == torch.int32 and slots.is_contiguous()
    if out is None:
        out = torch.empty((n, 576), dtype=torch.bfloat16, device=cache.device)
    assert out.dtype == torch.bfloat16 and out.is_contiguous() and out.numel() == n * 576
    rc = load().mla_gather_upconvert(kv_cache(cache), slots.data_ptr(), n, int(pe_dim), out.data_ptr(),
                                     _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_gather_upconvert")
    return out


def rope_spec(inv_freq, axis=None, interleaved: bool = False, scale: float = 1.0, inverse: bool = False) -> RopeSpec:
    """Rotary frequencies of the 32 pairs (radians per position) and the axis each pair turns by (default: axis 0)."""
    inv, ax = list(inv_freq), [0] * 32 if axis is None else [int(a) for a in axis]
    if len(inv) != 32 or len(ax) != 32 or min(ax) < 0 or max(ax) > 3:
        raise ValueError("rope_spec takes 32 frequencies and 32 axes in 0..3")
    return RopeSpec((ctypes.c_double * 32)(*inv), scale, max(ax) + 1, int(interleaved), int(inverse),
                    (ctypes.c_uint8 * 32)(*ax))


def _same_device(*ts) -> None:
    """Device tensors, all on the current device (whose stream and kernels the call uses)."""
    dev = _device() if torch.cuda.is_initialized() else -2
    for t in ts:
        if t is not None and t.get_device() != dev:
            _require_cuda(t)
            raise ValueError(f"a tensor on {t.device} while the current device is cuda:{torch.cuda.current_device()}")


def _positions(pos: torch.Tensor, n: int, n_axes: int) -> int:
    """Checks positions int32 [n] or [axes, n]; returns the stride between axes (0: one row of positions for all)."""
    shape = pos.shape
    if pos.dtype != torch.int32 or len(shape) not in (1, 2) or shape[-1] != n or (n > 1 and pos.stride(-1) != 1):
        raise ValueError("positions must be int32 [n] or [axes, n], contiguous along n")
    if (1 if len(shape) == 1 else shape[0]) < n_axes:
        raise ValueError(f"positions for {n_axes} axes expected")
    if n_axes == 1:
        return 0                                            # never used
    stride = pos.stride(0)
    if 0 < stride < n:
        raise ValueError("the axes of positions may not overlap, unless they are one row for all (stride 0)")
    return stride


def _rope_view(x: torch.Tensor, n: int):
    """(pointer, row stride, head stride, heads) of a bf16 [n, heads, 64] or [n, 64] view."""
    shape, stride = x.shape, x.stride()
    if x.dtype != torch.bfloat16 or len(shape) not in (2, 3) or shape[0] != n or shape[-1] != 64 or stride[-1] != 1:
        raise ValueError("rotary values must be bf16 [n, heads, 64] or [n, 64], contiguous along the 64")
    if len(shape) == 2:
        return x.data_ptr(), stride[0], 0, 1
    return x.data_ptr(), stride[0], stride[1], shape[1]


def mla_rope(x: torch.Tensor, pos: torch.Tensor, rope: RopeSpec, out: torch.Tensor | None = None,
             stream=None) -> torch.Tensor:
    """Rotates x bf16 [n, heads, 64] (or [n, 64], any row and head strides that are multiples of 8) by positions
    int32 [n] or [axes, n] (a broadcast row, pos.expand(3, n), too); out may be x."""
    if out is None:
        with _on(stream):
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(x, pos, out)
    n = int(x.shape[0])
    stride = _positions(pos, n, rope.n_axes)
    if out.shape != x.shape:
        raise ValueError("out must have the shape of x")
    xp, xr, xh, heads = _rope_view(x, n)
    yp, yr, yh, _ = _rope_view(out, n)
    rc = load().mla_rope(xp, xr, xh, yp, yr, yh, n, heads, pos.data_ptr(), stride, ctypes.byref(rope), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_rope")
    return out


def mla_rope_kv_write(cache: torch.Tensor, slot_idx: torch.Tensor, latent: torch.Tensor, k_pe: torch.Tensor,
                      pos: torch.Tensor, rope: RopeSpec, q_pe: torch.Tensor | None = None,
                      q_out: torch.Tensor | None = None, reserved_slot: int = 0, stream=None) -> None:
    """mla_kv_write with k_pe [n, 64] rotated on the way; q_pe [n, heads, 64] (a view, for example the last 64 values of
    a query projection) rotated into q_out (default: in place) in the same launch."""
    if q_pe is not None and q_out is None:
        q_out = q_pe
    _same_device(cache, slot_idx, latent, k_pe, pos, q_pe, q_out)
    n = int(slot_idx.shape[0])
    assert slot_idx.dtype == torch.int64 and slot_idx.is_contiguous()
    assert latent.dtype == torch.bfloat16 and latent.is_contiguous() and latent.numel() == n * 512
    assert k_pe.dtype == torch.bfloat16 and k_pe.is_contiguous() and k_pe.numel() == n * 64
    stride = _positions(pos, n, rope.n_axes)
    xp = yp = None
    xr = xh = yr = yh = heads = 0
    if q_pe is not None:
        if q_out.shape != q_pe.shape:
            raise ValueError("q_out must have the shape of q_pe")
        xp, xr, xh, heads = _rope_view(q_pe, n)
        yp, yr, yh, _ = _rope_view(q_out, n)
    elif q_out is not None:
        raise ValueError("q_out without q_pe")
    rc = load().mla_rope_kv_write(kv_cache(cache), slot_idx.data_ptr(), latent.data_ptr(), k_pe.data_ptr(), n,
                                  int(reserved_slot), pos.data_ptr(), stride, ctypes.byref(rope), xp, xr, xh, yp, yr, yh,
                                  heads, _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_rope_kv_write")


def mla_chunk_attention_workspace_bytes(T: int, H: int, n_seq: int) -> int:
    return int(load().mla_chunk_attention_workspace_bytes(int(T), int(H), int(n_seq)))


def alloc_chunk_workspace(T: int, H: int, n_seq: int, device=None) -> torch.Tensor:
    return torch.empty(max(16, mla_chunk_attention_workspace_bytes(T, H, n_seq)), dtype=torch.uint8,
                       device=device or "cuda")


def mla_chunk_attention(q: torch.Tensor, cache: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                        block_table: torch.Tensor, page_size: int, sm_scale: float, causal: bool = True,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """Attention of new tokens over the paged cache, ragged batch: q bf16 [T, H, d_qk]; q_start int32 [n_seq + 1];
    kv_len int32 [n_seq] (new tokens included); block_table int32 [n_seq, max_pages]. Returns (out bf16 [T, H, 512],
    lse fp32 [T, H]); without `out` and `lse`, tokens outside every sequence get 0 and -inf."""
    _same_device(q, cache, q_start, kv_len, block_table, out, lse, workspace)
    T, H, d_qk = (int(s) for s in q.shape)
    n_seq = int(kv_len.shape[0])
    assert q.dtype == torch.bfloat16 and q.is_contiguous()
    assert q_start.dtype == torch.int32 and q_start.is_contiguous() and q_start.numel() == n_seq + 1
    assert kv_len.dtype == torch.int32 and kv_len.is_contiguous()
    assert block_table.dtype == torch.int32 and block_table.is_contiguous() and block_table.dim() == 2
    assert block_table.shape[0] == n_seq
    if out is None or lse is None or workspace is None:
        with _on(stream):
            if out is None:
                out = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=q.device)
            if lse is None:
                lse = torch.full((T, H), float("-inf"), dtype=torch.float32, device=q.device)
            if workspace is None:
                workspace = alloc_chunk_workspace(T, H, n_seq, q.device)
    assert out.dtype == torch.bfloat16 and out.is_contiguous() and out.numel() == T * H * 512
    assert lse.dtype == torch.float32 and lse.is_contiguous() and lse.numel() == T * H
    rc = load().mla_chunk_attention(q.data_ptr(), T, H, d_qk, kv_cache(cache), q_start.data_ptr(), kv_len.data_ptr(),
                                    block_table.data_ptr(), n_seq, int(block_table.shape[1]), int(page_size),
                                    int(bool(causal)), float(sm_scale), out.data_ptr(), lse.data_ptr(),
                                    workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_chunk_attention")
    return out, lse


def _ints(*ts) -> None:
    i32 = torch.int32
    for t in ts:
        if t is not None:
            assert t.dtype is i32 and t.is_contiguous()


def _batch(q_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor | None) -> int:
    """Checks a ragged batch's lengths and table; returns its number of sequences."""
    i32 = torch.int32
    n_seq = kv_len.numel()
    assert q_start.dtype is i32 and q_start.is_contiguous() and q_start.numel() == n_seq + 1
    assert kv_len.dtype is i32 and kv_len.is_contiguous()
    if block_table is not None:
        assert block_table.dtype is i32 and block_table.is_contiguous()
        assert block_table.dim() == 2 and block_table.shape[0] == n_seq
    return n_seq


def mla_block_keys(cache: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                   page_size: int, keys: torch.Tensor, n_tokens: int, stream=None) -> torch.Tensor:
    """Mean keys of the pages that the new tokens completed, into keys bf16 [num_pages, 576 or 512]; n_tokens: the tokens
    that q_start counts. With q_start counting all of kv_len, the keys of every complete page."""
    _same_device(cache, q_start, kv_len, block_table, keys)
    n_seq = _batch(q_start, kv_len, block_table)
    assert keys.dtype is torch.bfloat16 and keys.is_contiguous() and keys.dim() == 2
    rc = load().mla_block_keys(kv_cache(cache), keys.shape[1], q_start.data_ptr(), kv_len.data_ptr(),
                               block_table.data_ptr(), n_seq, block_table.shape[1], int(page_size), int(n_tokens),
                               keys.data_ptr(), keys.shape[0], _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_block_keys")
    return keys


def mla_block_scores(q: torch.Tensor, keys: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                     block_table: torch.Tensor, page_size: int, sm_scale: float, scores: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """scores fp32 [T, max_pages]: per token, summed over heads, the softmax of q . key over the complete blocks before its
    own. Other columns are left alone (without `scores`: -inf)."""
    _same_device(q, keys, q_start, kv_len, block_table, scores)
    T, H, d_qk = q.shape
    n_seq = _batch(q_start, kv_len, block_table)
    assert q.dtype is torch.bfloat16 and q.is_contiguous()
    assert keys.dtype is torch.bfloat16 and keys.is_contiguous() and keys.dim() == 2 and keys.shape[1] == d_qk
    if scores is None:
        with _on(stream):
            scores = torch.full((T, block_table.shape[1]), float("-inf"), dtype=torch.float32, device=q.device)
    assert scores.dtype is torch.float32 and scores.is_contiguous() and scores.shape == (T, block_table.shape[1])
    rc = load().mla_block_scores(q.data_ptr(), T, H, d_qk, keys.data_ptr(), keys.shape[0], q_start.data_ptr(),
                                 kv_len.data_ptr(), block_table.data_ptr(), n_seq, block_table.shape[1],
                                 int(page_size), float(sm_scale), scores.data_ptr(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_block_scores")
    return scores


def mla_block_select(scores: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, page_size: int, width: int,
                     sink: int = 1, local: int = 1, blocks: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """blocks int32 [T, width]: the first `sink` blocks, the last `local` up to the token's own, and the best others by
    scores [T, max_pages]; ascending, then -1 (without `blocks`, -1 for tokens outside every sequence)."""
    _same_device(scores, q_start, kv_len, blocks)
    n_seq = _batch(q_start, kv_len, None)
    assert scores.dtype is torch.float32 and scores.is_contiguous() and scores.dim() == 2
    T = scores.shape[0]
    if blocks is None:
        with _on(stream):
            blocks = torch.full((T, int(width)), -1, dtype=torch.int32, device=scores.device)
    _ints(blocks)
    assert blocks.shape == (T, int(width))
    rc = load().mla_block_select(scores.data_ptr(), T, scores.shape[1], q_start.data_ptr(), kv_len.data_ptr(), n_seq,
                                 int(page_size), int(sink), int(local), int(width), blocks.data_ptr(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_block_select")
    return blocks


def mla_block_attention_workspace_bytes(T: int, H: int, width: int) -> int:
    return int(load().mla_block_attention_workspace_bytes(int(T), int(H), int(width)))


def alloc_block_workspace(T: int, H: int, width: int, device=None) -> torch.Tensor:
    return torch.empty(max(16, mla_block_attention_workspace_bytes(T, H, width)), dtype=torch.uint8,
                       device=device or "cuda")


def mla_block_attention(q: torch.Tensor, cache: torch.Tensor, blocks: torch.Tensor, q_start: torch.Tensor,
                        kv_len: torch.Tensor, block_table: torch.Tensor, page_size: int, sm_scale: float,
                        out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, stream=None):
    """Attention of each token over the positions up to its own of its blocks (int32 [T, width], -1: none): q bf16
    [T, H, d_qk]. Returns (out bf16 [T, H, 512], lse fp32 [T, H]); without `out` and `lse`, tokens outside every sequence
    get 0 and -inf."""
    _same_device(q, cache, blocks, q_start, kv_len, block_table, out, lse, workspace)
    T, H, d_qk = q.shape
    n_seq = _batch(q_start, kv_len, block_table)
    assert q.dtype is torch.bfloat16 and q.is_contiguous()
    _ints(blocks)
    assert blocks.dim() == 2 and blocks.shape[0] == T
    width = blocks.shape[1]
    out, lse = _outputs(q, out, lse, stream)
    if workspace is None:
        with _on(stream):
            workspace = alloc_block_workspace(T, H, width, q.device)
    rc = load().mla_block_attention(q.data_ptr(), T, H, d_qk, kv_cache(cache), blocks.data_ptr(), width,
                                    q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), n_seq,
                                    block_table.shape[1], int(page_size), float(sm_scale), out.data_ptr(),
                                    lse.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_block_attention")
    return out, lse


def _outputs(q: torch.Tensor, out: torch.Tensor | None, lse: torch.Tensor | None, stream):
    """out bf16 [T, H, 512] and lse fp32 [T, H] as given, or made: 0 and -inf."""
    T, H = q.shape[:2]
    if out is None or lse is None:
        with _on(stream):
            if out is None:
                out = torch.zeros((T, H, 512), dtype=torch.bfloat16, device=q.device)
            if lse is None:
                lse = torch.full((T, H), float("-inf"), dtype=torch.float32, device=q.device)
    assert out.dtype is torch.bfloat16 and out.is_contiguous() and out.numel() == T * H * 512
    assert lse.dtype is torch.float32 and lse.is_contiguous() and lse.numel() == T * H
    return out, lse


def mla_tree_mask(parent: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, words: int | None = None,
                  mask: torch.Tensor | None = None, positions: torch.Tensor | None = None, stream=None):
    """For drafted tokens with parents int32 [T] (indices within their sequence; negative: none): (mask int32 [T, words],
    bits for the token and its ancestors; positions int32 [T], for the rotary write). `words`: 32 tokens of a sequence
    each, where no mask is given (2 unless said)."""
    _same_device(parent, q_start, kv_len, mask, positions)
    n_seq = _batch(q_start, kv_len, None)
    T = parent.numel()
    if mask is None or positions is None:
        with _on(stream):
            if mask is None:
                mask = torch.zeros((T, 2 if words is None else int(words)), dtype=torch.int32, device=parent.device)
            if positions is None:
                positions = torch.zeros(T, dtype=torch.int32, device=parent.device)
    _ints(parent, mask, positions)
    assert mask.dim() == 2 and mask.shape[0] == T and positions.numel() == T
    rc = load().mla_tree_mask(parent.data_ptr(), T, q_start.data_ptr(), kv_len.data_ptr(), n_seq, mask.data_ptr(),
                              mask.shape[1], positions.data_ptr(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_tree_mask")
    return mask, positions


def mla_tree_attention(q: torch.Tensor, cache: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor,
                       block_table: torch.Tensor, page_size: int, sm_scale: float, mask: torch.Tensor,
                       out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """mla_chunk_attention with a mask among the new tokens (int32 [T, words], as mla_tree_mask makes it). The workspace is
    alloc_chunk_workspace's."""
    _same_device(q, cache, q_start, kv_len, block_table, mask, out, lse, workspace)
    T, H, d_qk = q.shape
    n_seq = _batch(q_start, kv_len, block_table)
    assert q.dtype is torch.bfloat16 and q.is_contiguous()
    _ints(mask)
    assert mask.dim() == 2 and mask.shape[0] == T
    out, lse = _outputs(q, out, lse, stream)
    if workspace is None:
        with _on(stream):
            workspace = alloc_chunk_workspace(T, H, n_seq, q.device)
    rc = load().mla_tree_attention(q.data_ptr(), T, H, d_qk, kv_cache(cache), q_start.data_ptr(), kv_len.data_ptr(),
                                   block_table.data_ptr(), n_seq, block_table.shape[1], int(page_size),
                                   mask.data_ptr(), mask.shape[1], float(sm_scale), out.data_ptr(), lse.data_ptr(),
                                   workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_tree_attention")
    return out, lse


def mla_tree_commit(cache: torch.Tensor, q_start: torch.Tensor, kv_len: torch.Tensor, block_table: torch.Tensor,
                    page_size: int, path: torch.Tensor, path_len: torch.Tensor, kv_len_out: torch.Tensor | None = None,
                    stream=None) -> None:
    """Rows of the accepted tokens path[s, :path_len[s]] (int32 [n_seq, max_path], ascending indices within the sequence)
    to the front of the drafted ones; kv_len_out (may be kv_len) receives the new lengths."""
    _same_device(cache, q_start, kv_len, block_table, path, path_len, kv_len_out)
    n_seq = _batch(q_start, kv_len, block_table)
    _ints(path, path_len, kv_len_out)
    assert path.dim() == 2 and path.shape[0] == n_seq and path_len.numel() == n_seq
    assert kv_len_out is None or kv_len_out.numel() == n_seq
    rc = load().mla_tree_commit(kv_cache(cache), q_start.data_ptr(), kv_len.data_ptr(), block_table.data_ptr(), n_seq,
                                block_table.shape[1], int(page_size), path.data_ptr(), path_len.data_ptr(),
                                path.shape[1], kv_len_out.data_ptr() if kv_len_out is not None else None,
                                _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_tree_commit")


def mla_page_workspace_bytes(num_pages: int, n_forks: int = 0) -> int:
    return int(load().mla_page_workspace_bytes(int(num_pages), int(n_forks)))


def alloc_page_workspace(num_pages: int, n_forks: int = 0, device=None) -> torch.Tensor:
    return torch.empty(mla_page_workspace_bytes(num_pages, n_forks), dtype=torch.uint8, device=device or "cuda")


def mla_page_copy(dst_cache: torch.Tensor, src_cache: torch.Tensor, page_size: int, dst: torch.Tensor,
                  src: torch.Tensor, stream=None) -> None:
    """Pages src (int32 [n]) of src_cache to pages dst of dst_cache (which may be the same cache)."""
    _same_device(dst_cache, src_cache, dst, src)
    _ints(dst, src)
    assert dst.numel() == src.numel()
    rc = load().mla_page_copy(kv_cache(dst_cache), kv_cache(src_cache), int(page_size), dst.data_ptr(), src.data_ptr(),
                              int(dst.numel()), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_copy")


def mla_page_free(refcount: torch.Tensor, block_table: torch.Tensor, rows: torch.Tensor, stream=None) -> None:
    """Rows (int32 [n]) of block_table let go of their pages."""
    _same_device(refcount, block_table, rows)
    _ints(refcount, block_table, rows)
    rc = load().mla_page_free(refcount.data_ptr(), int(refcount.numel()), block_table.data_ptr(),
                              int(block_table.shape[0]), int(block_table.shape[1]), rows.data_ptr(), int(rows.numel()),
                              _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_free")


def mla_page_fork(cache: torch.Tensor, page_size: int, refcount: torch.Tensor, block_table: torch.Tensor,
                  parent: torch.Tensor, child: torch.Tensor, lens: torch.Tensor,
                  workspace: torch.Tensor | None = None, stream=None) -> None:
    """Row child[i] of block_table becomes a copy of row parent[i] up to lens[i] positions: whole pages shared, a last
    page that is not full copied to a free page."""
    _same_device(cache, refcount, block_table, parent, child, lens, workspace)
    _ints(refcount, block_table, parent, child, lens)
    n = int(parent.numel())
    assert child.numel() == n and lens.numel() == n
    if workspace is None:
        with _on(stream):
            workspace = alloc_page_workspace(refcount.numel(), n, cache.device)
    rc = load().mla_page_fork(kv_cache(cache), int(page_size), refcount.data_ptr(), int(refcount.numel()),
                              block_table.data_ptr(), int(block_table.shape[0]), int(block_table.shape[1]),
                              parent.data_ptr(), child.data_ptr(), lens.data_ptr(), n, workspace.data_ptr(),
                              workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_fork")


def mla_page_compact(cache: torch.Tensor, page_size: int, refcount: torch.Tensor, block_table: torch.Tensor,
                     refcount_out: torch.Tensor | None = None, table_out: torch.Tensor | None = None,
                     page_map: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None) -> None:
    """Moves the live pages to 1 .. live. Counts and table are updated in place unless refcount_out / table_out are
    given; page_map (int32 [num_pages]) receives where each page went."""
    refcount_out = refcount if refcount_out is None else refcount_out
    table_out = block_table if table_out is None else table_out
    _same_device(cache, refcount, block_table, refcount_out, table_out, page_map, workspace)
    _ints(refcount, block_table, refcount_out, table_out, page_map)
    assert refcount_out.numel() == refcount.numel() and table_out.shape == block_table.shape
    assert page_map is None or page_map.numel() == refcount.numel()
    if workspace is None:
        with _on(stream):
            workspace = alloc_page_workspace(refcount.numel(), 0, cache.device)
    rc = load().mla_page_compact(kv_cache(cache), int(page_size), refcount.data_ptr(), refcount_out.data_ptr(),
                                 int(refcount.numel()), block_table.data_ptr(), table_out.data_ptr(),
                                 int(block_table.shape[0]), int(block_table.shape[1]),
                                 page_map.data_ptr() if page_map is not None else None, workspace.data_ptr(),
                                 workspace.numel() * workspace.element_size(), _stream(stream))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_page_compact")


def mla_get_error() -> int:
    v = ctypes.c_int32(0)
    rc = load().mla_get_error(ctypes.byref(v))
    if rc != MLA_OK:
        raise MlaError(rc, "mla_get_error")
    return int(v.value)
