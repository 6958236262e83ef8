"""Python binding of the 4-bit KV cache operators (include/kv_mxfp4.h).

As the MoE binding: tensors are checked, outputs and the workspace are made
with PyTorch when the caller passes none, and the C ABI is called with raw
device pointers on the current CUDA stream of the tensors' device.  Everything
is computed in the library's kernels.

One serving step: ``kv_page_tables`` (block tables and slot maps from request
lengths) -> ``kv_append_mxfp4`` (new keys and values, quantised, to their slots)
-> ``attention_kv_mxfp4`` (the step's queries over the cache).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _native
from ._native import KvAttnStruct, KvCacheStruct, int32

_i32 = torch.int32


# The current stream's handle by device index; torch.cuda.current_stream() builds
# a Stream object for it (2.9 us on the GB300's host cores, against 0.1).
_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _stream(stream, t):
    # a call belongs on its tensors' device: the library launches on the current one
    i = t.get_device()
    if i != _current_device():
        raise ValueError(f"tensors are on {t.device}, the current device is cuda:{_current_device()}")
    return _raw_stream(i) if stream is None else stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """An output made for the caller: from the allocator's pool of the stream it is written on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _need(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _cuda(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _flat(t, dtype, shape, device) -> bool:
    """Whether ``_need`` would pass (a call of a few microseconds asks this first and names what is wrong after)."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device


class KvCacheMxfp4:
    """One layer's paged key/value cache in MXFP4.

    ``data`` is uint8 [num_pages, num_kv_heads, page_size / 16, 17 * head_dim]
    (the record layout is that of ``kv_mxfp4_cache_t``); it is allocated on
    ``device`` when not given.  ``head_dim`` 64 or 128, ``page_size`` 16, 32, 64,
    128 or 256.  A slot is ``page * page_size + offset``."""

    def __init__(self, num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, data=None, device="cuda"):
        self.num_pages, self.page_size, self.num_kv_heads, self.head_dim = num_pages, page_size, num_kv_heads, head_dim
        self._struct = KvCacheStruct(None, num_pages, page_size, num_kv_heads, head_dim)
        if _native.load().kv_mxfp4_cache_bytes(ctypes.byref(self._struct)) == 0:
            raise ValueError(f"unsupported cache: {num_pages} pages of {page_size} tokens, {num_kv_heads} heads of {head_dim}")
        shape = (num_pages, num_kv_heads, page_size // 16, 17 * head_dim)
        if data is None:
            data = torch.empty(shape, dtype=torch.uint8, device=device)
        self.device = _cuda(data, "data")
        _need(data, "data", torch.uint8, shape, self.device)
        self.data = data
        self._struct.data = data.data_ptr()
        self._ref = ctypes.byref(self._struct)


class PageTables(NamedTuple):
    """``kv_page_tables``'s outputs (the block table and the ring are updated in place)."""

    seq_lens: torch.Tensor
    query_start: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    ring_state: torch.Tensor


def kv_page_tables(cached_lens, new_lens, block_table, free_ring, ring_state, page_size: int, max_tokens: int,
                   seq_lens=None, query_start=None, slots=None, positions=None, ring_state_out=None,
                   stream=None) -> PageTables:
    """Block tables and slot maps of one step, on the GPU, from request lengths.

    ``cached_lens`` int32 [R] tokens held, ``new_lens`` int32 [R] tokens added
    (-1: finished, gives its pages back), ``block_table`` int32 [R, max_blocks]
    (entries of new pages are written), ``free_ring`` int32 [ring size] and
    ``ring_state`` int32 [2] {head, free pages} (pages are taken at the head,
    given back at the end).  Returns ``seq_lens`` [R] (-1 for a refused request),
    ``query_start`` [R+1], ``slots`` and ``positions`` [max_tokens] (-1 padding)
    and the ring's new state; pass that state into the next step.  Outputs may not
    share memory with one another or with an input (``seq_lens`` is not
    ``cached_lens``: copy it over them after the call, but for -1)."""
    dev = _cuda(cached_lens, "cached_lens")
    R = cached_lens.shape[0]
    if block_table.dim() != 2 or free_ring.dim() != 1:
        raise ValueError("block_table must be [R, max_blocks] and free_ring [ring size]")
    mb, C = block_table.shape[1], free_ring.shape[0]
    seq_lens = _empty(R, _i32, dev, stream) if seq_lens is None else seq_lens
    query_start = _empty(R + 1, _i32, dev, stream) if query_start is None else query_start
    slots = _empty(max_tokens, _i32, dev, stream) if slots is None else slots
    positions = _empty(max_tokens, _i32, dev, stream) if positions is None else positions
    ring_state_out = _empty(2, _i32, dev, stream) if ring_state_out is None else ring_state_out
    for t, name, shape in ((cached_lens, "cached_lens", (R,)), (new_lens, "new_lens", (R,)),
                           (block_table, "block_table", (R, mb)), (free_ring, "free_ring", (C,)),
                           (ring_state, "ring_state", (2,)), (seq_lens, "seq_lens", (R,)),
                           (query_start, "query_start", (R + 1,)), (slots, "slots", (max_tokens,)),
                           (positions, "positions", (max_tokens,)), (ring_state_out, "ring_state_out", (2,))):
        if t.dtype is not _i32 or t.shape != shape or not t.is_contiguous() or t.device != dev:
            _need(t, name, _i32, shape, dev)
    if ring_state_out.data_ptr() == ring_state.data_ptr():
        raise ValueError("ring_state_out must not be ring_state")
    rc = _native.load().kv_mxfp4_page_tables(
        R, page_size, mb, max_tokens, C, cached_lens.data_ptr(), new_lens.data_ptr(), block_table.data_ptr(),
        free_ring.data_ptr(), ring_state.data_ptr(), seq_lens.data_ptr(), query_start.data_ptr(), slots.data_ptr(),
        positions.data_ptr(), ring_state_out.data_ptr(), _stream(stream, cached_lens))
    _native.check("kv_mxfp4_page_tables", rc)
    return PageTables(seq_lens, query_start, slots, positions, ring_state_out)


def _rows(x, name, cache, N, dtypes):
    """Checks [N, heads, head_dim] rows with any token stride; returns that stride in elements."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    H, D = cache.num_kv_heads, cache.head_dim
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {x.dtype}")
    if x.shape != (N, H, D):
        raise ValueError(f"{name} must have shape {(N, H, D)}, got {tuple(x.shape)}")
    if x.device != cache.device:
        raise ValueError(f"{name} must be on {cache.device}, got {x.device}")
    st = x.stride()
    if st[2] != 1 or (H > 1 and st[1] != D):
        raise ValueError(f"{name}: a token's heads must be dense")
    return st[0] if N > 1 else H * D


def _queries(q, cache, dtype):
    """Checks queries [N, Hq, head_dim] with any token stride; returns N, Hq and that stride in elements."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if q.dtype != dtype:
        raise TypeError(f"q must be {dtype}, got {q.dtype}")
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError(f"q must have shape [N, Hq, {cache.head_dim}], got {tuple(q.shape)}")
    if q.device != cache.device:
        raise ValueError(f"q must be on {cache.device}, got {q.device}")
    N, Hq, D = q.shape
    st = q.stride()
    if st[2] != 1 or (Hq > 1 and st[1] != D):
        raise ValueError("q: a token's heads must be dense")
    return N, Hq, st[0] if N > 1 else Hq * D


def kv_append_mxfp4(cache: KvCacheMxfp4, k, v, slots, stream=None) -> None:
    """Quantise ``k``, ``v`` [N, kv heads, head_dim] (bf16 or float32; token rows may be strided, as slices of a
    fused projection) and write them to ``slots`` int32 [N] (-1: not written)."""
    _cuda(slots, "slots")
    N = slots.shape[0]
    _need(slots, "slots", _i32, (N,), cache.device)
    ks = _rows(k, "k", cache, N, (torch.bfloat16, torch.float32))
    vs = _rows(v, "v", cache, N, (k.dtype,))
    rc = _native.load().kv_mxfp4_append(cache._ref, k.data_ptr(), v.data_ptr(), 1 if k.dtype == torch.float32 else 0,
                                        ks, vs, N, slots.data_ptr(), _stream(stream, slots))
    _native.check("kv_mxfp4_append", rc)


def kv_gather_mxfp4(cache: KvCacheMxfp4, slots, k_out=None, v_out=None, stream=None):
    """The keys and values that ``slots`` int32 [N] hold: two bf16 [N, kv heads, head_dim] (exact; zeros for -1)."""
    _cuda(slots, "slots")
    dev = cache.device
    N = slots.shape[0]
    if slots.dtype is not _i32 or slots.dim() != 1 or not slots.is_contiguous() or slots.device != dev:
        _need(slots, "slots", _i32, (N,), dev)
    shape = (N, cache.num_kv_heads, cache.head_dim)
    if k_out is None:
        k_out = _empty(shape, torch.bfloat16, dev, stream)
    elif not isinstance(k_out, torch.Tensor) or not _flat(k_out, torch.bfloat16, shape, dev):
        _need(k_out, "k_out", torch.bfloat16, shape, dev)
    if v_out is None:
        v_out = _empty(shape, torch.bfloat16, dev, stream)
    elif not isinstance(v_out, torch.Tensor) or not _flat(v_out, torch.bfloat16, shape, dev):
        _need(v_out, "v_out", torch.bfloat16, shape, dev)
    rc = _native.load().kv_mxfp4_gather(cache._ref, slots.data_ptr(), N, k_out.data_ptr(), v_out.data_ptr(),
                                        _stream(stream, slots))
    _native.check("kv_mxfp4_gather", rc)
    return k_out, v_out


def attention_workspace_bytes(cache: KvCacheMxfp4, R: int, N: int, Hq: int, max_blocks: int, max_q_len: int) -> int:
    """Bytes of workspace for ``attention_kv_mxfp4`` calls of at most these sizes' kind."""
    D = cache.head_dim
    a = KvAttnStruct(int32(R), int32(N), int32(Hq), int32(max_blocks), int32(max_q_len), 1, 0, Hq * D, 1.0)
    return int(_native.load().kv_mxfp4_attention_workspace_bytes(cache._ref, ctypes.byref(a)))


def attention_kv_mxfp4(q, cache: KvCacheMxfp4, block_table, seq_lens, query_start, max_q_len: int, scale=None,
                       causal: bool = True, window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Attention of ``q`` bf16 [N, Hq, head_dim] over the 4-bit cache; returns bf16 [N, Hq, head_dim].

    ``block_table`` int32 [R, max_blocks], ``seq_lens`` int32 [R] (keys of each
    request, the step's new tokens included), ``query_start`` int32 [R+1] (first
    query row of each request), ``max_q_len`` the largest number of rows of one
    request.  ``scale`` defaults to head_dim ** -0.5.  ``causal``: row i of q rows
    sits at position seq_len - q + i; ``window``: only the last ``window`` keys.
    ``lse`` float32 [N, Hq], when given, receives ln sum exp of the scores.  A row
    without a visible key gets zeros (lse -inf).  Pass ``workspace`` (uint8,
    ``attention_workspace_bytes``, first 4 bytes zeroed once) to allocate nothing,
    and to learn of waits that ran out (``attention_read_status``): those of a
    workspace made here go unseen."""
    dev = cache.device
    N, Hq, q_stride = _queries(q, cache, torch.bfloat16)
    D = cache.head_dim
    R = seq_lens.shape[0]
    if block_table.dim() != 2:
        raise ValueError("block_table must be [R, max_blocks]")
    mb = block_table.shape[1]
    for t, name, shape in ((block_table, "block_table", (R, mb)), (seq_lens, "seq_lens", (R,)),
                           (query_start, "query_start", (R + 1,))):
        if t.dtype is not _i32 or t.shape != shape or not t.is_contiguous() or t.device != dev:
            _need(t, name, _i32, shape, dev)
    if out is None:
        out = _empty((N, Hq, D), torch.bfloat16, dev, stream)
    _need(out, "out", torch.bfloat16, (N, Hq, D), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (N, Hq), dev)
    # (a window past the C ABI's int hides nothing: no request has that many keys)
    a = KvAttnStruct(int32(R), N, Hq, int32(mb), int32(max_q_len), 1 if causal else 0, int32(window), q_stride,
                     D ** -0.5 if scale is None else scale)
    lib = _native.load()
    ref = ctypes.byref(a)
    if workspace is None:
        workspace = _empty(max(256, lib.kv_mxfp4_attention_workspace_bytes(cache._ref, ref)), torch.uint8, dev, stream)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    rc = lib.kv_mxfp4_attention(cache._ref, ref, q.data_ptr(), block_table.data_ptr(), seq_lens.data_ptr(),
                                query_start.data_ptr(), out.data_ptr(), None if lse is None else lse.data_ptr(),
                                workspace.data_ptr(), workspace.numel(), _stream(stream, q))
    _native.check("kv_mxfp4_attention", rc)
    return out


def attention_read_status(workspace, stream=None) -> int:
    """Read and clear the status word of an attention workspace (synchronises the stream)."""
    v = ctypes.c_uint32(0)
    rc = _native.load().kv_mxfp4_read_status(workspace.data_ptr(), ctypes.byref(v), _stream(stream, workspace))
    _native.check("kv_mxfp4_read_status", rc)
    return int(v.value)
