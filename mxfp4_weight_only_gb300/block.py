"""Python binding of the attention block's operators (include/block_mxfp4.h).

As the cache's binding: tensors are checked, outputs and the workspace are made
with PyTorch when the caller passes none, and the C ABI is called with raw
device pointers on the current CUDA stream of the tensors' device.  Everything
is computed in the library's kernels.

One layer's attention block: ``linear_a16w4_mxfp4`` (queries, keys and values) ->
``kv_append_rope_mxfp4`` (rotated, keys and values quantised to their slots) ->
``attention_kv_mxfp4``, or ``attention_kv_mxfp4_shared`` behind a common prefix ->
``linear_a16w4_mxfp4`` (output, added to the residual stream).
"""

from __future__ import annotations

import ctypes

import torch

from . import _native
from ._native import KvAttnStruct, KvRopeStruct, LinearStruct, int32
from .kv_cache import KvCacheMxfp4, _empty, _flat, _i32, _need, _queries, _rows, _stream

_ACTS = {None: 0, "none": 0, "silu": 1, "gelu": 2, "swiglu": 3}
_T, _bf16, _u8 = torch.Tensor, torch.bfloat16, torch.uint8
_BF16, _OUT = (torch.bfloat16,), (torch.bfloat16, torch.float32)


def linear_workspace_bytes(T: int, N: int, K: int) -> int:
    """Bytes of workspace for ``linear_a16w4_mxfp4`` calls of these sizes."""
    d = LinearStruct(int32(T), int32(K), int32(N), 0, 0, -(-K // 8) * 8, N, N)
    return int(_native.load().linear_mxfp4_workspace_bytes(ctypes.byref(d)))


def _matrix(t, name, dtypes, rows, cols, device):
    """Checks a matrix [rows, cols] of dense rows; returns the rows' stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {dtypes}, got {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    st = t.stride()
    if cols > 1 and st[1] != 1:
        raise ValueError(f"{name}: rows must be dense")
    return st[0] if rows > 1 else cols


def linear_a16w4_mxfp4(x, w, w_scale, bias=None, act=None, residual=None, out=None, out_dtype=torch.bfloat16,
                       workspace=None, stream=None):
    """``act(x @ W.T + bias) + residual`` on an MXFP4 weight, float32 sums, rounded once.

    ``x`` bf16 [T, K] (rows may be strided by a multiple of 8 elements), ``w`` uint8
    [N, K / 2] (packed E2M1), ``w_scale`` uint8 [N, K / 32] (E8M0), ``bias`` bf16 [N].
    ``act``: None, "silu", "gelu" (erf) or "swiglu" (SiLU of the first N / 2 columns times the
    others: N / 2 columns).  ``residual`` bf16 [T, columns], rows strided at will.
    Returns ``out`` [T, columns], bf16 or float32 (``out_dtype``, or that of the ``out`` given, whose
    rows may be strided; a bf16 ``out`` may be ``residual`` itself).  Pass ``workspace``
    (uint8, ``linear_workspace_bytes``, first 4 bytes zeroed once) to allocate nothing
    but a missing ``out``, and to learn of waits that ran out (``linear_read_status``)."""
    if not isinstance(x, _T) or not isinstance(w, _T) or not isinstance(w_scale, _T):
        raise TypeError("x, w and w_scale must be torch.Tensors")
    xs, ws = x.shape, w.shape
    if len(xs) != 2 or len(ws) != 2:
        raise ValueError("x must be [T, K] and w [N, K / 2]")
    i = x.get_device()
    if i < 0:
        raise ValueError("x must be a CUDA tensor")
    code = _ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {tuple(_ACTS)}, got {act!r}")
    (T, K), N = xs, ws[0]
    if N + K > 0x7FFFFFFF:  # (an int32 each in the C ABI; T: more than memory holds)
        raise ValueError(f"the weight is too large: {N} rows of {K}")
    cols = N
    if code == 3:
        if N % 2:
            raise ValueError(f"swiglu needs an even number of weight rows, got {N}")
        cols = N // 2
    # (conditions written out: a call of a few microseconds feels a function a tensor)
    xs = x.stride()
    if x.dtype is not _bf16 or (K > 1 and xs[1] != 1):
        _matrix(x, "x", _BF16, T, K, x.device)
    xs = xs[0] if T > 1 else -(-K // 8) * 8
    if w.dtype is not _u8 or ws[1] != K // 2 or not w.is_contiguous() or w.get_device() != i:
        _need(w, "w", _u8, (N, K // 2), x.device)
    if w_scale.dtype is not _u8 or w_scale.shape != (N, K // 32) or not w_scale.is_contiguous() or w_scale.get_device() != i:
        _need(w_scale, "w_scale", _u8, (N, K // 32), x.device)
    if bias is not None:
        if not isinstance(bias, _T) or bias.dtype is not _bf16 or bias.shape != (N,) or not bias.is_contiguous() or bias.get_device() != i:
            _need(bias, "bias", _bf16, (N,), x.device)
    rs = cols
    if residual is not None:
        rs = _matrix(residual, "residual", _BF16, T, cols, x.device)
    if out is None:
        if out_dtype not in _OUT:
            raise TypeError(f"out_dtype must be torch.bfloat16 or torch.float32, got {out_dtype}")
        out = _empty((T, cols), out_dtype, x.device, stream)
        os = cols
    elif isinstance(out, _T) and out.dtype is _bf16 and out.shape == (T, cols) and out.is_contiguous() and out.get_device() == i:
        os = cols
    else:
        os = _matrix(out, "out", _OUT, T, cols, x.device)
    lib = _native.load()
    d = LinearStruct(T, K, N, code, 1 if out.dtype is torch.float32 else 0, xs, rs, os)
    ref = ctypes.byref(d)
    if workspace is None:
        workspace = _empty(max(256, lib.linear_mxfp4_workspace_bytes(ref)), torch.uint8, x.device, stream)
    elif workspace.dtype is not _u8 or workspace.get_device() != i or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {x.device}")
    # (arguments keep their tensors to here: one that only this call holds would give its memory to ``out`` or the workspace)
    rc = lib.linear_a16w4_mxfp4(ref, x.data_ptr(), w.data_ptr(), w_scale.data_ptr(), None if bias is None else bias.data_ptr(),
                                None if residual is None else residual.data_ptr(), out.data_ptr(), workspace.data_ptr(),
                                workspace.numel(), _stream(stream, x))
    if rc:
        _native.check("linear_a16w4_mxfp4", rc)
    return out


def linear_read_status(workspace, stream=None) -> int:
    """Read and clear the status word of a linear layer's workspace (synchronises the stream)."""
    v = ctypes.c_uint32(0)
    rc = _native.load().linear_mxfp4_read_status(workspace.data_ptr(), ctypes.byref(v), _stream(stream, workspace))
    _native.check("linear_mxfp4_read_status", rc)
    return int(v.value)


def kv_append_rope_mxfp4(cache: KvCacheMxfp4, q, k, v, positions, slots, cos_sin, interleaved: bool = False,
                         position_offset: int = 0, q_out=None, stream=None):
    """Rotate ``q`` [N, Hq, head_dim] and ``k`` [N, kv heads, head_dim] by their positions, write the rotated keys
    and ``v``, quantised, to ``slots`` int32 [N] (-1: not written), and return the rotated queries, bf16 [N, Hq, head_dim].

    q, k, v: bf16 or float32, token rows may be strided (slices of a fused
    projection); ``q`` may be None.  ``positions`` int32 [N], each plus ``position_offset``
    (the length of a prefix that the requests share); a negative one is padding (a row
    of zeros, nothing written).  ``cos_sin`` float32 [positions, rotary_dim]: a position's cosines,
    then its sines; rotary_dim, a multiple of 16, leading elements of a head are rotated, in pairs
    (i, i + rotary_dim / 2) or, with ``interleaved``, (2i, 2i + 1).  A position past the table
    makes its token NaN."""
    if not isinstance(positions, _T) or not isinstance(slots, _T) or not isinstance(cos_sin, _T):
        raise TypeError("positions, slots and cos_sin must be torch.Tensors")
    dev = cache.device
    N = positions.shape[0]
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rotary_dim]")
    if positions.dtype is not _i32 or positions.dim() != 1 or not positions.is_contiguous() or positions.device != dev:
        _need(positions, "positions", _i32, (N,), dev)
    if slots.dtype is not _i32 or slots.shape != (N,) or not slots.is_contiguous() or slots.device != dev:
        _need(slots, "slots", _i32, (N,), dev)
    if cos_sin.dtype is not torch.float32 or not cos_sin.is_contiguous() or cos_sin.device != dev:
        _need(cos_sin, "cos_sin", torch.float32, cos_sin.shape, dev)
    ks = _rows(k, "k", cache, N, (torch.bfloat16, torch.float32))
    vs = _rows(v, "v", cache, N, (k.dtype,))
    Hq, qs, D = 0, 0, cache.head_dim
    if q is not None:
        rows, Hq, qs = _queries(q, cache, k.dtype)
        if rows != N:
            raise ValueError(f"q must have shape [{N}, Hq, {D}], got {tuple(q.shape)}")
        if q_out is None:
            q_out = _empty((N, Hq, D), torch.bfloat16, dev, stream)
        elif not isinstance(q_out, _T) or not _flat(q_out, _bf16, (N, Hq, D), dev):
            _need(q_out, "q_out", _bf16, (N, Hq, D), dev)
    elif q_out is not None:
        raise ValueError("q_out without q")
    r = KvRopeStruct(int32(N), Hq, 1 if k.dtype == torch.float32 else 0, cos_sin.shape[1], 1 if interleaved else 0,
                     int32(cos_sin.shape[0]), int32(position_offset), qs, ks, vs)
    rc = _native.load().kv_mxfp4_append_rope(
        cache._ref, ctypes.byref(r), None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
        positions.data_ptr(), slots.data_ptr(), cos_sin.data_ptr(), None if q_out is None else q_out.data_ptr(),
        _stream(stream, positions))
    if rc:
        _native.check("kv_mxfp4_append_rope", rc)
    return q_out


def attention_shared_workspace_bytes(cache: KvCacheMxfp4, R: int, N: int, Hq: int, max_blocks: int, max_q_len: int,
                                     shared_blocks: int) -> int:
    """Bytes of workspace for ``attention_kv_mxfp4_shared`` calls of these sizes, or of fewer requests and rows."""
    D = cache.head_dim
    a = KvAttnStruct(int32(R), int32(N), int32(Hq), int32(max_blocks), int32(max_q_len), 1, 0, Hq * D, 1.0)
    return int(_native.load().kv_mxfp4_attention_shared_workspace_bytes(cache._ref, ctypes.byref(a), int32(shared_blocks)))


def attention_kv_mxfp4_shared(q, cache: KvCacheMxfp4, shared_table, shared_len, block_table, seq_lens, query_start,
                              max_q_len: int, scale=None, causal: bool = True, out=None, lse=None, workspace=None,
                              stream=None):
    """Attention of ``q`` bf16 [N, Hq, head_dim] over a prefix that all requests share and each request's own keys.

    ``shared_table`` int32 [shared blocks] and ``shared_len`` int32 [1]: the prefix's pages
    and keys, read once for the whole batch.  ``block_table`` int32 [R, max_blocks] and
    ``seq_lens`` int32 [R]: what each request holds after it, on pages of its own, positions
    from 0 (the step's new tokens included); 0: only the prefix, negative: an empty
    place in the batch, whose rows are zeros (lse -inf).  Every row sees the whole prefix.  The rest as
    ``attention_kv_mxfp4``; the workspace's size is ``attention_shared_workspace_bytes``, its status
    is read by ``attention_read_status``.  For decoding batches behind a long prefix (some 200,000 tokens of
    prefix times requests); for less, and for prompts, ``attention_kv_mxfp4`` with the prefix's pages repeated in
    every row of ``block_table`` takes as long or less."""
    dev = cache.device
    N, Hq, qs = _queries(q, cache, torch.bfloat16)
    D = cache.head_dim
    if not isinstance(block_table, torch.Tensor) or not isinstance(shared_table, torch.Tensor) or not isinstance(seq_lens, torch.Tensor):
        raise TypeError("shared_table, block_table and seq_lens must be torch.Tensors")
    if block_table.dim() != 2 or shared_table.dim() != 1 or seq_lens.dim() != 1:
        raise ValueError("block_table must be [R, max_blocks], shared_table [shared blocks], seq_lens [R]")
    R, mb, sb = seq_lens.shape[0], block_table.shape[1], shared_table.shape[0]
    for t, name, shape in ((shared_table, "shared_table", (sb,)), (shared_len, "shared_len", (1,)),
                           (block_table, "block_table", (R, mb)), (seq_lens, "seq_lens", (R,)),
                           (query_start, "query_start", (R + 1,))):
        if not isinstance(t, torch.Tensor) or not _flat(t, _i32, shape, dev):
            _need(t, name, _i32, shape, dev)
    if out is None:
        out = _empty((N, Hq, D), torch.bfloat16, dev, stream)
    if not isinstance(out, torch.Tensor) or not _flat(out, torch.bfloat16, (N, Hq, D), dev):
        _need(out, "out", torch.bfloat16, (N, Hq, D), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (N, Hq), dev)
    sb = int32(sb)
    a = KvAttnStruct(int32(R), N, Hq, int32(mb), int32(max_q_len), 1 if causal else 0, 0, qs, D ** -0.5 if scale is None else scale)
    lib, ref = _native.load(), ctypes.byref(a)
    if workspace is None:
        workspace = _empty(max(256, lib.kv_mxfp4_attention_shared_workspace_bytes(cache._ref, ref, sb)), torch.uint8, dev, stream)
    elif workspace.dtype != torch.uint8 or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {dev}")
    rc = lib.kv_mxfp4_attention_shared(cache._ref, ref, sb, q.data_ptr(), shared_table.data_ptr(), shared_len.data_ptr(),
                                       block_table.data_ptr(), seq_lens.data_ptr(), query_start.data_ptr(), out.data_ptr(),
                                       None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                       _stream(stream, q))
    _native.check("kv_mxfp4_attention_shared", rc)
    return out
