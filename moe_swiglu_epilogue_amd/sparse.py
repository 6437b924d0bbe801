"""ctypes binding of the sparse-attention operators (include/nvfp4_sparse.h).

Argument marshalling only, as in ``serving``, whose helpers and rules hold here:
tensors are checked for type, device and shape, missing outputs and workspaces
are allocated with ``torch.empty``, and the launch goes to the tensors' device
and to torch's current stream there unless ``stream`` names another.
"""
from __future__ import annotations

import ctypes as C
import functools
import math

import torch

from . import binding as _b
from .serving import (_BF16, _F32, _I32, _I32_MAX, _I64, _U8, _all, _at_most, _check, _cuda, _current, _elsewhere, _empty,
                      _heads, _scalar, _table, _vector, _workspace)

EXPORTS = ("nvfp4_rope_append", "nvfp4_page_keys", "nvfp4_select_pages", "nvfp4_select_pages_workspace",
           "nvfp4_sparse_attention", "nvfp4_sparse_attention_workspace")

_LIB = None
_I8 = torch.int8
_vp, _i64, _i32, _f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_float


def _lib():
    global _LIB
    if _LIB is None:
        L = _b.raw()
        L.nvfp4_rope_append.argtypes = [_vp, _i64, _i64, _i32, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _i64, _i32, _vp, _vp,
                                        _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp]
        L.nvfp4_page_keys.argtypes = [_vp, _vp, _i64, _i32, _i32, _i32, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _vp]
        L.nvfp4_select_pages.argtypes = [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _i64, _i32, _vp, _i64, _i64, _vp, _vp,
                                         _i64, _i32, _i32, _i32, _vp, _vp, _i64, _vp]
        L.nvfp4_select_pages_workspace.argtypes = [_i64, _i32, _i32, _i64, _i64]
        L.nvfp4_sparse_attention.argtypes = [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64, _i32, _vp, _i64, _i64,
                                             _vp, _vp, _i64, _vp, _i64, _f32, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp]
        L.nvfp4_sparse_attention_workspace.argtypes = [_i64, _i32, _i32, _i32, _i32, _i64, _i64]
        for fn in (L.nvfp4_rope_append, L.nvfp4_page_keys, L.nvfp4_select_pages, L.nvfp4_sparse_attention):
            fn.restype = C.c_int
        L.nvfp4_select_pages_workspace.restype = _i64
        L.nvfp4_sparse_attention_workspace.restype = _i64
        _LIB = L
    return _LIB


def raw():
    """The loaded ctypes library with these calls' argument types set."""
    return _lib()


def _run(launch, device, stream):
    st = _current(device, stream)
    if st is not None:
        return launch(st)
    with _elsewhere(device, stream) as st:
        return launch(st)


# The checks of a call that passes, in as few steps as they take (a call of a few
# microseconds looks at a dozen tensors); what does not pass goes to serving's checks,
# which say what is wrong.
def _rows(t, name, device, index):
    """Pitch of the rows of [tokens, heads, head_dim]."""
    if t.dtype is _BF16 and t.get_device() == index and t.dim() == 3:
        n, h, d = t.shape
        row, head, one = t.stride()
        if head == d and one == 1:
            if n <= 1:
                return h * d
            if row >= h * d:
                return row
    return _heads(t, name, device)


def _line(t, name, dtype, device, index, n):
    """Pointer of a contiguous vector of n values."""
    if t.dtype is dtype and t.get_device() == index and t.dim() == 1 and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    return _vector(t, name, dtype, device, n)


def _caches(tensors, names, device, index, codes, scales):
    """Pointers of packed and scale caches in turn."""
    for t, shape in zip(tensors, (codes, scales, codes, scales)):
        if t.dtype is not _U8 or t.get_device() != index or t.shape != shape or not t.is_contiguous():
            return _all(tensors, names, _U8, device, (codes, scales, codes, scales)[:len(tensors)])
    return [t.data_ptr() for t in tensors]


def _one(t, name, device, index):
    """Pointer of a global scale, or None."""
    if t is None:
        return None
    if t.dtype is _F32 and t.get_device() == index and t.numel() == 1:
        return t.data_ptr()
    return _scalar(t, name, _F32, device)


def _page_size(v):
    if not 1 <= v <= _I32_MAX:
        raise ValueError("page_size must be at least 1 and fit 32 bits")


_CACHES = ("k_packed", "k_scales", "v_packed", "v_scales")


@functools.lru_cache(maxsize=256)
def _select_workspace(*sizes):
    return _lib().nvfp4_select_pages_workspace(*sizes)


@functools.lru_cache(maxsize=256)
def _sparse_workspace(*sizes):
    return _lib().nvfp4_sparse_attention_workspace(*sizes)


# ---- entry points --------------------------------------------------------------
def nvfp4_rope_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                      cos_sin: torch.Tensor, slot_mapping: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor,
                      v_packed: torch.Tensor, v_scales: torch.Tensor, *, pair_axis: torch.Tensor | None = None,
                      interleaved: bool = False, k_gs: torch.Tensor | None = None, v_gs: torch.Tensor | None = None,
                      q_out: torch.Tensor | None = None, stream=None):
    """Rotates q BF16 [tokens, heads, head_dim] and k BF16 [tokens, kv_heads,
    head_dim] by their positions and writes k and v into rows slot_mapping (int64
    [tokens]) of the NVFP4 caches, in place, as nvfp4_quantize_paged does with
    k_gs and v_gs; tokens whose slot is outside the cache are not written there.
    q, k and v may be views of one projection (only the token stride is free).
    positions int32 [tokens], or [axes, tokens] with pair_axis int32 [rot_dim / 2]
    the axis of each pair of dimensions (without it: the first); cos_sin FP32
    [max_position, rot_dim], a position's cosines, then its sines. Pairs are
    (j, j + rot_dim / 2), or (2 j, 2 j + 1) with interleaved; dimensions from
    rot_dim on and pairs without a valid position or axis stay as they are.
    Returns the rotated q (BF16, like q; a new tensor, or q_out), or None without
    q."""
    device = _cuda(k, "k")
    index = device.index
    ld_k, ld_v = _rows(k, "k", device, index), _rows(v, "v", device, index)
    shape = k.shape
    tokens, kv, dim = shape
    if v.shape != shape:
        raise ValueError("v must have k's shape")
    ld_q = heads = 0
    if q is not None:
        ld_q = _rows(q, "q", device, index)
        n, heads, d = q.shape
        if n != tokens or d != dim:
            raise ValueError("q must be [tokens, heads, head_dim] with k's tokens and head_dim")
        if heads < 1:
            raise ValueError("q must have at least one head")
    elif q_out is not None:
        raise ValueError("q_out without q")
    axes = positions.dim()
    if positions.dtype is not _I32 or positions.get_device() != index or not 1 <= axes <= 2:
        raise TypeError("positions must be an int32 tensor [tokens] or [axes, tokens] on the input's device")
    if axes == 2:
        axes, n = positions.shape
        ld_pos, step = positions.stride()
    else:
        n, ld_pos, step = positions.numel(), tokens, positions.stride(0)
    if n != tokens or axes < 1:
        raise ValueError("positions must hold one value per token and axis")
    if tokens > 1 and step != 1:
        raise TypeError("positions must have unit token stride")
    if axes == 1:
        ld_pos = tokens
    elif ld_pos < tokens:
        raise ValueError("positions' axes must not overlap")
    if cos_sin.dtype is not _F32 or cos_sin.get_device() != index or cos_sin.dim() != 2 or not cos_sin.is_contiguous():
        raise TypeError("cos_sin must be a contiguous 2-D float32 tensor on the input's device")
    most, rot = cos_sin.shape
    if rot % 2 or rot > dim:
        raise ValueError("cos_sin must be [max_position, rot_dim] with rot_dim even, at most head_dim")
    axis = None if pair_axis is None else _line(pair_axis, "pair_axis", _I32, device, index, rot // 2)
    slots = _line(slot_mapping, "slot_mapping", _I64, device, index, tokens)
    if k_packed.dim() != 2:
        raise ValueError("k_packed must be [num_slots, kv_heads * head_dim / 2]")
    rows, cols = k_packed.shape[0], kv * dim
    kp, ks, vp, vs = _caches((k_packed, k_scales, v_packed, v_scales), _CACHES, device, index, (rows, cols // 2),
                             (rows, cols // 16))
    kg, vg = _one(k_gs, "k_gs", device, index), _one(v_gs, "v_gs", device, index)

    def launch(st):
        out, op, ld_out = q_out, None, 0
        if q is not None:
            if out is None:
                out = _empty(tokens, heads, dim, dtype=_BF16, device=device)
                ld_out = heads * dim
            else:
                ld_out = _rows(out, "q_out", device, index)
                if out.shape != q.shape:
                    raise ValueError("q_out must have q's shape")
            op = out.data_ptr()
        # a tensor without elements has no address: without rows nothing is looked at
        _check(_lib().nvfp4_rope_append(None if q is None else q.data_ptr(), tokens, ld_q, heads, k.data_ptr(), ld_k,
                                        v.data_ptr(), ld_v, kv, dim, positions.data_ptr(), ld_pos, axes, axis,
                                        cos_sin.data_ptr(), most, rot, 1 if interleaved else 0, kg, vg, slots, rows, kp, ks,
                                        vp, vs, op, ld_out, st), "nvfp4_rope_append")
        return out

    return _run(launch, device, stream)


def _requests(block_table, seq_lens, query_offsets, device, index):
    n = seq_lens.numel()
    lens = _line(seq_lens, "seq_lens", _I32, device, index, n)
    offsets = _line(query_offsets, "query_offsets", _I32, device, index, n + 1)
    if block_table.dtype is _I32 and block_table.get_device() == index and block_table.dim() == 2 and block_table.is_contiguous():
        rows, width = block_table.shape
        if rows == n:
            return n, block_table.data_ptr(), width, width, lens, offsets
    ld, width = _table(block_table, n, device)
    return n, block_table.data_ptr(), ld, width, lens, offsets


def _page_keys(keys, exponents, index):
    if keys.dtype is not _I8 or keys.get_device() != index or keys.dim() != 3 or not keys.is_contiguous():
        raise TypeError("keys must be a contiguous int8 tensor [pages, kv_heads, head_dim] on the input's device")
    pages, kv, dim = keys.shape
    if exponents.dtype is not _I8 or exponents.get_device() != index or not exponents.is_contiguous():
        raise TypeError("exponents must be a contiguous int8 tensor on the input's device")
    if exponents.shape != (pages, kv):
        raise ValueError("exponents must be [pages, kv_heads]")
    return pages, kv, dim


def nvfp4_page_keys(k_packed: torch.Tensor, k_scales: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                    query_offsets: torch.Tensor, keys: torch.Tensor, exponents: torch.Tensor, *, page_size: int,
                    max_query_len: int, stream=None):
    """Writes the keys of the pages that the new tokens of each request complete
    (seq_lens and query_offsets as kv_block_tables gives them, the tokens in the
    cache) into keys int8 [pages, kv_heads, head_dim] and exponents int8 [pages,
    kv_heads], in place; other pages' keys keep their values. max_query_len, the
    most new tokens of a request, steers the speed only. Returns (keys, exponents)."""
    device = _cuda(k_packed, "k_packed")
    index = device.index
    pages, kv, dim = _page_keys(keys, exponents, index)
    _page_size(page_size)
    rows = pages * page_size
    kp, ks = _caches((k_packed, k_scales), _CACHES, device, index, (rows, kv * dim // 2), (rows, kv * dim // 16))
    n, table, ld, width, lens, offsets = _requests(block_table, seq_lens, query_offsets, device, index)
    max_query_len = _at_most(max_query_len, "max_query_len")

    def launch(st):
        _check(_lib().nvfp4_page_keys(kp, ks, rows, kv, dim, page_size, table, ld, width, lens, offsets, n, max_query_len,
                                      keys.data_ptr(), exponents.data_ptr(), st), "nvfp4_page_keys")
        return keys, exponents

    return _run(launch, device, stream)


def nvfp4_select_pages(q: torch.Tensor, keys: torch.Tensor, exponents: torch.Tensor, block_table: torch.Tensor,
                       seq_lens: torch.Tensor, query_offsets: torch.Tensor, *, page_size: int, top_k: int, first: int = 1,
                       local: int = 2, pages: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, stream=None):
    """The pages that each token of q BF16 [tokens, heads, head_dim] attends to, for
    each key/value head: the first `first` pages of its request, the last `local`
    up to its own, and the top_k others with the largest score by the page keys
    (ties to the lower page). Returns int32 [tokens, kv_heads, first + top_k +
    local], page numbers within the request in ascending order, -1 behind them.
    Rows of no request are left as they were (``pages`` allocated here holds
    nothing there). The work is cut by the table's width: of a table wider than the
    longest request pass the columns that it needs, ``block_table[:, :n]``."""
    device = _cuda(q, "q")
    index = device.index
    ld_q = _rows(q, "q", device, index)
    tokens, heads, dim = q.shape
    count, kv, key_dim = _page_keys(keys, exponents, index)
    if key_dim != dim:
        raise ValueError("keys must have q's head_dim")
    _page_size(page_size)
    listed = first + top_k + local
    if first < 0 or top_k < 0 or local < 1 or listed > 2048:
        raise ValueError("first and top_k must be at least 0, local at least 1, and their sum at most 2048")
    n, table, ld, width, lens, offsets = _requests(block_table, seq_lens, query_offsets, device, index)
    need = _select_workspace(tokens, heads, kv, n, width)

    def launch(st):
        out = pages
        if out is None:
            out = _empty(tokens, kv, listed, dtype=_I32, device=device)
        else:
            _b._out(out, (tokens, kv, listed), _I32, device, "pages")
        work, wp, size = _workspace(workspace, need, device)
        _check(_lib().nvfp4_select_pages(q.data_ptr(), tokens, ld_q, heads, kv, dim, keys.data_ptr(), exponents.data_ptr(),
                                         count * page_size, page_size, table, ld, width, lens, offsets, n, top_k, first,
                                         local, out.data_ptr(), wp, size, st), "nvfp4_select_pages")
        return out

    return _run(launch, device, stream)


def nvfp4_sparse_attention(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor, v_packed: torch.Tensor,
                           v_scales: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                           query_offsets: torch.Tensor, pages: torch.Tensor, *, page_size: int, scale: float | None = None,
                           k_gs: torch.Tensor | None = None, v_gs: torch.Tensor | None = None,
                           out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None,
                           workspace: torch.Tensor | None = None, stream=None):
    """nvfp4_paged_attention over listed pages alone: each token of q BF16 [tokens,
    heads, head_dim] attends to the tokens up to its own position in the pages
    pages[token, kv head] (int32 [tokens, kv_heads, list_len], page numbers within
    the request, as nvfp4_select_pages gives them; -1 and other numbers outside the
    table show nothing, a page listed twice counts twice). Returns out (BF16, like
    q) and, with ``lse`` True or a tensor, also lse FP32 [tokens, heads]. Rows of
    no request are left as they were."""
    device = _cuda(q, "q")
    index = device.index
    ld_q = _rows(q, "q", device, index)
    tokens, heads, dim = q.shape
    if pages.dtype is not _I32 or pages.get_device() != index or pages.dim() != 3 or not pages.is_contiguous():
        raise TypeError("pages must be a contiguous int32 tensor [tokens, kv_heads, list_len] on the input's device")
    lists, kv, listed = pages.shape
    if lists != tokens:
        raise ValueError("pages must have one list per token")
    if k_packed.dim() != 2:
        raise ValueError("k_packed must be [num_slots, kv_heads * head_dim / 2]")
    rows, cols = k_packed.shape[0], kv * dim
    kp, ks, vp, vs = _caches((k_packed, k_scales, v_packed, v_scales), _CACHES, device, index, (rows, cols // 2),
                             (rows, cols // 16))
    _page_size(page_size)
    if rows % page_size:
        raise ValueError("the cache must hold whole pages")
    n, table, ld, width, lens, offsets = _requests(block_table, seq_lens, query_offsets, device, index)
    kg, vg = _one(k_gs, "k_gs", device, index), _one(v_gs, "v_gs", device, index)
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    need = _sparse_workspace(tokens, heads, kv, dim, page_size, n, listed)

    def launch(st):
        o, z, zp = out, None, None
        if o is None:
            o = _empty(tokens, heads, dim, dtype=_BF16, device=device)
            ld_out = heads * dim
        else:
            ld_out = _rows(o, "out", device, index)
            if o.shape != q.shape:
                raise ValueError("out must have q's shape")
        if lse is not None and lse is not False:
            z = (_empty(tokens, heads, dtype=_F32, device=device) if lse is True
                 else _b._out(lse, (tokens, heads), _F32, device, "lse"))
            zp = z.data_ptr()
        work, wp, size = _workspace(workspace, need, device)
        _check(_lib().nvfp4_sparse_attention(q.data_ptr(), tokens, ld_q, heads, kv, dim, kp, ks, vp, vs, rows, page_size, table,
                                             ld, width, lens, offsets, n, pages.data_ptr(), listed, scale, kg, vg,
                                             o.data_ptr(), ld_out, zp, wp, size, st), "nvfp4_sparse_attention")
        return o if z is None else (o, z)

    return _run(launch, device, stream)
