"""ctypes binding of the decoding-step operators (include/nvfp4_serving.h).

Argument marshalling only, as in ``binding``: tensors are checked for type,
device and shape, missing outputs and workspaces are allocated with
``torch.empty``, and the C ABI gets raw pointers, sizes and a stream. The
launch goes to the tensors' device, whichever device is current, and to torch's
current stream there unless ``stream`` names another; what a call allocates
belongs to the stream that it launches on.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math

import torch

from . import binding as _b

EXPORTS = ("kv_block_tables", "nvfp4_paged_attention", "nvfp4_paged_attention_workspace",
           "moe_layer_nvfp4", "moe_layer_bf16", "moe_layer_workspace")

_LIB = None
_vp, _i64, _i32, _f32 = C.c_void_p, C.c_int64, C.c_int32, C.c_float


def _lib():
    global _LIB
    if _LIB is None:
        L = _b.raw()
        L.kv_block_tables.argtypes = [_vp, _vp, _i64, _i32, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp,
                                      _vp, _i64, _vp, _vp]
        L.nvfp4_paged_attention.argtypes = [_vp, _i64, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i64,
                                            _i32, _vp, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _f32, _i32,
                                            _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp]
        L.nvfp4_paged_attention_workspace.argtypes = [_i64, _i32, _i32, _i32, _i64, _i64, _i64, _i64]
        L.moe_layer_nvfp4.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i32,
                                      _i32, _i32, _vp, _i64, _vp, _vp, _vp, _i64, _vp]
        L.moe_layer_bf16.argtypes = [_vp, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _i32, _i32, _i32, _vp,
                                     _i64, _vp, _vp, _vp, _i64, _vp]
        L.moe_layer_workspace.argtypes = [_i64, _i64, _i64, _i32, _i32]
        for fn in (L.kv_block_tables, L.nvfp4_paged_attention, L.moe_layer_nvfp4, L.moe_layer_bf16):
            fn.restype = C.c_int
        L.nvfp4_paged_attention_workspace.restype = _i64
        L.moe_layer_workspace.restype = _i64
        _LIB = L
    return _LIB


def raw():
    """The loaded ctypes library with these calls' argument types set."""
    return _lib()


# ---- marshalling helpers -----------------------------------------------------
# A decoding step makes these calls for a few microseconds of GPU work each, so
# the checks below are written to be cheap: identity of dtypes, one comparison
# of shapes, and torch's raw stream handle in place of a Stream object.
_ptr = _b._ptr
_pitch = _b._pitch
Nvfp4Error = _b.Nvfp4Error
_empty = torch.empty
_I32_MAX, _I64_MAX = 2 ** 31 - 1, 2 ** 63 - 1
_BF16, _F32, _I32, _I64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


@contextlib.contextmanager
def _elsewhere(device, stream):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
        else:
            if not isinstance(stream, torch.cuda.Stream):
                # 0 is the default stream
                stream = (torch.cuda.ExternalStream(int(stream), device=device) if int(stream)
                          else torch.cuda.default_stream(device))
            elif stream.device != device:
                raise ValueError("stream belongs to another device than the tensors")
            with torch.cuda.stream(stream):
                yield stream.cuda_stream


def _current(device, stream):
    """torch's raw current stream where nothing has to be set or restored for a
    launch on `device`, else None (the default stream's handle is 0)."""
    if stream is None and device.index == torch.cuda.current_device():
        return torch._C._cuda_getCurrentRawStream(device.index)
    return None


def _check(status, what):
    if status != 0:
        raise Nvfp4Error(status, what)


def _fits(v, name, bits):
    """A size that the C call takes as a signed integer of `bits` bits; ctypes
    would cut a larger one short."""
    if not -(1 << (bits - 1)) <= v < 1 << (bits - 1):
        raise ValueError("%s does not fit %d bits" % (name, bits))
    return v


def _at_most(v, name):
    """A size of which every value past 64 bits means the same as the largest."""
    return _I64_MAX if v > _I64_MAX else _fits(v, name, 64)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    return t.device


def _vector(t, name, dtype, device, n=None):
    if t.dtype is not dtype or t.device != device or t.dim() != 1 or not t.is_contiguous():
        raise TypeError("%s must be a contiguous 1-D %s tensor on the input's device" % (name, dtype))
    if n is not None and t.numel() != n:
        raise ValueError("%s must hold %d values" % (name, n))
    return t.data_ptr()


def _all(tensors, names, dtype, device, shapes):
    """Pointers of contiguous tensors of one dtype with these shapes."""
    for t, shape in zip(tensors, shapes):
        if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
            break
    else:
        return [t.data_ptr() for t in tensors]
    for t, name, shape in zip(tensors, names, shapes):
        if t.dtype is not dtype or t.device != device or not t.is_contiguous():
            raise TypeError("%s must be a contiguous %s tensor on the input's device" % (name, dtype))
        if t.shape != shape:
            raise ValueError("%s must have shape %s" % (name, shape))


def _scalar(t, name, dtype, device):
    if t is None:
        return None
    if t.dtype is not dtype or t.device != device or t.numel() != 1:
        raise TypeError("%s must be a %s tensor of one value on the input's device" % (name, dtype))
    return t.data_ptr()


def _new(t, shape, dtype, device, name):
    return _empty(shape, dtype=dtype, device=device) if t is None else _b._out(t, shape, dtype, device, name)


def _table(t, rows, device):
    """Row pitch and columns of a block table."""
    if t.dtype is not _I32 or t.device != device or t.dim() != 2:
        raise TypeError("block_table must be a 2-D int32 tensor on the input's device")
    n, width = t.shape
    if n != rows:
        raise ValueError("block_table must have one row per request")
    if t.is_contiguous():
        return width, width
    if width > 1 and t.stride(1) != 1:
        raise TypeError("block_table must have unit column stride")
    pitch = t.stride(0) if rows > 1 else width
    if pitch < width:
        raise ValueError("block_table's rows must not overlap")
    return pitch, width


def _workspace(t, need, device):
    """The workspace's tensor (to be kept until the launch), pointer and bytes."""
    if t is None:
        if need <= 0:
            return None, None, 0
        t = _empty(need, dtype=_U8, device=device)
        return t, t.data_ptr(), need
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    return t, t.data_ptr(), t.numel() * t.element_size()


# ---- entry points --------------------------------------------------------------
def kv_block_tables(context_lens: torch.Tensor | None, query_lens: torch.Tensor,
                    block_table: torch.Tensor, page_size: int, max_tokens: int, *,
                    free_pages: torch.Tensor | None = None, free_begin: torch.Tensor | None = None,
                    slots: torch.Tensor | None = None, query_offsets: torch.Tensor | None = None,
                    seq_lens: torch.Tensor | None = None, free_end: torch.Tensor | None = None,
                    stream=None):
    """Pages and slots of requests that hold context_lens (int32 [B], None: 0)
    cached tokens and bring query_lens (int32 [B]) new ones. Pages they lack are
    taken from free_pages (int32, from free_begin[0] on) into block_table
    (int32 [B, max_pages], in place; without free_pages every page is there
    already). Returns (slots int64 [max_tokens], -1 behind the last token;
    query_offsets int32 [B + 1]; seq_lens int32 [B]; free_end int32 [1])."""
    device = _cuda(query_lens, "query_lens")
    query = _vector(query_lens, "query_lens", _I32, device)
    n = query_lens.numel()
    context = None if context_lens is None else _vector(context_lens, "context_lens", _I32, device, n)
    ld, width = _table(block_table, n, device)
    free, num_free = None, -1
    if free_pages is not None:
        free, num_free = _vector(free_pages, "free_pages", _I32, device), free_pages.numel()
    begin = _scalar(free_begin, "free_begin", _I32, device)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    if not 0 <= page_size <= _I32_MAX:
        _fits(page_size, "page_size", 32)

    def launch(st, slots, query_offsets, seq_lens, free_end):
        if slots is None:
            slots = _empty(max_tokens, dtype=_I64, device=device)
        else:
            _b._out(slots, (max_tokens,), _I64, device, "slots")
        if query_offsets is None and seq_lens is None and free_end is None:
            query_offsets, seq_lens, free_end = _empty(2 * n + 2, dtype=_I32, device=device).split_with_sizes((n + 1, n, 1))
        else:
            query_offsets = _new(query_offsets, (n + 1,), _I32, device, "query_offsets")
            seq_lens = _new(seq_lens, (n,), _I32, device, "seq_lens")
            free_end = _new(free_end, (1,), _I32, device, "free_end")
        lens, end = seq_lens.data_ptr(), free_end.data_ptr()
        if n and (lens == query or lens == context or end == begin):
            raise ValueError("outputs must not share memory with the lengths or free_begin")
        _check(_lib().kv_block_tables(context, query, n, page_size, free, num_free, begin, block_table.data_ptr(), ld, width,
                                      query_offsets.data_ptr(), lens, slots.data_ptr(), max_tokens, end, st),
               "kv_block_tables")
        return slots, query_offsets, seq_lens, free_end

    st = _current(device, stream)
    if st is not None:
        return launch(st, slots, query_offsets, seq_lens, free_end)
    with _elsewhere(device, stream) as st:
        return launch(st, slots, query_offsets, seq_lens, free_end)


def _heads(t, name, device):
    """Pitch of the rows of [tokens, heads, head_dim]."""
    if t.dtype is not _BF16 or t.device != device or t.dim() != 3:
        raise TypeError("%s must be a bfloat16 tensor [tokens, heads, head_dim] on the input's device" % name)
    n, h, d = t.shape
    if t.is_contiguous():
        return h * d
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError("%s must have packed heads (only the token stride is free)" % name)
    pitch = t.stride(0) if n > 1 else h * d
    if pitch < h * d:
        raise ValueError("%s's rows must not overlap" % name)
    return pitch


@functools.lru_cache(maxsize=256)
def _attention_workspace(*sizes):
    return _lib().nvfp4_paged_attention_workspace(*sizes)


@functools.lru_cache(maxsize=256)
def _moe_workspace(*sizes):
    return _lib().moe_layer_workspace(*sizes)


def nvfp4_paged_attention(q: torch.Tensor, k_packed: torch.Tensor, k_scales: torch.Tensor,
                          v_packed: torch.Tensor, v_scales: torch.Tensor, block_table: torch.Tensor,
                          seq_lens: torch.Tensor, query_offsets: torch.Tensor, *, kv_heads: int,
                          page_size: int, max_query_len: int, max_seq_len: int | None = None,
                          scale: float | None = None, causal: bool = True, window: int = 0,
                          k_gs: torch.Tensor | None = None, v_gs: torch.Tensor | None = None,
                          out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None,
                          workspace: torch.Tensor | None = None, stream=None):
    """q BF16 [tokens, heads, head_dim] attends to the NVFP4 cache that
    nvfp4_quantize_paged writes (packed [num_slots, kv_heads * head_dim / 2],
    scales [num_slots, kv_heads * head_dim / 16]) through block_table int32
    [B, max_pages]; request b owns rows query_offsets[b]..query_offsets[b+1]
    of q, at the end of its seq_lens[b] tokens. max_query_len and max_seq_len
    (default: the table's width) steer the speed only; a max_seq_len far above
    the real lengths costs time and workspace. scale defaults to
    head_dim ** -0.5; window > 0 keeps the last `window` positions. Returns out
    (BF16, like q) and, with ``lse`` True or a tensor, also lse FP32
    [tokens, heads]. Rows of no request are left as they were (``out`` and
    ``lse`` allocated here hold nothing there)."""
    device = _cuda(q, "q")
    ld_q = _heads(q, "q", device)
    tokens, heads, dim = q.shape
    if k_packed.dim() != 2:
        raise ValueError("k_packed must be [num_slots, kv_heads * head_dim / 2]")
    slots, cols = k_packed.shape[0], kv_heads * dim
    codes, scales = (slots, cols // 2), (slots, cols // 16)
    kp, ks, vp, vs = _all((k_packed, k_scales, v_packed, v_scales), ("k_packed", "k_scales", "v_packed", "v_scales"), _U8,
                          device, (codes, scales, codes, scales))
    lens = _vector(seq_lens, "seq_lens", _I32, device)
    n = seq_lens.numel()
    offsets = _vector(query_offsets, "query_offsets", _I32, device, n + 1)
    ld_table, max_pages = _table(block_table, n, device)
    kg = _scalar(k_gs, "k_gs", _F32, device)
    vg = _scalar(v_gs, "v_gs", _F32, device)
    if max_seq_len is None:
        max_seq_len = max_pages * page_size
    if not (0 <= page_size <= _I32_MAX and 0 <= max_query_len <= _I64_MAX and 0 <= max_seq_len <= _I64_MAX
            and 0 <= window <= _I64_MAX):
        _fits(page_size, "page_size", 32)
        max_query_len, window = _at_most(max_query_len, "max_query_len"), _at_most(window, "window")
        max_seq_len = _at_most(max_seq_len, "max_seq_len")
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    L = _lib()
    need = _attention_workspace(tokens, heads, kv_heads, dim, n, max_query_len, max_seq_len, window)

    def launch(st, out, lse):
        if out is None:
            out = _empty((tokens, heads, dim), dtype=_BF16, device=device)
            ld_out = heads * dim
        else:
            ld_out = _heads(out, "out", device)
            if out.shape != q.shape:
                raise ValueError("out must have q's shape")
        zp = None
        if lse is None or lse is False:
            lse = None
        else:
            lse = _new(None if lse is True else lse, (tokens, heads), _F32, device, "lse")
            zp = lse.data_ptr()
        work, wp, size = _workspace(workspace, need, device)
        _check(L.nvfp4_paged_attention(q.data_ptr(), tokens, ld_q, heads, kv_heads, dim, kp, ks, vp, vs, slots, page_size,
                                       block_table.data_ptr(), ld_table, max_pages, lens, offsets, n, max_query_len,
                                       max_seq_len, scale, 1 if causal else 0, window, kg, vg, out.data_ptr(), ld_out, zp,
                                       wp, size, st), "nvfp4_paged_attention")
        return out if lse is None else (out, lse)

    st = _current(device, stream)
    if st is not None:
        return launch(st, out, lse)
    with _elsewhere(device, stream) as st:
        return launch(st, out, lse)


def _moe(fn, what, x, logits, top_k, inter, weights, renormalize, out, topk_ids, topk_weights, workspace, stream):
    device = x.device
    tokens, hidden = x.shape
    experts = logits.shape[1]
    if not 0 <= top_k <= _I32_MAX:
        _fits(top_k, "top_k", 32)
    need = _moe_workspace(tokens, hidden, inter, experts, top_k)

    def launch(st, out, topk_ids, topk_weights):
        if out is None:
            out = _empty((tokens, hidden), dtype=_BF16, device=device)
        elif (out.dtype is not _BF16 or out.device != device or out.shape != (tokens, hidden)
              or (hidden > 1 and out.stride(1) != 1)):
            raise ValueError("out must be a bfloat16 tensor of shape (tokens, hidden) with unit column stride")
        topk_ids = _new(topk_ids, (tokens, max(top_k, 0)), _I32, device, "topk_ids")
        topk_weights = _new(topk_weights, (tokens, max(top_k, 0)), _F32, device, "topk_weights")
        work, wp, size = _workspace(workspace, need, device)
        _check(fn(x.data_ptr(), tokens, _pitch(x), logits.data_ptr(), *weights, hidden, inter, experts, top_k,
                  1 if renormalize else 0, out.data_ptr(), _pitch(out), topk_ids.data_ptr(), topk_weights.data_ptr(), wp,
                  size, st), what)
        return out, topk_ids, topk_weights

    st = _current(device, stream)
    if st is not None:
        return launch(st, out, topk_ids, topk_weights)
    with _elsewhere(device, stream) as st:
        return launch(st, out, topk_ids, topk_weights)


def _moe_inputs(x, logits):
    device = _cuda(x, "x")
    if x.dtype is not _BF16 or x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise TypeError("x must be a 2-D bfloat16 tensor with unit column stride")
    if logits.dim() != 2 or logits.shape[0] != x.shape[0]:
        raise ValueError("logits must be [tokens, num_experts]")
    if logits.dtype is not _F32 or logits.device != device or not logits.is_contiguous():
        raise TypeError("logits must be a contiguous float32 tensor on x's device")
    return device


def moe_layer_nvfp4(x: torch.Tensor, logits: torch.Tensor, w1_packed: torch.Tensor, w1_scales: torch.Tensor,
                    w2_packed: torch.Tensor, w2_scales: torch.Tensor, top_k: int,
                    gs1: torch.Tensor | None = None, gs2: torch.Tensor | None = None, *,
                    renormalize: bool = True, out: torch.Tensor | None = None,
                    topk_ids: torch.Tensor | None = None, topk_weights: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, stream=None):
    """A whole mixture-of-experts layer for 1 to 64 tokens with NVFP4 weights:
    x BF16 [tokens, H], logits FP32 [tokens, E], w1 [E, 2I, H] (rows = interleaved
    [gate x8, up x8, ...] columns) and w2 [E, H, I] as nvfp4_quantize writes their
    rows (packed uint8 [.., cols / 2], scales uint8 [.., cols / 16], gs FP32 [E]).
    Returns (out BF16 [tokens, H], topk_ids int32 [tokens, top_k],
    topk_weights FP32 [tokens, top_k])."""
    device = _moe_inputs(x, logits)
    e, hidden = logits.shape[1], x.shape[1]
    if w1_packed.dim() != 3 or w1_packed.shape[1] % 2:
        raise ValueError("w1_packed must be [E, 2I, H / 2]")
    inter = w1_packed.shape[1] // 2
    w1p, w1s, w2p, w2s = _all((w1_packed, w1_scales, w2_packed, w2_scales), ("w1_packed", "w1_scales", "w2_packed", "w2_scales"),
                              _U8, device, ((e, 2 * inter, hidden // 2), (e, 2 * inter, hidden // 16),
                                            (e, hidden, inter // 2), (e, hidden, inter // 16)))
    weights = (w1p, w1s, None if gs1 is None else _vector(gs1, "gs1", _F32, device, e),
               w2p, w2s, None if gs2 is None else _vector(gs2, "gs2", _F32, device, e))
    return _moe(_lib().moe_layer_nvfp4, "moe_layer_nvfp4", x, logits, top_k, inter, weights, renormalize, out, topk_ids,
                topk_weights, workspace, stream)


def moe_layer_bf16(x: torch.Tensor, logits: torch.Tensor, w1: torch.Tensor, w2: torch.Tensor, top_k: int, *,
                   renormalize: bool = True, out: torch.Tensor | None = None,
                   topk_ids: torch.Tensor | None = None, topk_weights: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """moe_layer_nvfp4 with BF16 weights: w1 [E, 2I, H] (as for moe_l1_gemm_bf16)
    and w2 [E, H, I]."""
    device = _moe_inputs(x, logits)
    e, hidden = logits.shape[1], x.shape[1]
    if w1.dim() != 3 or w1.shape[1] % 2:
        raise ValueError("w1 must be [E, 2I, H]")
    inter = w1.shape[1] // 2
    weights = _all((w1, w2), ("w1", "w2"), _BF16, device, ((e, 2 * inter, hidden), (e, hidden, inter)))
    return _moe(_lib().moe_layer_bf16, "moe_layer_bf16", x, logits, top_k, inter, weights, renormalize, out, topk_ids,
                topk_weights, workspace, stream)
