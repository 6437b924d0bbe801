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
_ptr = _b._ptr
_pitch = _b._pitch
_call = _b._call


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


def _launch(device, stream):
    """Context of the allocations and the launch; gives the raw stream."""
    if stream is None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext(torch.cuda.current_stream(device).cuda_stream)
    return _elsewhere(device, stream)


def _cuda(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    return t.device


def _vector(t, name, dtype, device, n=None):
    if t.dtype != dtype or t.device != device or t.dim() != 1 or not t.is_contiguous():
        raise TypeError("%s must be a contiguous 1-D %s tensor on the input's device" % (name, dtype))
    if n is not None and t.numel() != n:
        raise ValueError("%s must hold %d values" % (name, n))
    return t


def _scalar(t, name, dtype, device):
    if t is None:
        return None
    if t.dtype != dtype or t.device != device or t.numel() != 1:
        raise TypeError("%s must be a %s tensor of one value on the input's device" % (name, dtype))
    return t


def _new(t, shape, dtype, device, name):
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _b._out(t, shape, dtype, device, name)


def _table(t, rows, device):
    if t.dtype != torch.int32 or t.device != device or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise TypeError("block_table must be a 2-D int32 tensor with unit column stride on the input's device")
    if t.shape[0] != rows:
        raise ValueError("block_table must have one row per request")
    pitch = t.stride(0) if rows > 1 else t.shape[1]
    if pitch < t.shape[1]:
        raise ValueError("block_table's rows must not overlap")
    return pitch


def _workspace(t, need, device):
    if t is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    if t.device != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the input's device")
    return t


def _bytes(t):
    return 0 if t is None else t.numel() * t.element_size()


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
    _vector(query_lens, "query_lens", torch.int32, device)
    n = query_lens.numel()
    if context_lens is not None:
        _vector(context_lens, "context_lens", torch.int32, device, n)
    ld = _table(block_table, n, device)
    if free_pages is not None:
        _vector(free_pages, "free_pages", torch.int32, device)
    _scalar(free_begin, "free_begin", torch.int32, device)
    if max_tokens < 0:
        raise ValueError("max_tokens must not be negative")
    with _launch(device, stream) as st:
        slots = _new(slots, (max_tokens,), torch.int64, device, "slots")
        query_offsets = _new(query_offsets, (n + 1,), torch.int32, device, "query_offsets")
        seq_lens = _new(seq_lens, (n,), torch.int32, device, "seq_lens")
        free_end = _new(free_end, (1,), torch.int32, device, "free_end")
        if n and (seq_lens.data_ptr() in (query_lens.data_ptr(), 0 if context_lens is None else context_lens.data_ptr())
                  or (free_begin is not None and free_end.data_ptr() == free_begin.data_ptr())):
            raise ValueError("outputs must not share memory with the lengths or free_begin")
        _call(_lib().kv_block_tables, "kv_block_tables", _ptr(context_lens), query_lens.data_ptr(), n,
              page_size, _ptr(free_pages), -1 if free_pages is None else free_pages.numel(), _ptr(free_begin),
              block_table.data_ptr(), ld, block_table.shape[1], query_offsets.data_ptr(), seq_lens.data_ptr(),
              slots.data_ptr(), max_tokens, free_end.data_ptr(), st)
    return slots, query_offsets, seq_lens, free_end


def _heads(t, name, device):
    if t.dtype != torch.bfloat16 or t.device != device or t.dim() != 3:
        raise TypeError("%s must be a bfloat16 tensor [tokens, heads, head_dim] on the input's device" % name)
    n, h, d = t.shape
    if (d > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != d):
        raise ValueError("%s must have packed heads (only the token stride is free)" % name)
    pitch = t.stride(0) if n > 1 else h * d
    if pitch < h * d:
        raise ValueError("%s's rows must not overlap" % name)
    return pitch


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
    (default: the table's width) steer the speed only. scale defaults to
    head_dim ** -0.5; window > 0 keeps the last `window` positions. Returns out
    (BF16, like q) and, with ``lse`` True or a tensor, also lse FP32
    [tokens, heads]. Rows of no request are left as they were (``out`` and
    ``lse`` allocated here hold nothing there)."""
    device = _cuda(q, "q")
    ld_q = _heads(q, "q", device)
    tokens, heads, dim = q.shape
    for t, name, w in ((k_packed, "k_packed", 2), (k_scales, "k_scales", 16), (v_packed, "v_packed", 2),
                       (v_scales, "v_scales", 16)):
        if t.dtype != torch.uint8 or t.device != device or t.dim() != 2 or not t.is_contiguous():
            raise TypeError("%s must be a contiguous 2-D uint8 tensor on the input's device" % name)
        if t.shape[0] != k_packed.shape[0] or t.shape[1] != kv_heads * dim // w:
            raise ValueError("%s must be [num_slots, kv_heads * head_dim / %d]" % (name, w))
    num_slots = k_packed.shape[0]
    _vector(seq_lens, "seq_lens", torch.int32, device)
    n = seq_lens.numel()
    _vector(query_offsets, "query_offsets", torch.int32, device, n + 1)
    ld_table = _table(block_table, n, device)
    max_pages = block_table.shape[1]
    _scalar(k_gs, "k_gs", torch.float32, device)
    _scalar(v_gs, "v_gs", torch.float32, device)
    if max_seq_len is None:
        max_seq_len = max_pages * page_size
    if scale is None:
        scale = 1.0 / math.sqrt(dim) if dim else 1.0
    L = _lib()
    need = L.nvfp4_paged_attention_workspace(tokens, heads, kv_heads, dim, n, max_query_len, max_seq_len, window)
    with _launch(device, stream) as st:
        if out is None:
            out = torch.empty((tokens, heads, dim), dtype=torch.bfloat16, device=device)
        ld_out = _heads(out, "out", device)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
        z = None
        if lse is True:
            z = torch.empty((tokens, heads), dtype=torch.float32, device=device)
        elif isinstance(lse, torch.Tensor):
            z = _b._out(lse, (tokens, heads), torch.float32, device, "lse")
        work = _workspace(workspace, need, device)
        _call(L.nvfp4_paged_attention, "nvfp4_paged_attention", q.data_ptr(), tokens, ld_q, heads, kv_heads, dim,
              k_packed.data_ptr(), k_scales.data_ptr(), v_packed.data_ptr(), v_scales.data_ptr(), num_slots,
              page_size, block_table.data_ptr(), ld_table, max_pages, seq_lens.data_ptr(),
              query_offsets.data_ptr(), n, max_query_len, max_seq_len, scale, int(causal), window, _ptr(k_gs),
              _ptr(v_gs), out.data_ptr(), ld_out, _ptr(z), _ptr(work), _bytes(work), st)
    return out if z is None else (out, z)


def _matrix(t, name, dtype, device, shape):
    if t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise TypeError("%s must be a contiguous %s tensor on the input's device" % (name, dtype))
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s" % (name, shape))
    return t


def _moe(fn, what, x, logits, top_k, inter, weights, renormalize, out, topk_ids, topk_weights, workspace, stream):
    device = x.device
    tokens, hidden = x.shape
    experts = logits.shape[1]
    need = _lib().moe_layer_workspace(tokens, hidden, inter, experts, top_k)
    with _launch(device, stream) as st:
        if out is None:
            out = torch.empty((tokens, hidden), dtype=torch.bfloat16, device=device)
        if (out.dtype != torch.bfloat16 or out.device != device or tuple(out.shape) != (tokens, hidden)
                or (hidden > 1 and out.stride(1) != 1)):
            raise ValueError("out must be a bfloat16 tensor of shape (tokens, hidden) with unit column stride")
        topk_ids = _new(topk_ids, (tokens, max(top_k, 0)), torch.int32, device, "topk_ids")
        topk_weights = _new(topk_weights, (tokens, max(top_k, 0)), torch.float32, device, "topk_weights")
        work = _workspace(workspace, need, device)
        _call(fn, what, x.data_ptr(), tokens, _pitch(x), logits.data_ptr(), *[_ptr(w) for w in weights], hidden,
              inter, experts, top_k, int(renormalize), out.data_ptr(), _pitch(out), topk_ids.data_ptr(),
              topk_weights.data_ptr(), _ptr(work), _bytes(work), st)
    return out, topk_ids, topk_weights


def _moe_inputs(x, logits):
    device = _cuda(x, "x")
    if x.dtype != torch.bfloat16 or x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise TypeError("x must be a 2-D bfloat16 tensor with unit column stride")
    if logits.dim() != 2 or logits.shape[0] != x.shape[0]:
        raise ValueError("logits must be [tokens, num_experts]")
    _matrix(logits, "logits", torch.float32, device, tuple(logits.shape))
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
    for t, name, shape in ((w1_packed, "w1_packed", (e, 2 * inter, hidden // 2)),
                           (w1_scales, "w1_scales", (e, 2 * inter, hidden // 16)),
                           (w2_packed, "w2_packed", (e, hidden, inter // 2)),
                           (w2_scales, "w2_scales", (e, hidden, inter // 16))):
        _matrix(t, name, torch.uint8, device, shape)
    for t, name in ((gs1, "gs1"), (gs2, "gs2")):
        if t is not None:
            _vector(t, name, torch.float32, device, e)
    return _moe(_lib().moe_layer_nvfp4, "moe_layer_nvfp4", x, logits, top_k, inter,
                (w1_packed, w1_scales, gs1, w2_packed, w2_scales, gs2), renormalize, out, topk_ids, topk_weights,
                workspace, stream)


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
    _matrix(w1, "w1", torch.bfloat16, device, (e, 2 * inter, hidden))
    _matrix(w2, "w2", torch.bfloat16, device, (e, hidden, inter))
    return _moe(_lib().moe_layer_bf16, "moe_layer_bf16", x, logits, top_k, inter, (w1, w2), renormalize, out, topk_ids,
                topk_weights, workspace, stream)
