"""Plain definitions of the decoding-step operators (include/nvfp4_serving.h)
in Python integers and float64, with the error bounds their GPU results must
keep. CPU only; shares no code with the product.

Bounds count roundings: a rounding to a type is off by at most eps / 2 relative
(BF16 2^-8, FP16 2^-11, FP32 2^-24); an FP32 sum of n terms is off by at most
n 2^-24 times the sum of their magnitudes; a hardware exp or log by 2^-21
relative.
"""
import math

import numpy as np
import torch

MAGNITUDES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def nvfp4_values(packed, scales):
    """uint8 [..., n/2], [..., n/16] -> float64 [..., n]."""
    p = packed.long()
    code = torch.stack([p & 15, p >> 4], -1).flatten(-2)
    v = MAGNITUDES[code & 7] * torch.where(code >= 8, -1.0, 1.0).double()
    s = scales.long()
    e, m = s >> 3, (s & 7).double()
    s = torch.where(e == 0, m / 512, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return v * s.repeat_interleave(16, -1)


def random_nvfp4(g, *shape):
    """Random codes and scales (subnormal, small and large ones) for values [*shape]."""
    packed = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(0x20, 0x41, (*shape[:-1], shape[-1] // 16), generator=g, dtype=torch.uint8)
    scales[..., 0].random_(0, 0x7f, generator=g) if shape[-1] > 64 else None
    return packed, scales


# ---- block tables ----------------------------------------------------------------
def kv_block_tables(context, query, table, page, max_tokens, free=None, begin=None):
    """All arguments plain lists / ints; `table` a list of rows that is changed in place."""
    top = 2 ** 31 - 1
    width = len(table[0]) if table else 0
    first = 0 if begin is None else begin
    pages = list(free) if free is not None else []
    if first < 0 or first > len(pages):
        first, pages = 0, []
    slots, offsets, lens, taken = [], [0], [], 0
    for b, n in enumerate(query):
        c = max(context[b], 0) if context is not None else 0
        total = min(c + max(n, 0), top)
        want = min(-(-total // page), width)
        held = want if free is None else min(-(-c // page), want)
        for p in range(held, want):
            table[b][p] = pages[first + taken] if first + taken < len(pages) else -1
            taken += 1
        for t in range(c, min(total, c + max_tokens)):
            entry = table[b][t // page] if t // page < width else -1
            if len(slots) < max_tokens:
                slots.append(entry * page + t % page if entry >= 0 else -1)
        offsets.append(min(offsets[-1] + total - c, top))
        lens.append(total)
    slots += [-1] * (max_tokens - len(slots))
    return slots, offsets, lens, min(first + taken, top)


# ---- attention ---------------------------------------------------------------------
def paged_attention(q, kp, ks, vp, vs, table, lens, offsets, kv_heads, page, scale, causal=True, window=0,
                    k_gs=1.0, v_gs=1.0):
    """float64 (out, lse) and the bounds of their errors; rows of no request are NaN."""
    tokens, heads, dim = q.shape
    group, width, pages = heads // kv_heads, table.shape[1], kp.shape[0] // page
    out = torch.full((tokens, heads, dim), math.nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), math.nan, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    qd = q.double()
    for b in range(len(lens)):
        n0, n1 = int(offsets[b]), int(offsets[b + 1])
        length = min(max(int(lens[b]), 0), width * page)
        pos = torch.arange(length)
        entry = table[b].long()[pos // page] if length else pos
        inside = (entry >= 0) & (entry < pages)
        slot = torch.where(inside, entry, 0) * page + pos % page
        k = nvfp4_values(kp[slot], ks[slot]).view(length, kv_heads, dim) * k_gs
        v = nvfp4_values(vp[slot], vs[slot]).view(length, kv_heads, dim) * v_gs
        for t in range(n0, n1):
            p = length - (n1 - t)
            seen = inside.clone()
            if causal:
                seen &= pos <= p
            if window:
                seen &= pos > p - window
            at = seen.nonzero().flatten()
            n = at.numel()
            if n == 0:
                out[t], lse[t] = 0.0, -math.inf
                continue
            kk = k[at].repeat_interleave(group, 1)
            vv = v[at].repeat_interleave(group, 1)
            s = torch.einsum("hd,nhd->hn", qd[t], kk) * scale
            mag = torch.einsum("hd,nhd->hn", qd[t].abs(), kk.abs()) * abs(scale)
            lse[t] = torch.logsumexp(s, 1)
            w = torch.softmax(s, 1)
            out[t] = torch.einsum("hn,nhd->hd", w, vv)
            a = torch.einsum("hn,nhd->hd", w, vv.abs())
            # a score's error moves its exponential by that much relative
            d = (dim + 8) * 2.0 ** -24 * mag.amax(1) + 2.0 ** -21
            out_tol[t] = (2.0 ** -8 * out[t].abs() + a * (2.0 ** -11 + 2 * d[:, None] + (n + 8) * 2.0 ** -24)
                          + n * 2.0 ** -25 * vv.abs().amax(0))
            lse_tol[t] = d + (n + 8) * 2.0 ** -24 + 2.0 ** -22 * (1 + lse[t].abs())
    return out, lse, out_tol, lse_tol


# ---- mixture of experts ---------------------------------------------------------------
def route(logits, top_k, renormalize):
    """ids and float64 weights of plain lists of float logits."""
    ids, weights = [], []
    for row in logits.tolist():
        left = [(v, e) for e, v in enumerate(row) if v == v and v != -math.inf]
        order = [e for v, e in sorted(left, key=lambda p: (-p[0], p[1]))][:top_k]
        top = max((v for v, _ in left), default=0.0)
        part = {e: 1.0 if v == top else math.exp(v - top) for v, e in left}
        total = sum(part[e] for e in order) if renormalize else sum(part.values())
        pad = top_k - len(order)
        ids.append(order + [-1] * pad)
        weights.append([part[e] / total for e in order] + [0.0] * pad)
    return np.array(ids, np.int32), np.array(weights, np.float64)


def moe_layer(x, logits, w1, w2, top_k, renormalize, h_eps):
    """float64 out and its error bound; w1 [E, 2I, H], w2 [E, H, I] float64
    (global scales applied); h_eps: relative error of h as the second product
    reads it."""
    ids, weights = route(logits, top_k, renormalize)
    t, hidden = x.shape
    inter = w2.shape[2]
    j = torch.arange(inter)
    gate_rows, up_rows = 16 * (j // 8) + j % 8, 16 * (j // 8) + 8 + j % 8
    out, tol = torch.zeros(t, hidden, dtype=torch.float64), torch.zeros(t, hidden, dtype=torch.float64)
    xd = x.double()
    for a in range(t):
        for k in range(top_k):
            e, w = int(ids[a, k]), float(weights[a, k])
            if e < 0:
                continue
            acc, mag = w1[e] @ xd[a], w1[e].abs() @ xd[a].abs()
            err = (hidden + 8) * 2.0 ** -24 * mag
            g, u = acc[gate_rows], acc[up_rows]
            silu = g * torch.sigmoid(g)
            h = silu * u
            # |silu'| <= 1.1; sigmoid, product and gs roundings within 2^-19
            dh = 1.1 * err[gate_rows] * (u.abs() + err[up_rows]) + silu.abs() * err[up_rows] + h.abs() * (2.0 ** -19 + h_eps)
            dh = dh + h.abs().amax() * 2.0 ** -26      # values far below the largest lose bits in a scaled type
            y = w2[e] @ h
            m = w2[e].abs() @ h.abs()
            out[a] += w * y
            tol[a] += w * (w2[e].abs() @ dh + m * ((inter * top_k + 16) * 2.0 ** -24 + 2.0 ** -20))
    return out, tol + 2.0 ** -8 * out.abs(), ids, weights
