"""Plain definitions of the sparse-attention operators (include/nvfp4_sparse.h) in
Python integers, float64 and explicit roundings, with the error bounds that the
attention's GPU results must keep (counted as in tests/serving_ref.py). CPU
only; shares no code with the product.
"""
import math

import numpy as np
import torch

import oracle
from serving_ref import nvfp4_values


def f32(x):
    """float64 rounded to binary32. A product of two binary32 numbers is exact in
    float64; a sum of two is rounded twice, which for 53 >= 2 * 24 + 2 bits gives the
    rounded sum."""
    return x.float().double()


# ---- rotation and append ---------------------------------------------------------
def rotate(x, positions, cos_sin, pair_axis=None, interleaved=False):
    """BF16 [tokens, heads, dim], int [axes, tokens], FP32 [most, rot] -> the binary32
    values of the turned heads, as float64."""
    most, rot = cos_sin.shape
    half, axes, tokens = rot // 2, positions.shape[0], x.shape[0]
    out = x.double().clone()
    for j in range(half):
        axis = 0 if pair_axis is None else int(pair_axis[j])
        if not 0 <= axis < axes:
            continue
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        p = positions[axis].long()
        ok = (p >= 0) & (p < most)
        row = cos_sin.double()[torch.where(ok, p, 0)] if most else torch.zeros(tokens, rot, dtype=torch.float64)
        c, s = row[:, j, None], row[:, half + j, None]
        xa, xb = x[..., a].double(), x[..., b].double()
        ok = ok[:, None]
        out[..., a] = torch.where(ok, f32(f32(xa * c) - f32(xb * s)), xa)
        out[..., b] = torch.where(ok, f32(f32(xb * c) + f32(xa * s)), xb)
    return out


def rope_append(q, k, v, positions, cos_sin, slots, caches, pair_axis=None, interleaved=False, k_gs=None, v_gs=None):
    """Returns the rotated q (BF16) and the four caches (NumPy uint8) behind the call."""
    kp, ks, vp, vs = [c.copy() for c in caches]
    tokens = k.shape[0]
    for x, gs, p, s in ((rotate(k, positions, cos_sin, pair_axis, interleaved), k_gs, kp, ks), (v.double(), v_gs, vp, vs)):
        rows = np.ascontiguousarray(x.flatten(1).float().numpy())
        packed, scales = oracle.quantize_f32(rows, None if gs is None else np.full(tokens, gs, np.float32))
        for t in range(tokens):
            if 0 <= int(slots[t]) < p.shape[0]:
                p[int(slots[t])], s[int(slots[t])] = packed[t], scales[t]
    out = None if q is None else rotate(q, positions, cos_sin, pair_axis, interleaved).to(torch.bfloat16)
    return out, (kp, ks, vp, vs)


# ---- page keys -------------------------------------------------------------------
def page_keys(kp, ks, table, lens, offsets, keys, exponents, page):
    """keys, exponents, and keys with the other neighbour where a sum lies half way
    between two numbers. (The factor 2^-e may be an ulp, 2^-53, low: S 2^-e below
    2^7 is then off by less than 2^-45, while a sum that is not half way is at least
    2^-e away from it, and e is at most 23 for pages of up to 256 tokens (256 6 448 2^10 < 2^30).)"""
    keys, exponents = keys.clone(), exponents.clone()
    pages, kv, dim = keys.shape
    other = keys.clone()
    for b in range(len(lens)):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        n = max(int(offsets[b + 1]) - int(offsets[b]), 0)
        for j in range(max(length - n, 0) // page, length // page):
            entry = int(table[b, j])
            if not 0 <= entry < pages:
                continue
            rows = slice(entry * page, (entry + 1) * page)
            total = (nvfp4_values(kp[rows], ks[rows]) * 1024).long().sum(0).view(kv, dim)
            for h in range(kv):
                e = max(0, int(total[h].abs().max()).bit_length() - 7)
                exponents[entry, h] = e
                for d in range(dim):
                    s = abs(int(total[h, d]))
                    low, rest, half = s >> e, s & ((1 << e) - 1), 1 << e >> 1
                    tie = e > 0 and rest == half
                    up = e > 0 and (rest > half or (tie and low & 1))
                    sign = -1 if int(total[h, d]) < 0 else 1
                    keys[entry, h, d] = sign * min(127, low + up)
                    other[entry, h, d] = sign * min(127, low + (not up if tie else up))
    return keys, exponents, other


# ---- selection -------------------------------------------------------------------
def requests(tokens, table, lens, offsets, page):
    """(token, request, position) of the tokens of all requests."""
    for b in range(len(lens)):
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        for t in range(max(int(offsets[b]), 0), min(int(offsets[b + 1]), tokens)):
            yield t, b, length - (int(offsets[b + 1]) - t)


def q8(rows):
    """BF16 [group, dim] -> whole numbers with the rows' common exponent."""
    top = float(rows.abs().max())
    e = math.frexp(top)[1] - 7 if top else 0
    return [[int(math.copysign(min(127, abs(round(math.ldexp(x, -e)))), x)) for x in r] for r in rows.tolist()]


def select_pages(q, keys, exponents, table, lens, offsets, page, top_k, first, local, untouched=-7):
    tokens, heads, dim = q.shape
    count, kv, _ = keys.shape
    group = heads // kv
    out = torch.full((tokens, kv, first + top_k + local), untouched, dtype=torch.int32)
    for t, b, p in requests(tokens, table, lens, offsets, page):
        out[t] = -1
        if p < 0:
            continue
        own = p // page
        for h in range(kv):
            rows = torch.tensor(q8(q[t, h * group:(h + 1) * group]))
            listed = {j for j in range(own + 1) if j < first or j > own - local}
            scores = []
            for j in range(own + 1):
                entry = int(table[b, j])
                if j not in listed and 0 <= entry < count:
                    best = int((rows * keys[entry, h].long()).sum(1).max())
                    scores.append((-best * 2 ** int(exponents[entry, h]), j))
            listed |= {j for _, j in sorted(scores)[:top_k]}
            out[t, h, :len(listed)] = torch.tensor(sorted(listed), dtype=torch.int32)
    return out


# ---- attention -------------------------------------------------------------------
def sparse_attention(q, kp, ks, vp, vs, table, lens, offsets, pages, page, scale, k_gs=1.0, v_gs=1.0):
    """float64 (out, lse) and the bounds of their errors; rows of no request are NaN."""
    tokens, heads, dim = q.shape
    kv, count = pages.shape[1], kp.shape[0] // page
    group = heads // kv
    out = torch.full((tokens, heads, dim), math.nan, dtype=torch.float64)
    lse = torch.full((tokens, heads), math.nan, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    k = nvfp4_values(kp, ks).view(-1, kv, dim) * k_gs
    v = nvfp4_values(vp, vs).view(-1, kv, dim) * v_gs
    for t, b, p in requests(tokens, table, lens, offsets, page):
        for h in range(kv):
            slots = []
            for j in pages[t, h].tolist():
                entry = int(table[b, j]) if 0 <= j < table.shape[1] else -1
                if 0 <= entry < count:
                    slots += [entry * page + i for i in range(page) if j * page + i <= p]
            at, n, rows = torch.tensor(slots, dtype=torch.long), len(slots), slice(h * group, (h + 1) * group)
            if n == 0:
                out[t, rows], lse[t, rows] = 0.0, -math.inf
                continue
            kk, vv, qq = k[at, h], v[at, h], q[t, rows].double()
            s, mag = qq @ kk.T * scale, qq.abs() @ kk.abs().T * abs(scale)
            lse[t, rows] = torch.logsumexp(s, 1)
            w = torch.softmax(s, 1)
            out[t, rows] = w @ vv
            # a score's error moves its exponential by that much relative
            d = (dim + 8) * 2.0 ** -24 * mag.amax(1) + 2.0 ** -21
            out_tol[t, rows] = (2.0 ** -8 * out[t, rows].abs() + (w @ vv.abs()) * (2.0 ** -11 + 2 * d[:, None] + (n + 8) * 2.0 ** -24)
                                + n * 2.0 ** -25 * vv.abs().amax(0))
            lse_tol[t, rows] = d + (n + 8) * 2.0 ** -24 + 2.0 ** -22 * (1 + lse[t, rows].abs())
    return out, lse, out_tol, lse_tol
