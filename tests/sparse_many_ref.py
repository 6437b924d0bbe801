"""The selection and the page keys of tests/sparse_ref.py for many tokens at once
(float64 products of whole numbers, which are exact), and the rules by which the
library cuts the work, so that a test can say which path it takes. CPU only; shares
no code with the product."""
import numpy as np
import torch

from serving_ref import nvfp4_values


def select_pages(q, keys, exponents, table, lens, offsets, page, top_k, first, local, untouched=-7):
    tokens, heads, dim = q.shape
    count, kv, _ = keys.shape
    n_list = first + top_k + local
    out = torch.full((tokens, kv, n_list), untouched, dtype=torch.int32)
    for b in range(len(lens)):
        lo, hi = max(int(offsets[b]), 0), min(int(offsets[b + 1]), tokens)
        if lo >= hi:
            continue
        length = min(max(int(lens[b]), 0), table.shape[1] * page)
        pos = length - int(offsets[b + 1]) + torch.arange(lo, hi)
        own = torch.div(pos, page, rounding_mode="floor")[:, None, None]
        pages = max(int(own.max()) + 1, 0)
        entry = table[b, :pages].long()
        here = (entry >= 0) & (entry < count)
        k = keys[entry.where(here, 0)].double() * torch.pow(2.0, exponents[entry.where(here, 0)].double())[..., None] if count \
            else torch.zeros(pages, kv, dim, dtype=torch.float64)
        x = q[lo:hi].double().unflatten(1, (kv, -1))
        top = x.abs().amax((2, 3))
        e = torch.where(top > 0, torch.frexp(top).exponent - 7, 0)
        x = torch.ldexp(x, -e[..., None, None]).round().clamp(-127, 127)
        score = torch.matmul(x.permute(1, 0, 2, 3).flatten(1, 2), k.permute(1, 2, 0).contiguous())     # [kv, n group, pages]
        score = score.unflatten(1, (hi - lo, -1)).amax(2).transpose(0, 1)
        j = torch.arange(pages)
        others = (j >= first) & (j <= own - local) & here
        order = torch.argsort(score.masked_fill(~others, -np.inf), dim=-1, descending=True, stable=True)
        rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
        taken = (others & (rank < top_k)) | (((j < first) | (j > own - local)) & (j <= own))
        found = torch.where(taken, j, pages).sort(-1).values[..., :n_list]
        out[lo:hi] = -1
        out[lo:hi, :, :found.shape[-1]] = torch.where(found < pages, found, -1).int()
    return out


def page_sums(kp, ks, entries, kv, dim, page):
    """Sums of pages of the cache in units of 2^-10, int64 [pages, kv, dim]."""
    rows = (entries[:, None] * page + torch.arange(page)).flatten()
    return (nvfp4_values(kp[rows], ks[rows]) * 1024).long().unflatten(0, (-1, page)).sum(1).unflatten(1, (kv, dim))


def key_exponents(sums):
    bits = torch.frexp(sums.abs().amax(-1).double()).exponent      # 0 for 0
    return (bits - 7).clamp(min=0)


# ---- how the library cuts the work ----------------------------------------------
def append_plan(tokens, heads, kv, dim, rot, interleaved):
    """nvfp4_rope_append: (pair layout, workgroups of a token, tokens of a workgroup)."""
    layout = ("neighbours" if interleaved else "whole" if rot == dim and rot % 32 == 0 else "halves of 8" if rot % 16 == 0
              else "halves")
    at_once, units = 256 // (dim // (16 if layout == "whole" else 8)), heads + 2 * kv
    rounds = lambda n: -(-n * units // at_once)  # noqa: E731
    if tokens * rounds(1) <= 4096:
        return layout, rounds(1), 1
    together = 1
    while together < 4 and tokens // together >= 2048 and 10 * together * units < 9 * rounds(together) * at_once:
        together *= 2
    return layout, 1, together


def select_plan(tokens, heads, kv, seqs, width):
    """nvfp4_select_pages: (tokens of a workgroup, workgroups over a token's pages or 0,
    bytes of workspace)."""
    group, pitch, together = heads // kv, (width + 3) & ~3, 1
    while (together < 16 and together < tokens // max(seqs, 1) and (together + 1) * group <= 64
           and (together + 1) * pitch * 4 <= 16384):
        together += 1
    items, size = -(-tokens // together) * kv, tokens * kv * pitch * 4
    if items > 768 or size > 2 ** 28:
        return together, 0, 0
    return together, max(1, min(1024 // items, -(-pitch // 256))), size
