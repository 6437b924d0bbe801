"""The operators of sparse decoding over the paged NVFP4 cache, with cases to measure them on.

Four operators that run one after the other in a served model whose attention
reads a few pages of a long context:

* ``append``  the rotation of q and k by their positions (one axis, or several as
  images and video have) and the write of k and v into the cache
  (``nvfp4_rope_append``);
* ``keys``    one 8-bit key for each page that the new tokens complete
  (``nvfp4_page_keys``);
* ``select``  the pages that each new token attends to, by those keys
  (``nvfp4_select_pages``);
* ``sparse``  attention over the tokens of these pages (``nvfp4_sparse_attention``).

``run`` computes them in plain torch operations in FP32 where ``own`` is
false, and by the package's entry points where it is true. Formats are those
of ``include/moe_nvfp4.h``. Bytes of the cache, page keys and page lists are
defined bit by bit, so they are returned as they are and compared as whole numbers.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # one user, one token: latency
        dict(name="append_one", op="append", kind="decode", tokens=1, heads=32, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, page=16, longest=32768),
        # a full decoding batch; half of each head is rotated, by neighbouring pairs
        dict(name="append_batch", op="append", kind="decode", tokens=256, heads=64, kv_heads=8, dim=128, rot=64, axes=1,
             interleaved=True, page=16, longest=131072),
        # frames of a video between text: positions of three axes
        dict(name="append_video", op="append", kind="prompt", tokens=5003, heads=28, kv_heads=4, dim=128, rot=128, axes=3,
             interleaved=False, page=64, longest=32768),
        # a batch of long prompts, as they enter the cache
        dict(name="append_prompt", op="append", kind="prompt", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, axes=1,
             interleaved=False, page=64, longest=131072),
        # a decoding step of 256 requests: a few of them complete a page
        dict(name="keys_step", op="keys", seqs=256, longest=8192, new=1, kv_heads=8, dim=128, page=64),
        # ragged prompts: every page that they fill
        dict(name="keys_prompts", op="keys", seqs=6, longest=16384, new=16384, kv_heads=8, dim=128, page=64),
        # one user with a very long context
        dict(name="select_one", op="select", seqs=1, longest=131072, new=1, heads=32, kv_heads=8, dim=128, page=64, top=28,
             first=1, local=3),
        # a decoding batch with ragged contexts, smaller pages
        dict(name="select_batch", op="select", seqs=64, longest=32768, new=1, heads=64, kv_heads=8, dim=128, page=32, top=57,
             first=1, local=6),
        # a chunk of a long prompt: every token has pages of its own
        dict(name="select_chunk", op="select", seqs=1, longest=32000, new=2048, heads=32, kv_heads=8, dim=128, page=64, top=28,
             first=1, local=3),
        # one user with a very long context: the work of a row has to be split
        dict(name="sparse_one", op="sparse", seqs=1, longest=131072, new=1, heads=32, kv_heads=8, dim=128, page=64, top=28,
             first=1, local=3),
        # a full decoding batch with ragged contexts
        dict(name="sparse_batch", op="sparse", seqs=64, longest=32768, new=1, heads=64, kv_heads=8, dim=128, page=32, top=57,
             first=1, local=6),
        # a chunk of a long prompt
        dict(name="sparse_chunk", op="sparse", seqs=1, longest=17000, new=1000, heads=32, kv_heads=8, dim=128, page=64, top=28,
             first=1, local=3),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "keys", "select", "sparse"))
    if op == "append":
        dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
        kind = rng.choice(("decode", "prompt"))
        tokens = _log(rng, 1, 512) if kind == "decode" else _log(rng, 17, min(16384, (1 << 27) // ((heads + 2 * kv_heads) * dim)))
        return dict(op=op, kind=kind, tokens=tokens, heads=heads, kv_heads=kv_heads, dim=dim,
                    rot=rng.choice((dim, dim, dim // 2, 24, 2 * rng.randint(1, dim // 2))), axes=rng.choice((1, 1, 2, 3)),
                    interleaved=rng.choice((False, False, True)), page=rng.choice((1, 16, 24, 64)), longest=_log(rng, 20000, 131072))
    dim = rng.choice((64, 128, 256))
    kv_heads = rng.choice((1, 2, 4, 8))
    page = rng.choice((16, 24, 32, 64, 128))
    if op == "keys":
        longest = _log(rng, 100, 16384)
        new = rng.choice((1, 1, 5, _log(rng, 20, longest)))
        return dict(op=op, seqs=_log(rng, 1, 256 if new <= 5 else 6), longest=longest, new=new, kv_heads=kv_heads, dim=dim, page=page)
    heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8, 12))
    new = rng.choice((1, 1, 1, 4, _log(rng, 17, 1000)))
    longest = _log(rng, 1200, 32768)
    if op == "select":
        top = _log(rng, 4, 64)
        seqs = 1 if new > 4 else _log(rng, 1, 48 // new)
    else:
        # the tokens that a row attends to: at most the largest listed case's work
        top = _log(rng, 4, max(5, 2048 // page))
        new = min(new, max(1, (1 << 32) // (max(heads, kv_heads * 8) * dim * page * (top + 3))))
        seqs = 1 if new > 4 else _log(rng, 1, 48 // new)
    return dict(op=op, seqs=seqs, longest=longest, new=new, heads=heads, kv_heads=kv_heads, dim=dim, page=page, top=top,
                first=rng.choice((0, 1, 1, 2)), local=rng.choice((1, 2, 3)))


def _lengths(case):
    """The requests' cached and new lengths: ragged, the longest one present, the same for every seed."""
    r = random.Random(case["seqs"] * 1000003 + case["longest"])
    n, longest, new = case["seqs"], case["longest"], case["new"]
    total = [longest] + [_log(r, max(1, longest // 16), longest) for _ in range(n - 1)]
    if case["op"] == "keys" and new == 1:
        # about one request in a page's length completes one
        total = [t - t % case["page"] if i % case["page"] == 0 and t >= case["page"] else t for i, t in enumerate(total)]
    fresh = [min(new, t) for t in total]
    return [t - f for t, f in zip(total, fresh)], fresh


# ---- inputs ----------------------------------------------------------------------
def _nvfp4(x):
    """FP32 [..., n] -> codes [..., n/2] and scales [..., n/16], both uint8."""
    b = x.reshape(-1, 16)
    scale = (b.abs().amax(1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    m = (b.abs() / scale.float()).nan_to_num_(0.0, 6.0)
    code = (m > 0.25).to(torch.uint8)
    for border in (0.75, 1.25, 1.75, 2.5, 3.5, 5.0):
        code += m > border
    code += (b < 0).to(torch.uint8) * 8
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    lead = x.shape[:-1]
    return packed.reshape(*lead, x.shape[-1] // 2), scale.view(torch.uint8).reshape(*lead, x.shape[-1] // 16)


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _bytes(g, *shape, top=256):
    return torch.randint(0, top, shape, generator=g, device=DEVICE, dtype=torch.uint8)


def _prepare_append(case, g):
    n, heads, kv, dim, page, rot, axes = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "page", "rot", "axes"))
    longest = case["longest"]
    # a fused projection's rows: q, k and v side by side; some channels are larger
    qkv = torch.randn(n, heads + 2 * kv, dim, generator=g, device=DEVICE)
    qkv = (qkv * torch.exp(0.5 * torch.randn(dim, generator=g, device=DEVICE))).to(torch.bfloat16)
    pages = n // page + n // (4 * page) + 2
    slots = torch.randperm(pages, generator=g, device=DEVICE)[:, None] * page + torch.arange(page, device=DEVICE)
    slots = slots.reshape(-1)[:n].contiguous()
    if n >= 256:
        slots[n - n // 16:] = -1      # a padded batch
    t = torch.arange(n, device=DEVICE)
    if case["kind"] == "decode":
        base = torch.randint(0, longest, (n,), generator=g, device=DEVICE)
        positions = torch.stack([base] * axes)
    else:
        # axes of a picture or film: time, height, width; one axis: a text that ends at `longest`
        at = longest - n
        side = max(1, int(math.sqrt(n / 8)))
        positions = torch.stack([at + t] if axes == 1 else [at + t // (side * side), at + t // side % side, at + t % side][-axes:])
    angle = torch.arange(longest, device=DEVICE, dtype=torch.float64)[:, None] * torch.pow(
        1e6, -2.0 * torch.arange(rot // 2, device=DEVICE, dtype=torch.float64) / rot)
    s = dict(q=qkv[:, :heads], k=qkv[:, heads:heads + kv], v=qkv[:, heads + kv:], slots=slots, interleaved=case["interleaved"],
             positions=positions.to(torch.int32).contiguous(), cos_sin=torch.cat([angle.cos(), angle.sin()], 1).float(),
             pair_axis=None, k_gs=torch.rand(1, generator=g, device=DEVICE) * 0.01 + 0.002,
             v_gs=torch.rand(1, generator=g, device=DEVICE) * 0.01 + 0.002)
    if axes > 1:
        # a first run of pairs for the first axis, the others in turn behind it
        pair = torch.arange(rot // 2, device=DEVICE)
        s["pair_axis"] = torch.where(pair < rot // 8, 0, pair % axes).to(torch.int32)
    for name in ("k", "v"):
        s[name + "_packed"] = _bytes(g, pages * page, kv * dim // 2)
        s[name + "_scales"] = _bytes(g, pages * page, kv * dim // 16, top=127)
    return s


def _prepare_pages(case, g):
    """Lengths, offsets and a table of pages in random order."""
    cached, fresh = _lengths(case)
    page = case["page"]
    need = [-(-(c + f) // page) for c, f in zip(cached, fresh)]
    width, pages = max(need) + 1, sum(need) + 1
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    held = _ints(need)
    first = torch.cumsum(held, 0) - held
    col = torch.arange(width, device=DEVICE)
    table = torch.where(col[None, :] < held[:, None], order[(first[:, None] + col[None, :]).clamp_(max=pages - 1)], -1)
    total = [c + f for c, f in zip(cached, fresh)]
    return dict(table=table.to(torch.int32).contiguous(), lens=_ints(total), pages=pages, page=page, width=width,
                offsets=_ints([0] + torch.tensor(fresh).cumsum(0).tolist()), tokens=sum(fresh), max_query=max(fresh))


def _cache(g, rows, kv, dim):
    spread = torch.exp(0.5 * torch.randn(kv, dim, generator=g, device=DEVICE))
    shift = 0.5 * torch.randn(kv, dim, generator=g, device=DEVICE)
    x = torch.randn(rows, kv, dim, generator=g, device=DEVICE) * spread + shift
    return _nvfp4(x.reshape(rows, kv * dim))


def _prepare_keys(case, g):
    s = _prepare_pages(case, g)
    kv, dim = case["kv_heads"], case["dim"]
    s["k"], s["k_scales"] = _cache(g, s["pages"] * s["page"], kv, dim)
    s["keys"] = torch.randint(-127, 128, (s["pages"], kv, dim), generator=g, device=DEVICE, dtype=torch.int8)
    s["exponents"] = torch.randint(0, 20, (s["pages"], kv), generator=g, device=DEVICE, dtype=torch.int8)
    return s


def _prepare_select(case, g):
    s = _prepare_pages(case, g)
    kv, dim = case["kv_heads"], case["dim"]
    # page keys: what the heads' keys have in common, and each page's own part
    x = torch.randn(1, kv, dim, generator=g, device=DEVICE) + torch.randn(s["pages"], kv, dim, generator=g, device=DEVICE)
    x = x / x.abs().amax(2, keepdim=True)
    s["keys"] = (x * (64 + 63 * torch.rand(s["pages"], kv, 1, generator=g, device=DEVICE))).round().to(torch.int8)
    s["exponents"] = torch.randint(9, 12, (s["pages"], kv), generator=g, device=DEVICE, dtype=torch.int8)
    s["q"] = torch.randn(s["tokens"], case["heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    s.update(top=case["top"], first=case["first"], local=case["local"])
    return s


def _prepare_sparse(case, g):
    s = _prepare_pages(case, g)
    kv, dim, page, first, local = case["kv_heads"], case["dim"], case["page"], case["first"], case["local"]
    s["k"], s["k_scales"] = _cache(g, s["pages"] * page, kv, dim)
    s["v"], s["v_scales"] = _cache(g, s["pages"] * page, kv, dim)
    s["gs"] = torch.tensor([0.75, 1.25], device=DEVICE)
    s["q"] = torch.randn(s["tokens"], case["heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    # lists as a selection gives them: tokens that follow each other choose much the same pages
    b, position = _places(s)
    score = torch.randn(len(s["lens"]), kv, s["width"], generator=g, device=DEVICE)[b]
    score += 0.7 * torch.randn(score.shape, generator=g, device=DEVICE)
    s["list"] = _choose(score, position // page, case["top"], first, local)
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = {"append": _prepare_append, "keys": _prepare_keys, "select": _prepare_select, "sparse": _prepare_sparse}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


# ---- the plain forms ---------------------------------------------------------------
def _decode(packed, scales):
    """Codes [..., n/2] and scales [..., n/16] -> FP32 [..., n]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    pair = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).int()
    block = table[pair].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return block.flatten(-2)


def _places(s):
    """The request of every token and the token's position in it."""
    offsets, lens = s["offsets"].long(), s["lens"].long()
    t = torch.arange(s["tokens"], device=offsets.device)
    b = (t[:, None] >= offsets[None, 1:]).sum(1)
    return b, lens[b] - offsets[b + 1] + t


def _rotate(x, cos, sin, interleaved):
    """Pairs of x [tokens, heads, dim] turned by their angles [tokens, pairs]; dimensions behind them stay."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., 2 * half:]], -1)


def _quantize(x, gs):
    """FP32 [rows, n] -> NVFP4 bytes, each step rounded to FP32 (a quotient in 64 bits, then 32, is the rounded quotient)."""
    b = x.unflatten(-1, (-1, 16))
    scale = (b.abs().amax(-1).double() / (6 * gs).double()).float().clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (scale.float() * gs).unsqueeze(-1)
    v = torch.where(d == 0, 0.0, (b.abs().double() / d.double()).float())
    steps = (2 * v.clamp(max=6.0)).round().int()
    code = torch.tensor([0, 1, 2, 3, 4, 4, 5, 6, 6, 6, 6, 7, 7], dtype=torch.uint8, device=x.device)[steps]
    code = (code | torch.signbit(b).to(torch.uint8) << 3).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.view(torch.uint8)


def _plain_append(s):
    half = s["cos_sin"].shape[1] // 2
    pair = torch.arange(half, device=s["q"].device)
    at = s["positions"].long()
    at = at[0][:, None].expand(-1, half) if s["pair_axis"] is None else at[s["pair_axis"].long()].t()
    cos, sin = s["cos_sin"][at, pair], s["cos_sin"][at, half + pair]
    q = _rotate(s["q"].float(), cos, sin, s["interleaved"]).to(torch.bfloat16)
    here = s["slots"] >= 0
    to = s["slots"][here]
    k = _rotate(s["k"].float(), cos, sin, s["interleaved"]).flatten(1)[here]
    v = s["v"].float().flatten(1)[here]
    s["k_packed"][to], s["k_scales"][to] = _quantize(k, s["k_gs"])
    s["v_packed"][to], s["v_scales"][to] = _quantize(v, s["v_gs"])
    return q, s["k_packed"], s["k_scales"], s["v_packed"], s["v_scales"]


def _plain_keys(s):
    page, table = s["page"], s["table"].long()
    lens, offsets = s["lens"].long(), s["offsets"].long()
    before = lens - (offsets[1:] - offsets[:-1])
    col = torch.arange(s["width"], device=table.device)
    whole = table[(col >= (before // page)[:, None]) & (col < (lens // page)[:, None])]
    slots = whole[:, None] * page + torch.arange(page, device=table.device)
    k = _decode(s["k"][slots], s["k_scales"][slots]).view(*slots.shape, *s["keys"].shape[1:])
    total = (k * 1024).double().sum(1)
    bits = torch.frexp(total.abs().amax(-1)).exponent
    e = (bits - 7).clamp(min=0)
    s["keys"][whole] = (total * torch.pow(2.0, -e.double()).unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8)
    s["exponents"][whole] = e.to(torch.int8)
    return s["keys"], s["exponents"]


def _choose(score, current, top, first, local):
    """Lists of pages [tokens, kv heads, first + top + local]: the first pages, those up to `current`, and the best
    of the others by score [tokens, kv heads, pages], ties to the lower page; ascending, -1 behind them."""
    j = torch.arange(score.shape[-1], device=score.device)
    current = current[:, None, None]
    others = (j >= first) & (j <= current - local)
    order = torch.sort(score.masked_fill(~others, -math.inf), dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    taken = (others & (rank < top)) | ((j < first) & (j <= current)) | ((j > current - local) & (j <= current))
    n = first + top + local
    found = torch.sort(torch.where(taken, j, score.shape[-1]), dim=-1).values
    found = torch.nn.functional.pad(found, (0, max(0, n - found.shape[-1])), value=score.shape[-1])[..., :n]
    return torch.where(found < score.shape[-1], found, -1).to(torch.int32)


def _plain_select(s):
    q, kv, dim = s["q"].float(), s["keys"].shape[1], s["keys"].shape[2]
    b, position = _places(s)
    q = q.unflatten(1, (kv, -1))
    e = torch.frexp(q.abs().amax((2, 3))).exponent - 7
    q = (q.double() * torch.pow(2.0, -e.double())[..., None, None]).round().clamp(-127, 127).float()
    entry = s["table"].long().clamp(min=0)
    # sums of whole numbers below 2^24: exact in FP32, in any order
    keys = s["keys"][entry].float().permute(0, 2, 3, 1).contiguous()          # [seqs, kv, dim, pages]
    power = torch.pow(2.0, s["exponents"][entry].float()).permute(0, 2, 1)      # [seqs, kv, pages]
    if keys.shape[0] == 1:
        flat = q.permute(1, 0, 2, 3).flatten(1, 2)
        score = torch.matmul(flat, keys[0]).unflatten(1, (q.shape[0], -1)).amax(2).transpose(0, 1)
    else:
        score = torch.matmul(q, keys[b]).amax(2)
    return _choose(score * power[b], position // s["page"], s["top"], s["first"], s["local"])


def _plain_sparse(s):
    q, page, listed_pages = s["q"].float(), s["page"], s["list"].long()
    tokens, kv, n = listed_pages.shape
    dim = q.shape[2]
    b, position = _places(s)
    off = torch.arange(page, device=q.device)
    at = listed_pages[..., None] * page + off
    seen = ((listed_pages[..., None] >= 0) & (at <= position[:, None, None, None])).flatten(2)
    entry = s["table"].long()[b[:, None, None], listed_pages.clamp(min=0)]
    slots = (entry[..., None] * page + off).flatten(2)                          # [tokens, kv, listed tokens]
    head = torch.arange(kv, device=q.device)[:, None]
    cut = lambda c: c.unflatten(1, (kv, -1))[slots, head]                      # noqa: E731
    k = _decode(cut(s["k"]), cut(s["k_scales"])).transpose(2, 3).contiguous()
    score = torch.matmul(q.unflatten(1, (kv, -1)), k) * (s["gs"][0] / math.sqrt(dim))
    del k
    score = score.masked_fill_(~seen[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    norm = p.sum(-1, keepdim=True)
    out = torch.matmul(p, _decode(cut(s["v"]), cut(s["v_scales"]))) * (s["gs"][1] / norm)
    return out.flatten(1, 2).to(torch.bfloat16), (top + norm.log()).flatten(1)


def run(s):
    if not own:
        return {"append": _plain_append, "keys": _plain_keys, "select": _plain_select, "sparse": _plain_sparse}[s["op"]](s)
    import moe_swiglu_epilogue_amd as M
    if s["op"] == "append":
        q = M.nvfp4_rope_append(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_packed"], s["k_scales"],
                                s["v_packed"], s["v_scales"], pair_axis=s["pair_axis"], interleaved=s["interleaved"],
                                k_gs=s["k_gs"], v_gs=s["v_gs"])
        return q, s["k_packed"], s["k_scales"], s["v_packed"], s["v_scales"]
    if s["op"] == "keys":
        return M.nvfp4_page_keys(s["k"], s["k_scales"], s["table"], s["lens"], s["offsets"], s["keys"], s["exponents"],
                                 page_size=s["page"], max_query_len=s["max_query"])
    if s["op"] == "select":
        return M.nvfp4_select_pages(s["q"], s["keys"], s["exponents"], s["table"], s["lens"], s["offsets"], page_size=s["page"],
                                    top_k=s["top"], first=s["first"], local=s["local"])
    return M.nvfp4_sparse_attention(s["q"], s["k"], s["k_scales"], s["v"], s["v_scales"], s["table"], s["lens"], s["offsets"],
                                    s["list"], page_size=s["page"], k_gs=s["gs"][0:1], v_gs=s["gs"][1:2], lse=True)


# ---- what a pass cannot do without -----------------------------------------------
def work(case):
    kv, dim = case["kv_heads"], case["dim"]
    if case["op"] == "append":
        n, heads, rot = case["tokens"], case["heads"], case["rot"]
        table = min(n, case["longest"]) * rot * 4.0
        return {"bytes": n * (dim * (4.0 * heads + 4 * kv + 2 * kv * 9 / 16) + 4 * case["axes"] + 8) + table,
                "flops": 3.0 * n * rot * (heads + kv)}
    cached, fresh = _lengths(case)
    page = case["page"]
    if case["op"] == "keys":
        done = sum((c + f) // page - c // page for c, f in zip(cached, fresh))
        return {"bytes": done * kv * (page * dim * 9 / 16 + dim + 1) + 12.0 * len(fresh), "flops": 1.0 * done * page * kv * dim}
    heads, listed_pages = case["heads"], case["top"] + case["first"] + case["local"]
    if case["op"] == "select":
        pages = [(c + f) // page for c, f in zip(cached, fresh)]
        return {"bytes": sum(pages) * kv * (dim + 1.0) + sum(fresh) * (2.0 * heads * dim + 4.0 * kv * listed_pages),
                "flops": 2.0 * heads * dim * sum(p * f for p, f in zip(pages, fresh))}
    read = pairs = 0
    for c, f in zip(cached, fresh):
        # a chunk's tokens may share what they read: at most the request's cache, once
        read += min(c + f, f * listed_pages * page)
        pairs += f * min(c + f, listed_pages * page)
    n = sum(fresh)
    return {"bytes": read * kv * dim * 9 / 8 + n * (heads * (4.0 * dim + 4) + 4.0 * kv * listed_pages), "flops": 4.0 * pairs * heads * dim}


# ---- the definitions in 64 bits ----------------------------------------------------
def _exact_values(packed, scales):
    """NVFP4 in float64, from the fields of the two formats."""
    n = packed.shape[-1] * 2
    code = torch.empty(*packed.shape[:-1], n, dtype=torch.uint8, device=packed.device)
    code[..., 0::2] = packed % 16
    code[..., 1::2] = packed // 16
    expo, man = (code // 2) % 4, (code % 2).double()
    value = torch.where(expo == 0, man * 0.5, (1 + man / 2) * torch.pow(2.0, expo.double() - 1))
    value = torch.where(code >= 8, -value, value)
    expo, man = ((scales // 8) % 16).double(), (scales % 8).double()
    scale = torch.where(expo == 0, man / 512, (1 + man / 8) * torch.pow(2.0, expo - 7))
    return value * scale.repeat_interleave(16, dim=-1)


def _exact_append(case, s):
    x = s["q"].double()
    rot, half = case["rot"], case["rot"] // 2
    out = x.clone()
    for j in range(half):
        axis = 0 if s["pair_axis"] is None else int(s["pair_axis"][j])
        row = s["cos_sin"][s["positions"][axis].long()].double()
        c, z = row[:, j, None], row[:, half + j, None]
        a, b = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + half)
        out[..., a] = x[..., a] * c - x[..., b] * z
        out[..., b] = x[..., a] * z + x[..., b] * c
    return out, None, None, None, None      # the bytes' definition rounds to FP32 step by step


def _exact_keys(case, s):
    page, kv, dim = case["page"], case["kv_heads"], case["dim"]
    keys, exponents, table = s["keys"].clone(), s["exponents"].clone(), s["table"].tolist()
    for b, (c, f) in enumerate(zip(*_lengths(case))):
        for j in range(c // page, (c + f) // page):
            rows = slice(table[b][j] * page, table[b][j] * page + page)
            total = (_exact_values(s["k"][rows], s["k_scales"][rows]) * 1024).long().sum(0).view(kv, dim)
            e = torch.log2(total.abs().amax(1).double().clamp(min=0.5)).floor().long().sub(6).clamp(min=0)
            keys[table[b][j]] = torch.round(total / torch.pow(2.0, e.double())[:, None]).clamp(-127, 127).to(torch.int8)
            exponents[table[b][j]] = e.to(torch.int8)
    return keys, exponents


def _exact_select(case, s):
    top, first, local, page, kv = case["top"], case["first"], case["local"], case["page"], case["kv_heads"]
    out = torch.full((s["tokens"], kv, top + first + local), -1, dtype=torch.int32)
    q, row = s["q"].double().unflatten(1, (kv, -1)), 0
    whole = torch.floor(torch.log2(q.abs().amax((2, 3)))) - 6
    q = torch.round(q / torch.pow(2.0, whole)[..., None, None]).clamp(-127, 127)
    for b, (c, f) in enumerate(zip(*_lengths(case))):
        entry = s["table"][b, : -(-(c + f) // page)].long()
        keys = s["keys"][entry].double() * torch.pow(2.0, s["exponents"][entry].double()).unsqueeze(-1)
        for i in range(f):
            now = (c + i) // page
            best = (keys[:, :, None] * q[row + i]).sum(-1).amax(-1)
            for h in range(kv):
                span = torch.arange(first, max(first, now - local + 1), device=q.device)
                order = torch.argsort(best[span, h], descending=True, stable=True)[:top]
                pages = set(range(min(first, now + 1))) | set(range(max(0, now - local + 1), now + 1)) | set(span[order].tolist())
                out[row + i, h, : len(pages)] = torch.tensor(sorted(pages), dtype=torch.int32)
        row += f
    return out


def _exact_sparse(case, s):
    q, dim, kv, page = s["q"].double(), case["dim"], case["kv_heads"], case["page"]
    gs = s["gs"].double().tolist()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    q = q.unflatten(1, (kv, -1)) * (gs[0] / math.sqrt(dim))
    row = 0
    for b, (c, f) in enumerate(zip(*_lengths(case))):
        pos = torch.arange(c + f, device=q.device)
        slot = s["table"][b].long()[pos // page] * page + pos % page
        k = _exact_values(s["k"][slot], s["k_scales"][slot]).view(-1, kv, dim).permute(1, 0, 2).contiguous()
        v = _exact_values(s["v"][slot], s["v_scales"][slot]).view(-1, kv, dim).permute(1, 0, 2).contiguous() * gs[1]
        for i in range(f):
            hit = (pos[None, None, :] // page == s["list"][row + i].long()[..., None]).any(1) & (pos <= c + i)    # [kv, tokens]
            z = (q[row + i] @ k.transpose(1, 2)).masked_fill(~hit[:, None], -math.inf)
            lse[row + i] = torch.logsumexp(z, 2).reshape(-1)
            out[row + i] = (torch.softmax(z, 2) @ v).reshape(-1, dim)
        row += f
    return out, lse


def exact(case, seed):
    if case["op"] == "select" and case["new"] * case["seqs"] * case["kv_heads"] > 4096:
        return None      # a list for each token and head, one by one: too long
    s = prepare(case, seed)
    return {"append": _exact_append, "keys": _exact_keys, "select": _exact_select, "sparse": _exact_sparse}[case["op"]](case, s)
