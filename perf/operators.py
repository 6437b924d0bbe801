"""The operators of one decoding step over NVFP4 data, with cases to measure them on.

Three operators that run one after the other in a served model:

* ``tables``  page allocation and slot maps of a paged cache from the requests'
  lengths (``kv_block_tables``);
* ``attn``    attention over the paged NVFP4 key/value cache, from single
  tokens to whole prompts (``nvfp4_paged_attention``);
* ``moe``     a whole mixture-of-experts layer for a few tokens, from the
  router's logits to the summed output (``moe_layer_nvfp4`` with weights in
  NVFP4, ``moe_layer_bf16`` with BF16 weights).

``run`` computes them in plain torch operations in FP32 where ``own`` is
false, and by the package's entry points where it is true. Formats are those
of ``include/moe_nvfp4.h``: a row of NVFP4 values is cols/2 bytes of E2M1 codes
(the even element in the low nibble) and cols/16 E4M3 scale bytes.
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
        # one new token for each of 256 running requests: the launch's latency
        dict(name="tables_step", op="tables", kind="step", seqs=256, longest=8192, new=1, page=16),
        # a batch of ragged prompts entering the cache
        dict(name="tables_prompts", op="tables", kind="prompts", seqs=48, longest=16384, new=8192, page=64),
        # one user, one token: latency
        dict(name="attn_one", op="attn", kind="decode", seqs=1, longest=2048, new=1, heads=32, kv_heads=8,
             dim=128, page=16, window=0),
        # a full decoding batch with ragged contexts
        dict(name="attn_batch", op="attn", kind="decode", seqs=64, longest=8192, new=1, heads=64, kv_heads=8,
             dim=128, page=16, window=0),
        # two users with very long contexts: the work of a row has to be split
        dict(name="attn_long", op="attn", kind="decode", seqs=2, longest=131072, new=1, heads=32, kv_heads=4,
             dim=128, page=64, window=0),
        # five drafted tokens a request to verify, small heads, a sliding window
        dict(name="attn_verify", op="attn", kind="decode", seqs=24, longest=5000, new=5, heads=64, kv_heads=8,
             dim=64, page=32, window=1500),
        # whole prompts: causal attention, bound by the matrix cores
        dict(name="attn_prompt", op="attn", kind="prompt", seqs=3, longest=4096, new=4096, heads=32, kv_heads=8,
             dim=128, page=16, window=0),
        # a chunk of a long prompt behind a cached context, wide heads
        dict(name="attn_chunk", op="attn", kind="prompt", seqs=2, longest=17000, new=1000, heads=16, kv_heads=4,
             dim=256, page=64, window=0),
        # one token through a large layer with weights in 4 bits
        dict(name="moe_one", op="moe", weights="nvfp4", tokens=1, hidden=7168, inter=2048, experts=64, top_k=8,
             renormalize=True),
        # a decoding batch that reaches nearly every expert
        dict(name="moe_batch", op="moe", weights="nvfp4", tokens=32, hidden=7168, inter=2048, experts=64, top_k=8,
             renormalize=True),
        # a small layer in BF16, where launches and latency count
        dict(name="moe_bf16_few", op="moe", weights="bf16", tokens=3, hidden=1024, inter=512, experts=8, top_k=2,
             renormalize=False),
        # a decoding batch in BF16, odd sizes
        dict(name="moe_bf16_batch", op="moe", weights="bf16", tokens=57, hidden=4096, inter=1408, experts=16, top_k=4,
             renormalize=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tables", "attn", "attn", "moe"))
    if op == "tables":
        kind = rng.choice(("step", "prompts", "read"))
        longest = _log(rng, 40, 16384)
        return dict(op=op, kind=kind, seqs=_log(rng, 1, 1024 if kind == "step" else 48), longest=longest,
                    new=1 if kind == "step" else _log(rng, 20, max(20, min(longest, 8192))), page=rng.choice((1, 8, 16, 24, 64, 128)))
    if op == "attn":
        kind = rng.choice(("decode", "decode", "prompt"))
        dim = rng.choice((64, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8, 12))
        page = rng.choice((1, 16, 24, 32, 64))
        window = rng.choice((0, 0, 0, 100, 1023))
        if kind == "decode":
            longest = _log(rng, 30, 65536)
            new = min(longest, rng.choice((1, 1, 1, 2, 4, 7)))
            seqs = _log(rng, 1, max(1, min(64, (256 << 20) // (longest * kv_heads * dim))))
        else:
            longest = _log(rng, 33, 8192)
            most = (1 << 36) // (longest * heads * dim)     # the largest listed prompts' products
            new = _log(rng, 17, max(17, min(longest, most)))
            seqs = _log(rng, 1, max(1, min(4, most // new)))
        return dict(op=op, kind=kind, seqs=seqs, longest=longest, new=new, heads=heads, kv_heads=kv_heads, dim=dim,
                    page=page, window=window)
    weights = rng.choice(("nvfp4", "bf16"))
    experts = rng.choice((1, 4, 8, 24, 64 if weights == "nvfp4" else 16))
    return dict(op=op, weights=weights, tokens=_log(rng, 1, 64), hidden=32 * _log(rng, 4, 128),
                inter=32 * _log(rng, 2, 64), experts=experts, top_k=min(experts, rng.choice((1, 2, 4, 6, 8))),
                renormalize=rng.choice((True, False)))


def _lengths(case):
    """The requests' cached and new lengths: ragged, the longest one present, the same for every seed."""
    r = random.Random(case["seqs"] * 1000003 + case["longest"])
    n, longest, new = case["seqs"], case["longest"], case["new"]
    total = [longest] + [_log(r, max(1, longest // 16), longest) for _ in range(n - 1)]
    if case["kind"] in ("step", "decode"):
        fresh = [min(new, t) for t in total]
    else:
        fresh = [min(new, longest)] + [_log(r, max(1, new // 8), min(new, t)) if min(new, t) > max(1, new // 8)
                                       else min(new, t) for t in total[1:]]
    if case["kind"] == "read":
        fresh = list(total)
    return [t - f for t, f in zip(total, fresh)], fresh


# ---- inputs ----------------------------------------------------------------------
def _nvfp4(x):
    """FP32 [..., n] -> codes [..., n/2] and scales [..., n/16], both uint8."""
    b = x.reshape(-1, 16)
    scale = (b.abs().amax(1, keepdim=True) / 6).to(torch.float8_e4m3fn)
    m = (b.abs() / scale.float()).nan_to_num_(0.0, 6.0)
    code = (m > 0.25).to(torch.uint8)
    code += m > 0.75
    code += m > 1.25
    code += m > 1.75
    code += m > 2.5
    code += m > 3.5
    code += m > 5.0
    code += (b < 0).to(torch.uint8) * 8
    packed = code[:, 0::2] | (code[:, 1::2] << 4)
    lead = x.shape[:-1]
    return packed.reshape(*lead, x.shape[-1] // 2), scale.view(torch.uint8).reshape(*lead, x.shape[-1] // 16)


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _prepare_pages(case, g):
    """Lengths on the device, a table with the cached pages of each request and
    a list of free pages: all pages of the cache in random order."""
    cached, fresh = _lengths(case)
    page = case["page"]
    width = max(-(-(c + f) // page) for c, f in zip(cached, fresh)) + 1
    held = [-(-(c + f if case["kind"] == "read" else c) // page) for c, f in zip(cached, fresh)]
    need = sum(-(-(c + f) // page) for c, f in zip(cached, fresh))
    pages = need + need // 8 + 1
    order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    h = _ints(held)
    first = torch.cumsum(h, 0) - h
    col = torch.arange(width, device=DEVICE, dtype=torch.int64)
    table = torch.where(col[None, :] < h[:, None], order[(first[:, None] + col[None, :]).clamp_(max=pages - 1)], -1)
    return dict(cached=_ints(cached), fresh=_ints(fresh), table=table.to(torch.int32).contiguous(),
                free=order[sum(held):].contiguous(), page=page, pages=pages, total=sum(fresh), width=width)


def _prepare_tables(case, g):
    s = _prepare_pages(case, g)
    # a padded batch: some more rows than tokens, as a captured graph has them
    s["max_tokens"] = s["total"] + s["total"] // 10 + 3
    s["kind"] = case["kind"]
    return s


def _prepare_attn(case, g):
    s = _prepare_pages(case, g)
    page, pages, kv, dim = s["page"], s["pages"], case["kv_heads"], case["dim"]
    used = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    total = s["cached"] + s["fresh"]
    held = (total + page - 1) // page
    first = torch.cumsum(held, 0) - held
    col = torch.arange(s["width"], device=DEVICE, dtype=torch.int64)
    s["table"] = torch.where(col[None, :] < held[:, None], used[(first[:, None] + col[None, :]).clamp_(max=pages - 1)], -1
                             ).to(torch.int32).contiguous()
    spread = torch.exp(0.5 * torch.randn(2, kv, 1, generator=g, device=DEVICE))
    for name, f in (("k", spread[0]), ("v", spread[1])):
        x = torch.randn(pages * page, kv, dim, generator=g, device=DEVICE) * f
        s[name], s[name + "_scales"] = _nvfp4(x.reshape(pages * page, kv * dim))
        del x
    s["gs"] = torch.tensor([0.75, 1.25], device=DEVICE)
    s["q"] = torch.randn(s["total"], case["heads"], dim, generator=g, device=DEVICE).to(torch.bfloat16)
    cached, fresh = _lengths(case)
    s["offsets"] = torch.cat([s["fresh"].new_zeros(1), torch.cumsum(s["fresh"], 0).to(torch.int32)])
    s["lens"] = total.to(torch.int32)
    s.update(max_query=max(fresh), max_seq=max(c + f for c, f in zip(cached, fresh)), window=case["window"],
             kv_heads=kv, heads=case["heads"], dim=dim)
    return s


def _prepare_moe(case, g):
    e, h, i, t = case["experts"], case["hidden"], case["inter"], case["tokens"]
    s = dict(weights=case["weights"], top_k=case["top_k"], renormalize=case["renormalize"], inter=i)
    # hidden states after a norm: a few large channels
    x = torch.randn(t, h, generator=g, device=DEVICE) * torch.exp(0.5 * torch.randn(h, generator=g, device=DEVICE))
    s["x"] = x.to(torch.bfloat16)
    s["logits"] = 1.5 * torch.randn(t, e, generator=g, device=DEVICE) + 0.5 * torch.randn(e, generator=g, device=DEVICE)
    for name, rows, cols in (("w1", 2 * i, h), ("w2", h, i)):
        w = torch.randn(e, rows, cols, generator=g, device=DEVICE)
        if case["weights"] == "bf16":
            s[name] = (w / math.sqrt(cols)).to(torch.bfloat16)
        else:
            # two-level scaling: w / gs has block scales in the middle of E4M3's range
            s[name], s[name + "_scales"] = _nvfp4(w * 64)
            s["g" + name] = (0.8 + 0.4 * torch.rand(e, generator=g, device=DEVICE)) / (64 * math.sqrt(cols))
        del w
    return s


def prepare(case, seed):
    g = _generator(seed)
    s = {"tables": _prepare_tables, "attn": _prepare_attn, "moe": _prepare_moe}[case["op"]](case, g)
    s["op"] = case["op"]
    return s


# ---- the plain forms ---------------------------------------------------------------
def _decode(packed, scales):
    """Codes [..., n/2] and scales [..., n/16] -> FP32 [..., n]."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=packed.device)
    pair = torch.stack([packed & 15, packed >> 4], dim=-1).flatten(-2).int()
    block = table[pair].unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float().unsqueeze(-1)
    return block.flatten(-2)


def _plain_tables(s):
    page, table, free = s["page"], s["table"], s["free"]
    cached, fresh = s["cached"].long(), s["fresh"].long()
    total = cached + fresh
    ends = torch.cumsum(fresh, 0)
    offsets = torch.cat([ends.new_zeros(1), ends])
    held, want = (cached + page - 1) // page, (total + page - 1) // page
    taken = torch.zeros_like(want) if s["kind"] == "read" else want - held
    base = torch.cumsum(taken, 0) - taken
    col = torch.arange(table.shape[1], device=table.device)
    fresh_page = (col >= held[:, None]) & (col < (held + taken)[:, None])
    at = (base[:, None] + col - held[:, None]).clamp(0, free.numel() - 1)
    table = torch.where(fresh_page, free[at], table)
    i = torch.arange(s["max_tokens"], device=table.device)
    b = (i[:, None] >= ends[None, :]).sum(1)
    real = b < ends.numel()
    b = b.clamp(max=ends.numel() - 1)
    pos = cached[b] + i - offsets[b]
    slots = torch.where(real, table[b, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page, -1)
    return slots, offsets.int(), total.int(), taken.sum().int().reshape(1), table


def _plain_attn(s):
    q, dim, kv, page = s["q"], s["dim"], s["kv_heads"], s["page"]
    offsets, lens = s["offsets"].long(), s["lens"].long()
    group, seqs = s["heads"] // kv, lens.numel()
    pos = torch.arange(s["max_seq"], device=q.device)
    slots = s["table"][:, pos // page].long().clamp(min=0) * page + pos % page
    k = _decode(s["k"][slots], s["k_scales"][slots]).view(seqs, -1, kv, dim).permute(0, 2, 3, 1).contiguous()
    i = torch.arange(s["max_query"], device=q.device)
    at = (offsets[:-1, None] + i).clamp(max=q.shape[0] - 1)
    rows = q[at].float().view(seqs, -1, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(seqs, kv, -1, dim)
    score = torch.matmul(rows, k) * (s["gs"][0] / math.sqrt(dim))
    del k
    here = lens[:, None] - (offsets[1:] - offsets[:-1])[:, None] + i
    seen = (pos <= here[..., None]) & (pos < lens[:, None, None])
    if s["window"]:
        seen &= pos > here[..., None] - s["window"]
    score = score.view(seqs, kv, group, -1, pos.numel()).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = score.sub_(top).exp_()
    norm = p.sum(-1, keepdim=True)
    lse = (top + norm.log()).squeeze(-1)
    v = _decode(s["v"][slots], s["v_scales"][slots]).view(seqs, -1, kv, dim).permute(0, 2, 1, 3).contiguous()
    out = torch.matmul(p.view(seqs, kv, -1, pos.numel()), v).view(seqs, kv, group, -1, dim)
    out = out * s["gs"][1] / norm
    t = torch.arange(q.shape[0], device=q.device)
    b = (t[:, None] >= offsets[None, 1:]).sum(1)
    j = t - offsets[b]
    return out.permute(0, 3, 1, 2, 4)[b, j].reshape(q.shape).to(torch.bfloat16), lse.permute(0, 3, 1, 2)[b, j].reshape(q.shape[:2])


def _route(s):
    """Rank of every expert for each token (ties to the lower index), the
    top_k experts in order and their weights."""
    logits, k = s["logits"], s["top_k"]
    e = torch.arange(logits.shape[1], device=logits.device)
    above = (logits[:, None, :] > logits[:, :, None]) | ((logits[:, None, :] == logits[:, :, None]) & (e[None, :] < e[:, None]))
    rank = above.sum(2)
    ids = ((rank[:, None, :] == torch.arange(k, device=e.device)[:, None]) * e).sum(2)
    p = (logits - logits.amax(1, keepdim=True)).exp()
    p = p / p.sum(1, keepdim=True)
    w = p[torch.arange(p.shape[0], device=e.device)[:, None], ids]
    if s["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    return ids, w, rank < k


def _plain_weights(s, name, ids):
    """FP32 weights of the experts `ids` (None: of all)."""
    pick = (lambda v: v) if ids is None else (lambda v: v[ids])
    if s["weights"] == "bf16":
        return pick(s[name]).float()
    return _decode(pick(s[name]), pick(s[name + "_scales"])) * pick(s["g" + name])[:, None, None]


def _plain_moe(s):
    x, ids_w = s["x"].float(), _route(s)
    ids, w, chosen = ids_w
    t, k = ids.shape
    e, inter = s["logits"].shape[1], s["inter"]
    if t * k < e:
        # few tokens: the weights of each (token, choice) pair alone
        flat, rows = ids.reshape(-1), x.repeat_interleave(k, 0).unsqueeze(1)
        scale = w.reshape(-1, 1, 1)
    else:
        # every expert for every token; what a token did not choose gets weight 0
        flat, rows = None, x.unsqueeze(0).expand(e, -1, -1)
        scale = torch.zeros(t, e, device=x.device).scatter_(1, ids, w).t().reshape(e, t, 1)
    w1 = _plain_weights(s, "w1", flat)
    a = torch.matmul(rows, w1.transpose(1, 2).contiguous()).unflatten(-1, (inter // 8, 2, 8))
    del w1
    gate, up = a[..., 0, :].flatten(-2), a[..., 1, :].flatten(-2)
    h = gate / (1 + torch.exp(-gate)) * up * scale
    w2 = _plain_weights(s, "w2", flat)
    y = torch.matmul(h, w2.transpose(1, 2).contiguous())
    y = y.view(t, k, -1).sum(1) if flat is not None else y.sum(0)
    return y.to(torch.bfloat16), ids.int(), w


def run(s):
    if s["op"] == "tables":
        if not own:
            return _plain_tables(s)
        import moe_swiglu_epilogue_amd as M
        free = None if s["kind"] == "read" else s["free"]
        slots, offsets, lens, end = M.kv_block_tables(s["cached"], s["fresh"], s["table"], s["page"], s["max_tokens"],
                                                      free_pages=free)
        return slots, offsets, lens, end, s["table"]
    if s["op"] == "attn":
        if not own:
            return _plain_attn(s)
        import moe_swiglu_epilogue_amd as M
        return M.nvfp4_paged_attention(s["q"], s["k"], s["k_scales"], s["v"], s["v_scales"], s["table"], s["lens"],
                                       s["offsets"], kv_heads=s["kv_heads"], page_size=s["page"],
                                       max_query_len=s["max_query"], max_seq_len=s["max_seq"], window=s["window"],
                                       k_gs=s["gs"][0:1], v_gs=s["gs"][1:2], lse=True)
    if not own:
        return _plain_moe(s)
    import moe_swiglu_epilogue_amd as M
    if s["weights"] == "bf16":
        return M.moe_layer_bf16(s["x"], s["logits"], s["w1"], s["w2"], s["top_k"], renormalize=s["renormalize"])
    return M.moe_layer_nvfp4(s["x"], s["logits"], s["w1"], s["w1_scales"], s["w2"], s["w2_scales"], s["top_k"], s["gw1"],
                             s["gw2"], renormalize=s["renormalize"])


# ---- what a pass cannot do without -----------------------------------------------
def work(case):
    if case["op"] == "moe":
        e, h, i, t, k = (case[n] for n in ("experts", "hidden", "inter", "tokens", "top_k"))
        reached = e * (1 - (1 - k / e) ** t)      # experts that some token chooses, if choices were even
        each = 3 * i * h * (2 if case["weights"] == "bf16" else 9 / 16)
        return {"bytes": reached * each + t * (4 * h + 4 * e + 8 * k), "flops": 6.0 * t * k * i * h}
    cached, fresh = _lengths(case)
    if case["op"] == "tables":
        pages = sum(-(-(c + f) // case["page"]) for c, f in zip(cached, fresh))
        return {"bytes": 8.0 * sum(fresh) * 1.1 + 16.0 * len(fresh) + 8.0 * pages, "flops": 1.0 * sum(fresh)}
    window, keys, pairs = case["window"], 0, 0
    for c, f in zip(cached, fresh):
        keys += min(c + f, window + f - 1) if window else c + f
        lo, hi = c + 1, c + f                     # keys that the first and the last query see
        if window and lo >= window:
            pairs += window * f
        elif window and hi > window:
            pairs += (lo + window) * (window - lo + 1) // 2 + (hi - window) * window
        else:
            pairs += (lo + hi) * f // 2
    n, dim = sum(fresh), case["dim"]
    return {"bytes": keys * case["kv_heads"] * dim * 9 / 8 + n * case["heads"] * (4.0 * dim + 4),
            "flops": 4.0 * pairs * case["heads"] * dim}


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


def _exact_attn(case, s):
    q, dim, kv, page = s["q"].double(), s["dim"], s["kv_heads"], s["page"]
    group, gs = s["heads"] // kv, s["gs"].double().tolist()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    row = 0
    for b, (c, f) in enumerate(zip(*_lengths(case))):
        n = c + f
        pos = torch.arange(n, device=q.device)
        slot = s["table"][b].long()[pos // page] * page + pos % page
        k = _exact_values(s["k"][slot], s["k_scales"][slot]).view(n, kv, dim) * gs[0]
        v = _exact_values(s["v"][slot], s["v_scales"][slot]).view(n, kv, dim) * gs[1]
        here = torch.arange(c, n, device=q.device)
        hidden = pos[None, :] > here[:, None]
        if s["window"]:
            hidden |= pos[None, :] <= here[:, None] - s["window"]
        for h in range(s["heads"]):
            z = q[row:row + f, h] @ k[:, h // group].t().contiguous() / math.sqrt(dim)
            z[hidden] = -math.inf
            lse[row:row + f, h] = torch.logsumexp(z, 1)
            out[row:row + f, h] = torch.softmax(z, 1) @ v[:, h // group].contiguous()
        row += f
    return out, lse


def _exact_moe(case, s):
    x, logits = s["x"].double(), s["logits"].double()
    k = s["top_k"]
    order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
    prob = torch.softmax(logits, 1).gather(1, order)
    if s["renormalize"]:
        prob = prob / prob.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    j = torch.arange(s["inter"], device=x.device)
    for e in sorted(set(order.reshape(-1).tolist())):
        if s["weights"] == "bf16":
            w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        else:
            w1 = _exact_values(s["w1"][e], s["w1_scales"][e]) * float(s["gw1"][e])
            w2 = _exact_values(s["w2"][e], s["w2_scales"][e]) * float(s["gw2"][e])
        token, choice = (order == e).nonzero(as_tuple=True)
        a = x[token] @ w1.t().contiguous()
        gate, up = a[:, 16 * (j // 8) + j % 8], a[:, 16 * (j // 8) + 8 + j % 8]
        y = (gate * torch.sigmoid(gate) * up) @ w2.t().contiguous()
        out.index_add_(0, token, y * prob[token, choice].unsqueeze(1))
    return out, None, prob


def _exact_tables(case, s):
    page, table = s["page"], s["table"].tolist()
    free, cached, fresh = s["free"].tolist(), s["cached"].tolist(), s["fresh"].tolist()
    slots, offsets, lens, taken = [], [0], [], 0
    for b, (c, f) in enumerate(zip(cached, fresh)):
        if s["kind"] != "read":
            for p in range(-(-c // page), -(-(c + f) // page)):
                table[b][p] = free[taken]
                taken += 1
        slots += [table[b][t // page] * page + t % page for t in range(c, c + f)]
        offsets.append(len(slots))
        lens.append(c + f)
    slots += [-1] * (s["max_tokens"] - len(slots))
    whole = lambda v, t: torch.tensor(v, dtype=t)  # noqa: E731
    return whole(slots, torch.int64), whole(offsets, torch.int32), whole(lens, torch.int32), whole([taken], torch.int32), whole(table, torch.int32)


def exact(case, seed):
    s = prepare(case, seed)
    return {"tables": _exact_tables, "attn": _exact_attn, "moe": _exact_moe}[case["op"]](case, s)
