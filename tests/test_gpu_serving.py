"""The decoding-step operators on the GPU (include/nvfp4_serving.h) against
their plain definitions in 64 bits (tests/serving_ref.py): block tables and
slots exactly, attention and the MoE layer within bounds that count their
roundings; empty rows and requests, hidden pages, odd sizes, pitches, other
streams, captured graphs, and the operators run one after the other."""
import math

import numpy as np
import pytest
import torch

import serving_ref as R

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu]", *a, flush=True)


@pytest.fixture(scope="module")
def M():
    import moe_swiglu_epilogue_amd as M
    assert torch.cuda.is_available(), "these tests need the GPU"
    M.serving.raw()
    return M


def ints(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def host(t):
    torch.cuda.synchronize()
    return t.cpu()


# ---- block tables ----------------------------------------------------------------
def table_case(seed, seqs, longest, page, kind, spare=3):
    """Random lengths (zeros and a negative one among them), a table with the
    held pages, a free list."""
    r = np.random.default_rng(seed)
    context = r.integers(0, longest + 1, seqs)
    query = np.ones(seqs, np.int64) if kind == "step" else r.integers(0, longest + 1, seqs)
    context[::5] = 0
    query[3::7] = 0
    if seqs > 4:
        query[4] = -3
    pages_of = lambda n: -(-n // page)  # noqa: E731
    total = context + np.maximum(query, 0)
    width = int(pages_of(total).max()) + 1
    count = int(pages_of(total).sum()) + spare
    order = r.permutation(count)
    table, used = np.full((seqs, width), -7, np.int64), 0
    for b in range(seqs):
        held = pages_of(total[b] if kind == "read" else context[b])
        table[b, :held] = order[used:used + held]
        used += held
    return context.tolist(), query.tolist(), table.tolist(), order[used:].tolist()


def check_tables(M, context, query, table, page, max_tokens, free=None, begin=None, pitch=0):
    n, width = len(query), len(table[0]) if table else 0
    wide = torch.full((n, width + pitch), -99, dtype=torch.int32)
    wide[:, :width] = torch.tensor(table, dtype=torch.int32).reshape(n, width)
    dev = wide.cuda()
    got = M.kv_block_tables(None if context is None else ints(context), ints(query), dev[:, :width], page, max_tokens,
                            free_pages=None if free is None else ints(free),
                            free_begin=None if begin is None else ints([begin]))
    want_table = [list(r) for r in table]
    slots, offsets, lens, end = R.kv_block_tables(context, query, want_table, page, max_tokens, free, begin)
    assert host(got[0]).tolist() == slots
    assert host(got[1]).tolist() == offsets
    assert host(got[2]).tolist() == lens
    assert host(got[3]).tolist() == [end]
    wide[:, :width] = torch.tensor(want_table, dtype=torch.int32).reshape(n, width)
    assert torch.equal(host(dev), wide)


@pytest.mark.parametrize("seed,seqs,longest,page,kind", [
    (1, 1, 1, 1, "step"), (2, 5, 40, 16, "step"), (3, 256, 300, 16, "step"), (4, 257, 90, 7, "prompts"),
    (5, 33, 2000, 64, "prompts"), (6, 4096, 20, 3, "prompts"), (7, 64, 500, 24, "read"), (8, 3, 5000, 1, "prompts"),
    (9, 4095, 5, 1000, "step")])
def test_block_tables(M, seed, seqs, longest, page, kind):
    context, query, table, free = table_case(seed, seqs, longest, page, kind)
    if kind == "read":
        query = [c + max(q, 0) for c, q in zip(context, query)]
        context, free = None, None
    total = sum(max(q, 0) for q in query)
    for max_tokens in {total, total + 77, max(0, total // 2)}:
        say("kv_block_tables", seed, seqs, longest, page, kind, max_tokens)
        check_tables(M, context, query, table, page, max_tokens, free, pitch=seed % 3)


def test_block_tables_edges(M):
    context, query, table, free = table_case(11, 20, 100, 8, "prompts")
    total = sum(max(q, 0) for q in query)
    say("short, empty and shifted lists")
    for f, begin in ((free[:5], None), ([], None), (free, 2), (free + [5, 6, 7, 8], 4), (free, len(free)), (free, -1),
                     (free, len(free) + 1), ([], 0)):
        check_tables(M, context, query, table, 8, total, f, begin)
    say("no request, no token, no page")
    check_tables(M, [], [], [], 8, 5, [1, 2])
    check_tables(M, [], [], [], 8, 0)
    check_tables(M, [0, 0], [0, 0], [[-1], [-1]], 8, 3, [4])
    check_tables(M, [3, 9], [4, 1], [[], []], 8, 6, [4])
    say("a table too narrow for its requests")
    check_tables(M, [3, 9, 0], [40, 1, 5], [[1, 2], [3, 4], [0, 0]], 8, 50, [9, 8, 7, 6])
    check_tables(M, None, [40, 1, 0, 17], [[1, 2], [3, -1], [5, 6], [7, -1]], 8, 70)
    say("entries outside the cache are left to the reader; negative ones give no slot")
    check_tables(M, [20, 20], [3, 3], [[5, -2, 10 ** 9], [0, 1, -1]], 8, 6, [3])
    say("sums past 2^31 - 1 saturate")
    big = 2 ** 31 - 1
    check_tables(M, [big, 5, big], [big, big, 1], [[1], [2], [3]], big, 64, [4, 5])


# ---- attention ---------------------------------------------------------------------
def attn_case(seed, heads, kv_heads, dim, page, totals, news, hide=(), pad=0, width=None, scale=None):
    """Random q and caches, pages in random order; `hide`: (request, column,
    entry) replacements in the table; `pad` rows of q before and after."""
    g = torch.Generator().manual_seed(seed)
    seqs = len(totals)
    need = [-(-max(t, 0) // page) for t in totals]
    width = max(need + [1]) + 1 if width is None else width
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table, used = torch.full((seqs, width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :min(n, width)] = order[used:used + n][:width]
        used += n
    for b, col, entry in hide:
        table[b, col] = entry
    cols = kv_heads * dim
    kp, ks = R.random_nvfp4(g, pages * page, cols)
    vp, vs = R.random_nvfp4(g, pages * page, cols)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(news)]) + pad, dtype=torch.int32)
    tokens = int(offsets[-1]) + pad
    q = torch.randn(tokens, heads, dim, generator=g).to(torch.bfloat16)
    return dict(q=q, kp=kp, ks=ks, vp=vp, vs=vs, table=table, lens=torch.tensor(totals, dtype=torch.int32),
                offsets=offsets, kv_heads=kv_heads, page=page, scale=scale or 0.3 / math.sqrt(dim))


def call_attention(M, c, dev, out=None, lse=True, max_query_len=None, max_seq_len=None, **more):
    o = c["offsets"]
    return M.nvfp4_paged_attention(
        dev["q"], dev["kp"], dev["ks"], dev["vp"], dev["vs"], dev["table"], dev["lens"], dev["offsets"],
        kv_heads=c["kv_heads"], page_size=c["page"], scale=c["scale"], out=out, lse=lse,
        max_query_len=int((o[1:] - o[:-1]).max()) if max_query_len is None else max_query_len,
        max_seq_len=max(int(c["lens"].max()), 0) if max_seq_len is None else max_seq_len, **more)


def device(c):
    return {k: v.cuda() for k, v in c.items() if isinstance(v, torch.Tensor)}


def check_attention(M, c, causal=True, window=0, gs=None, **more):
    dev = device(c)
    k_gs, v_gs = (1.0, 1.0) if gs is None else gs
    scalar = lambda v: None if gs is None else torch.tensor([v], dtype=torch.float32).cuda()  # noqa: E731
    out = torch.full_like(dev["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    call_attention(M, c, dev, out=out, lse=lse, causal=causal, window=window, k_gs=scalar(k_gs), v_gs=scalar(v_gs), **more)
    ref, ref_lse, tol, lse_tol = R.paged_attention(
        c["q"], c["kp"], c["ks"], c["vp"], c["vs"], c["table"], c["lens"], c["offsets"], c["kv_heads"], c["page"],
        c["scale"], causal, window, k_gs, v_gs)
    got, got_lse = host(out).double(), host(lse).double()
    mine = ~torch.isnan(ref_lse[:, 0])
    assert bool((got[~mine] == 7.0).all()) and bool((got_lse[~mine] == 7.0).all())       # rows of no request
    assert torch.equal(torch.isinf(got_lse[mine]), torch.isinf(ref_lse[mine]))
    seen = mine[:, None] & ~torch.isinf(ref_lse)
    assert bool((got_lse[mine[:, None] & torch.isinf(ref_lse)] == -math.inf).all())
    worst = ((got - ref).abs() - tol)[mine]
    assert worst.numel() == 0 or worst.max() <= 0, (worst.max(), (got - ref).abs()[mine].max())
    z = ((got_lse - ref_lse).abs() - lse_tol)[seen]
    assert z.numel() == 0 or z.max() <= 0, z.max()
    assert bool((got[mine & torch.isinf(ref_lse[:, 0])] == 0).all())


@pytest.mark.parametrize("heads,kv_heads,dim,page", [
    (8, 8, 64, 16), (32, 8, 128, 16), (14, 2, 64, 7), (48, 1, 128, 1), (12, 4, 256, 24), (64, 8, 128, 64),
    (24, 3, 64, 32), (7, 7, 128, 5), (40, 2, 256, 16), (20, 5, 128, 16)])
def test_attention_decode(M, heads, kv_heads, dim, page):
    """One token a request, contexts from 1 to past several tiles."""
    totals = [1, 2, 15, 16, 17, 31, 33, 64, 100, 129, 300, 511]
    c = attn_case(heads * 7 + dim, heads, kv_heads, dim, page, totals, [1] * len(totals), pad=2)
    say("attention decode", heads, kv_heads, dim, page)
    check_attention(M, c, gs=(0.7, 1.9))
    check_attention(M, c, window=20)


@pytest.mark.parametrize("heads,kv_heads,dim,page,longest", [(16, 2, 128, 16, 4097), (4, 4, 64, 64, 9000),
                                                             (8, 1, 256, 48, 3001), (96, 1, 128, 16, 2500)])
def test_attention_long(M, heads, kv_heads, dim, page, longest):
    """Few requests with long contexts: the work of a row is split."""
    c = attn_case(dim + page, heads, kv_heads, dim, page, [longest, 700, 1], [1, 1, 1])
    say("attention long", heads, kv_heads, dim, page, longest)
    check_attention(M, c)
    check_attention(M, c, window=longest // 2 + 3)


@pytest.mark.parametrize("heads,kv_heads,dim,page,news", [
    (32, 8, 128, 16, [5, 3, 0, 8, 1]), (8, 8, 64, 16, [4, 4, 4, 4, 4]), (24, 2, 256, 32, [2, 7, 1, 0, 3]),
    (12, 3, 64, 9, [17, 2, 33, 1, 5])])
def test_attention_few_queries(M, heads, kv_heads, dim, page, news):
    totals = [700, 3, 129, 64, 17]
    c = attn_case(dim + heads, heads, kv_heads, dim, page, totals, news, pad=1)
    say("attention few queries", heads, kv_heads, dim, page, news)
    check_attention(M, c, gs=(1.25, 0.5))
    check_attention(M, c, window=11)
    check_attention(M, c, causal=False)
    check_attention(M, c, causal=False, window=40)


@pytest.mark.parametrize("heads,kv_heads,dim,page,totals,news", [
    (8, 2, 128, 16, [300, 129, 257], [300, 129, 257]), (4, 4, 64, 16, [513, 40], [100, 40]),
    (4, 1, 256, 64, [700, 65], [130, 65]), (6, 2, 128, 10, [333, 1, 200], [70, 1, 199]),
    (16, 1, 128, 32, [900], [64]), (3, 1, 64, 1, [150, 150], [150, 20])])
def test_attention_prompts(M, heads, kv_heads, dim, page, totals, news):
    c = attn_case(dim + heads + page, heads, kv_heads, dim, page, totals, news, pad=3)
    say("attention prompts", heads, kv_heads, dim, page, totals, news)
    check_attention(M, c, gs=(0.9, 1.1))
    check_attention(M, c, window=50)
    check_attention(M, c, causal=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_rows_that_see_nothing(M, dim):
    """Empty contexts, negative lengths, queries before the context, hidden
    pages (negative, past the cache) and a request all of whose pages are hidden."""
    totals, news = [0, -5, 3, 40, 80, 33, 130, 90], [1, 2, 6, 1, 3, 1, 40, 90]
    hide = [(3, 1, -1), (4, 0, 10 ** 9), (4, 2, -2 ** 31), (5, 0, -1), (5, 1, 2 ** 31 - 1), (5, 2, 500),
            (6, 0, -1), (6, 4, -1), (7, 1, -1), (7, 3, 10 ** 6)]
    for news_ in (news, [1] * 8):
        c = attn_case(dim, 8, 2, dim, 16, totals, news_, hide=hide, pad=1)
        say("attention hidden", dim, news_)
        check_attention(M, c)
        check_attention(M, c, causal=False)
        check_attention(M, c, window=7)


def test_attention_hints_steer_speed_only(M):
    """max_query_len and max_seq_len below the real lengths, or far above."""
    c = attn_case(5, 16, 4, 128, 16, [2000, 700, 90], [40, 3, 90])
    for mq, ms in ((1, 10), (1, 0), (0, 0), (90, 16), (4, 5000), (5000, 100000), (20, 2000)):
        say("attention hints", mq, ms)
        check_attention(M, c, max_query_len=mq, max_seq_len=ms)


def test_attention_table_narrower_than_length(M):
    c = attn_case(6, 8, 2, 64, 16, [100, 30], [1, 2], width=3)
    say("attention narrow table")
    check_attention(M, c)


@pytest.mark.parametrize("dim,page", [(64, 16), (64, 9), (128, 32), (128, 5)])
@pytest.mark.parametrize("news", [16, 17, 32, 33, 41, 48, 49, 64, 65, 96, 97, 128, 129])
def test_attention_row_blocks(M, dim, page, news):
    """Every size of a block of query rows, full and with a ragged end."""
    c = attn_case(news + dim, 2, 2, dim, page, [333, 140, 64], [news, 3, 1], pad=1)
    say("attention row blocks", dim, page, news)
    check_attention(M, c)
    check_attention(M, c, window=70)


@pytest.mark.parametrize("news", [[1, 2], [60, 70]])
@pytest.mark.parametrize("empty", ["cache", "table"])
def test_attention_without_cache_or_table(M, empty, news):
    """A cache of no slots, a table of no columns: every row sees nothing, and
    the null pointers of empty tensors are not read."""
    c = attn_case(12, 8, 2, 128, 16, [40, 70], news)
    if empty == "cache":
        for k in ("kp", "ks", "vp", "vs"):
            c[k] = c[k][:0]
    else:
        c["table"] = c["table"][:, :0]
    dev = device(c)
    say("attention without", empty, news)
    for window in (0, 9):
        out, lse = call_attention(M, c, dev, window=window)
        assert bool((host(out) == 0).all()) and bool((host(lse) == -math.inf).all())


@pytest.mark.parametrize("hint", [1, 600])
def test_attention_most_requests(M, hint):
    """The most (request, key/value head) pairs that are taken, nearly all of
    them without a query: grids stay inside what a launch takes."""
    n, totals, news = 65535, [5, 40], [1, 2]
    c = attn_case(14, 64, 64, 64, 16, totals, news)
    dev = device(c)
    want = call_attention(M, c, dev)
    offsets = torch.full((n + 1,), 3, dtype=torch.int32)
    offsets[:n - 1] = 0
    offsets[n - 1] = 1
    lens = torch.zeros(n, dtype=torch.int32)
    lens[n - 2:] = c["lens"]
    table = torch.full((n, c["table"].shape[1]), -1, dtype=torch.int32)
    table[n - 2:] = c["table"]
    dev.update(offsets=offsets.cuda(), lens=lens.cuda(), table=table.cuda())
    say("attention most requests", hint)
    got = call_attention(M, c, dev, max_query_len=hint)
    ref, ref_lse, tol, lse_tol = R.paged_attention(
        c["q"], c["kp"], c["ks"], c["vp"], c["vs"], c["table"], c["lens"], c["offsets"], 64, 16, c["scale"], True, 0, 1.0, 1.0)
    for out, lse in (want, got):
        assert bool(((host(out).double() - ref).abs() <= tol).all())
        assert bool(((host(lse).double() - ref_lse).abs() <= lse_tol).all())


@pytest.mark.parametrize("page,news", [(16, [1, 1, 1]), (10, [1, 1, 1]), (16, [5, 30, 100]), (6, [5, 30, 100])])
def test_attention_unseen_slots_may_hold_anything(M, page, news):
    """Slots behind a request's tokens, of hidden pages and of no request: NaN
    scales and any code there change no byte of the result."""
    c = attn_case(15, 8, 2, 128, page, [200, 37, 111], news, hide=[(0, 1, -1), (2, 0, 10 ** 7)])
    say("attention unseen slots", page, news)
    want = call_attention(M, c, device(c))
    mine = torch.zeros(c["kp"].shape[0], dtype=torch.bool)
    for b, n in enumerate(c["lens"].tolist()):
        for t in range(n):
            entry = int(c["table"][b, t // page])
            if 0 <= entry < len(mine) // page:
                mine[entry * page + t % page] = True
    for k, v in (("kp", 0xff), ("ks", 0x7f), ("vp", 0x77), ("vs", 0xff)):
        c[k] = c[k].clone()
        c[k][~mine] = v
    got = call_attention(M, c, device(c))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check_attention(M, c)


def test_attention_on_two_streams_at_once(M):
    """Two calls that split their rows, each with a workspace and stream of its own."""
    cases = [attn_case(16 + i, 16, 2, 128, 16, [3500, 900], [1, 1]) for i in range(2)]
    devs = [device(c) for c in cases]
    want = [call_attention(M, c, d) for c, d in zip(cases, devs)]
    need = M.serving.raw().nvfp4_paged_attention_workspace(2, 16, 2, 128, 2, 1, 3500, 0)
    assert need > 0
    work = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    say("attention on two streams")
    got = []
    for _ in range(4):
        for c, d, w, s in zip(cases, devs, work, streams):
            got.append(call_attention(M, c, d, workspace=w, stream=s))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_attention_widest_window(M):
    """Windows up to the type's largest value hide nothing, also for queries in
    front of the context (positions below 0)."""
    for news in ([1, 5], [30, 90]):
        c = attn_case(13, 8, 2, 64, 16, [200, 3], news)
        dev = device(c)
        say("attention wide windows", news)
        want = call_attention(M, c, dev, causal=False)
        for window in (2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1):
            got = call_attention(M, c, dev, causal=False, window=window)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), window


def test_attention_large_and_small_values(M):
    """q over BF16's range (rows scaled by 2^100 and 2^-100) with scores kept
    moderate by `scale`; scores far apart (one key takes all the weight)."""
    for power, scale in ((100, 2.0 ** -107), (-100, 2.0 ** 97), (0, 30.0)):
        for news in ([1, 1], [70, 3]):
            c = attn_case(9, 8, 2, 128, 16, [200, 77], news, scale=scale)
            c["q"] = (c["q"].float() * 2.0 ** power).to(torch.bfloat16)
            say("attention range", power, scale, news)
            check_attention(M, c)


def test_attention_pitched_rows_and_other_stream(M):
    c = attn_case(8, 8, 2, 128, 16, [90, 41], [1, 20])
    dev = device(c)
    want, want_lse = call_attention(M, c, dev)
    wide = torch.full((21, 3 * 8 * 128), 3.0, dtype=torch.bfloat16).cuda()
    wide[:, 1024:2048] = dev["q"].view(21, 1024)
    out = torch.full((21, 2 * 8 * 128), 5.0, dtype=torch.bfloat16).cuda()
    table = torch.full((2, c["table"].shape[1] + 5), -1, dtype=torch.int32).cuda()
    table[:, :c["table"].shape[1]] = dev["table"]
    d2 = dict(dev, q=wide[:, 1024:2048].view(21, 8, 128), table=table[:, :c["table"].shape[1]])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("attention pitched, side stream")
    _, lse = call_attention(M, c, d2, out=out[:, :1024].view(21, 8, 128), stream=side)
    side.synchronize()
    assert torch.equal(out[:, :1024].view(21, 8, 128), want) and bool((out[:, 1024:] == 5.0).all())
    assert torch.equal(lse, want_lse)
    assert torch.equal(call_attention(M, c, dev, lse=None), want)       # lse is optional


# ---- mixture of experts ---------------------------------------------------------------
def moe_case(seed, kind, tokens, hidden, inter, experts):
    g = torch.Generator().manual_seed(seed)
    c = dict(x=torch.randn(tokens, hidden, generator=g).to(torch.bfloat16),
             logits=torch.randn(tokens, experts, generator=g), kind=kind, inter=inter)
    if kind == "bf16":
        c["w1"] = (torch.randn(experts, 2 * inter, hidden, generator=g) / math.sqrt(hidden)).to(torch.bfloat16)
        c["w2"] = (torch.randn(experts, hidden, inter, generator=g) / math.sqrt(inter)).to(torch.bfloat16)
        c["w1d"], c["w2d"] = c["w1"].double(), c["w2"].double()
    else:
        c["w1"], c["s1"] = R.random_nvfp4(g, experts, 2 * inter, hidden)
        c["w2"], c["s2"] = R.random_nvfp4(g, experts, hidden, inter)
        c["gs1"] = (0.5 + torch.rand(experts, generator=g)) / math.sqrt(8 * hidden)
        c["gs2"] = (0.5 + torch.rand(experts, generator=g)) / math.sqrt(8 * inter)
        c["w1d"] = R.nvfp4_values(c["w1"], c["s1"]) * c["gs1"].double()[:, None, None]
        c["w2d"] = R.nvfp4_values(c["w2"], c["s2"]) * c["gs2"].double()[:, None, None]
    return c


def call_moe(M, c, dev, top_k, **more):
    if c["kind"] == "bf16":
        return M.moe_layer_bf16(dev["x"], dev["logits"], dev["w1"], dev["w2"], top_k, **more)
    return M.moe_layer_nvfp4(dev["x"], dev["logits"], dev["w1"], dev["s1"], dev["w2"], dev["s2"], top_k, dev.get("gs1"),
                             dev.get("gs2"), **more)


def check_moe(M, c, top_k, renormalize):
    out, ids, weights = call_moe(M, c, device(c), top_k, renormalize=renormalize)
    h_eps = 2.0 ** -17 if c["kind"] == "bf16" else 2.0 ** -11
    ref, tol, want_ids, want = R.moe_layer(c["x"], c["logits"], c["w1d"], c["w2d"], top_k, renormalize, h_eps)
    assert np.array_equal(host(ids).numpy(), want_ids)
    w = host(weights).double().numpy()
    assert np.all(np.abs(w - want) <= 2.0 ** -19 * want + 2.0 ** -140), np.abs(w - want).max()
    d = (host(out).double() - ref).abs() - tol
    assert d.numel() == 0 or d.max() <= 0, d.max()


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("tokens,hidden,inter,experts,top_k", [
    (1, 32, 32, 1, 1), (1, 256, 128, 8, 2), (3, 544, 96, 8, 2), (5, 128, 160, 64, 8), (16, 512, 64, 4, 4),
    (17, 160, 224, 6, 3), (33, 96, 96, 16, 2), (64, 256, 128, 10, 4), (64, 64, 64, 512, 1), (2, 1056, 544, 5, 5),
    (7, 64, 32, 40, 32), (48, 128, 64, 2, 1)])
def test_moe_layer(M, kind, tokens, hidden, inter, experts, top_k):
    c = moe_case(tokens + hidden, kind, tokens, hidden, inter, experts)
    for renormalize in (True, False):
        say("moe", kind, tokens, hidden, inter, experts, top_k, renormalize)
        check_moe(M, c, top_k, renormalize)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("tokens,top_k", [(64, 1), (50, 2), (33, 3)])
def test_moe_one_expert_takes_all(M, kind, tokens, top_k):
    """Far more tokens on one expert than its share: several passes."""
    c = moe_case(78, kind, tokens, 96, 64, 48)
    c["logits"][:, 41] = 20.0
    say("moe one expert", kind, tokens, top_k)
    check_moe(M, c, top_k, True)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
def test_moe_routing_edges(M, kind):
    """Ties, -inf and NaN logits, fewer experts left than top_k, one expert
    that takes every token, probabilities that underflow, +inf."""
    inf, nan = math.inf, math.nan
    for tokens in (1, 12):
        c = moe_case(77, kind, 12, 96, 64, 12)
        z = c["logits"]
        z[0] = 0.25
        z[1, 3:] = -inf
        z[2] = -inf
        z[3, ::2] = nan
        z[4] = nan
        z[5] = torch.arange(12).float() * 60
        z[6, 4], z[6, 7] = inf, 1.0
        z[7, 2], z[7, 9] = inf, inf
        z[8] = -0.0
        z[8, 5:] = 0.0
        z[9:] = torch.tensor([1.0 if e == 6 else -5.0 - e for e in range(12)])
        for first in range(0, 12, tokens):
            d = dict(c, x=c["x"][first:first + tokens].clone(), logits=z[first:first + tokens].clone())
            for top_k in (1, 4, 12):
                for renormalize in (True, False):
                    say("moe routing", kind, tokens, first, top_k, renormalize)
                    check_moe(M, d, top_k, renormalize)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
def test_moe_activation_range(M, kind):
    """x scaled by 2^40 and 2^-40 with the weights' scale against it; single
    huge channels; rows of zeros."""
    for power in (40, -40):
        c = moe_case(5, kind, 4, 256, 64, 4)
        c["x"] = (c["x"].float() * 2.0 ** power).to(torch.bfloat16)
        c["x"][1] = 0
        c["x"][2, 7] = c["x"][2, 7] * 1000
        if kind == "bf16":
            c["w1"] = (c["w1"].float() * 2.0 ** -power).to(torch.bfloat16)
            c["w1d"] = c["w1"].double()
        else:
            c["gs1"] = c["gs1"] * 2.0 ** -power
            c["w1d"] = c["w1d"] * 2.0 ** -power
        say("moe range", kind, power)
        check_moe(M, c, 2, True)


def test_moe_scales_are_optional_and_rows_pitched(M):
    c = moe_case(6, "nvfp4", 9, 128, 96, 5)
    dev = device(c)
    one = torch.ones(5).cuda()
    want = call_moe(M, c, dict(dev, gs1=one, gs2=one), 2)
    plain = dict(dev)
    plain.pop("gs1"), plain.pop("gs2")
    got = call_moe(M, c, plain, 2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    wide = torch.full((9, 300), 3.0, dtype=torch.bfloat16).cuda()[:, :296]
    wide[:, 8:136] = dev["x"]
    out = torch.full((9, 264), 5.0, dtype=torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("moe pitched, side stream")
    with pytest.raises(M.Nvfp4Error):
        call_moe(M, c, dict(plain, x=wide[:, 8:136]), 2)       # a 600-byte pitch
    wide = torch.full((9, 304), 3.0, dtype=torch.bfloat16).cuda()
    wide[:, 8:136] = dev["x"]
    torch.cuda.synchronize()
    got = call_moe(M, c, dict(plain, x=wide[:, 8:136]), 2, out=out[:, 8:136], stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and bool((out[:, :8] == 5.0).all()) and bool((out[:, 136:] == 5.0).all())


# ---- together ---------------------------------------------------------------------------
def step_state(M, seed=3):
    """A small layer's decoding state: 6 requests, pages of 16, 8/2 heads of 128."""
    g = torch.Generator().manual_seed(seed)
    s = dict(context=ints([40, 0, 17, 63, 100, 31]), query=ints([1, 5, 1, 2, 0, 1]),
             table=torch.full((6, 9), -1, dtype=torch.int32))
    order = torch.randperm(40, generator=g).to(torch.int32)
    used = 0
    for b, n in enumerate((3, 0, 2, 4, 7, 2)):
        s["table"][b, :n] = order[used:used + n]
        used += n
    s["free"] = order[used:].contiguous().cuda()
    s["table"] = s["table"].cuda()
    for n in ("k", "v"):
        p, sc = R.random_nvfp4(g, 40 * 16, 256)
        s[n], s[n + "s"] = p.cuda(), sc.cuda()
        s["new_" + n] = torch.randn(12, 256, generator=g).to(torch.bfloat16).cuda()
    s["q"] = torch.randn(12, 8, 128, generator=g).to(torch.bfloat16).cuda()
    w = moe_case(seed, "nvfp4", 12, 1024, 64, 6)
    s.update({k: v.cuda() for k, v in w.items() if isinstance(v, torch.Tensor)})
    return s


def one_step(M, s):
    slots, offsets, lens, end = M.kv_block_tables(s["context"], s["query"], s["table"], 16, 12, free_pages=s["free"])
    M.nvfp4_quantize_paged(s["new_k"], slots, s["k"], s["ks"])
    M.nvfp4_quantize_paged(s["new_v"], slots, s["v"], s["vs"])
    o, lse = M.nvfp4_paged_attention(s["q"], s["k"], s["ks"], s["v"], s["vs"], s["table"], lens, offsets, kv_heads=2,
                                     page_size=16, max_query_len=5, lse=True)
    y, ids, w = M.moe_layer_nvfp4(o.view(12, 1024), s["logits"], s["w1"], s["s1"], s["w2"], s["s2"], 2, s["gs1"], s["gs2"])
    return dict(slots=slots, offsets=offsets, lens=lens, end=end, table=s["table"], o=o[:10], lse=lse[:10], y=y[:10],
                ids=ids, w=w)


def test_one_decoding_step(M):
    """Pages, cache writes, attention and the MoE layer one after the other,
    against the definitions on what the cache then holds (read back through
    kv_block_tables' read map and nvfp4_dequantize_paged)."""
    s = step_state(M)
    say("one step")
    r = one_step(M, s)
    total = int(host(r["lens"]).sum())
    slots, _, _, _ = M.kv_block_tables(None, r["lens"], s["table"], 16, total)
    keys = host(M.nvfp4_dequantize_paged(s["k"], s["ks"], slots)).double()
    lens = host(r["lens"]).tolist()
    assert lens == [41, 5, 18, 65, 100, 32]
    c = dict(q=host(s["q"]), kp=host(s["k"]), ks=host(s["ks"]), vp=host(s["v"]), vs=host(s["vs"]), table=host(s["table"]),
             lens=host(r["lens"]), offsets=host(r["offsets"]))
    row = 0
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        at = c["table"][b].long()[pos // 16] * 16 + pos % 16
        assert torch.equal(keys[row:row + n], R.nvfp4_values(c["kp"][at], c["ks"][at]))
        row += n
    ref, ref_lse, tol, lse_tol = R.paged_attention(*[c[k] for k in ("q", "kp", "ks", "vp", "vs", "table", "lens", "offsets")],
                                                   2, 16, 1 / math.sqrt(128))
    assert ((host(r["o"]).double() - ref[:10]).abs() <= tol[:10]).all()
    assert ((host(r["lse"]).double() - ref_lse[:10]).abs() <= lse_tol[:10]).all()
    y, ytol, ids, _ = R.moe_layer(host(r["o"]).view(10, 1024), host(s["logits"])[:10],
                                  R.nvfp4_values(host(s["w1"]), host(s["s1"])) * host(s["gs1"]).double()[:, None, None],
                                  R.nvfp4_values(host(s["w2"]), host(s["s2"])) * host(s["gs2"]).double()[:, None, None],
                                  2, True, 2.0 ** -11)
    assert np.array_equal(host(r["ids"])[:10].numpy(), ids)
    assert ((host(r["y"]).double() - y).abs() <= ytol).all()


def test_graph_replays_match_eager(M):
    """The whole step captured into a graph and replayed, with eager steps
    (their own workspaces) and synchronizations in between."""
    s = step_state(M)
    want = {k: host(v).clone() for k, v in one_step(M, s).items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one_step(M, s)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = one_step(M, s)
    for r in range(4):
        for k, v in captured.items():
            if k != "table":
                v.zero_()
        if r % 2:
            one_step(M, s)
        torch.cuda.synchronize()
        say("graph replay", r)
        graph.replay()
        for k, v in captured.items():
            assert torch.equal(host(v), want[k]), (r, k)


def test_same_inputs_same_bytes(M):
    c = attn_case(12, 16, 2, 128, 16, [3000, 1500, 40], [1, 1, 1])
    dev = device(c)
    w = moe_case(13, "nvfp4", 20, 512, 128, 8)
    wd = device(w)
    a = [x.clone() for x in call_attention(M, c, dev)] + [x.clone() for x in call_moe(M, w, wd, 3)]
    for r in range(5):
        b = list(call_attention(M, c, dev)) + list(call_moe(M, w, wd, 3))
        assert all(torch.equal(x, y) for x, y in zip(a, b)), r
