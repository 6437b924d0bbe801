"""The sparse-attention operators on the GPU (include/nvfp4_sparse.h) against
their plain definitions (tests/sparse_ref.py): rotated queries, cache bytes, page
keys and page lists bit for bit, attention within bounds that count its roundings;
(a page key half way between two numbers may be either here, and is held to one in
test_gpu_sparse_routes.py)
empty rows and requests, hidden pages, odd sizes, pitches, other streams, captured
graphs, and the operators run one after the other."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import serving_ref as R
import sparse_ref as S

pytestmark = pytest.mark.gpu


def say(*a):
    print("[gpu]", *a, flush=True)


@pytest.fixture(scope="module")
def M():
    import moe_swiglu_epilogue_amd as M
    assert torch.cuda.is_available(), "these tests need the GPU"
    M.sparse.raw()
    return M


def host(t):
    torch.cuda.synchronize()
    return t.cpu()


def device(c):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}


# ---- rotation and append ---------------------------------------------------------
def append_case(seed, tokens, heads, kv, dim, rot, axes=1, most=500, slots=None, by_axis=None, table_of="angles"):
    """Rows of a fused projection, positions in and out of the table, slots in and
    out of the cache."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(tokens, heads + 2 * kv, dim, generator=g) * torch.exp(torch.randn(dim, generator=g))
    qkv[torch.rand(qkv.shape, generator=g) < 0.02] = 0.0
    qkv[torch.rand(qkv.shape, generator=g) < 0.02] = -0.0
    if tokens > 3:
        qkv[3] = 0.0
    num = tokens + 5 if slots is None else slots
    at = torch.randperm(num, generator=g)[:tokens] if num >= tokens else torch.randint(0, num, (tokens,), generator=g)
    if tokens > 6:
        at[1], at[4], at[6] = -1, num, 2 ** 62
    positions = torch.randint(0, most, (axes, tokens), generator=g, dtype=torch.int32)
    if tokens > 6:
        positions[0, 2], positions[-1, 5], positions[0, 6] = most, -1, 2 ** 31 - 1
    angle = torch.randint(0, 10 ** 6, (most, rot // 2), generator=g).double()
    cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float() * 1.2
    axis = None
    if axes > 1 or by_axis:
        axis = torch.randint(0, axes, (rot // 2,), generator=g, dtype=torch.int32)
        if by_axis:
            axis[0], axis[-1] = -1, axes
    return dict(qkv=qkv.to(torch.bfloat16), heads=heads, kv=kv, positions=positions, cos_sin=cos_sin, axis=axis, slots=at,
                kp=torch.randint(0, 256, (num, kv * dim // 2), generator=g, dtype=torch.uint8),
                ks=torch.randint(0, 127, (num, kv * dim // 16), generator=g, dtype=torch.uint8),
                vp=torch.randint(0, 256, (num, kv * dim // 2), generator=g, dtype=torch.uint8),
                vs=torch.randint(0, 127, (num, kv * dim // 16), generator=g, dtype=torch.uint8))


def parts(c):
    h, kv = c["heads"], c["kv"]
    return c["qkv"][:, :h], c["qkv"][:, h:h + kv], c["qkv"][:, h + kv:]


def call_append(M, c, with_q=True, gs=(None, None), interleaved=False, **more):
    q, k, v = parts(c)
    scalar = lambda x: None if x is None else torch.tensor([x], dtype=torch.float32).cuda()  # noqa: E731
    positions = c["positions"][0] if c["positions"].shape[0] == 1 else c["positions"]
    return M.nvfp4_rope_append(q if with_q else None, k, v, positions, c["cos_sin"], c["slots"], c["kp"], c["ks"], c["vp"],
                               c["vs"], pair_axis=c["axis"], interleaved=interleaved, k_gs=scalar(gs[0]), v_gs=scalar(gs[1]),
                               **more)


def check_append(M, c, with_q=True, gs=(None, None), interleaved=False, **more):
    dev = device(c)
    got = call_append(M, dev, with_q, gs, interleaved, **more)
    q, k, v = parts(c)
    want, caches = S.rope_append(q if with_q else None, k, v, c["positions"], c["cos_sin"], c["slots"],
                                 [c[n].numpy() for n in ("kp", "ks", "vp", "vs")], c["axis"], interleaved, *gs)
    if with_q:
        assert torch.equal(host(got).view(torch.int16), want.view(torch.int16))
    else:
        assert got is None
    for name, w in zip(("kp", "ks", "vp", "vs"), caches):
        assert np.array_equal(host(dev[name]).numpy(), w), name


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,kv,dim,rot,axes", [
    (1, 8, 2, 128, 128, 1), (7, 32, 8, 128, 64, 1), (33, 3, 1, 80, 80, 1), (12, 6, 2, 96, 24, 1), (9, 4, 4, 64, 20, 3),
    (40, 7, 7, 16, 10, 1), (11, 2, 1, 512, 512, 2), (64, 14, 2, 128, 128, 3), (5, 1, 1, 256, 2, 1), (300, 20, 5, 112, 56, 2),
    (8, 40, 3, 48, 0, 1), (1030, 2, 2, 64, 64, 1)])
def test_append(M, interleaved, tokens, heads, kv, dim, rot, axes):
    c = append_case(tokens + dim, tokens, heads, kv, dim, rot, axes)
    say("append", tokens, heads, kv, dim, rot, axes, interleaved)
    check_append(M, c, interleaved=interleaved)
    check_append(M, c, interleaved=interleaved, gs=(0.013, 3.7))
    check_append(M, c, with_q=False, interleaved=interleaved, gs=(None, 0.25))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 22])
def test_append_axes_and_positions_outside(M, interleaved, rot):
    """Pairs of an unknown axis and positions outside the table do not turn; a
    table without rows and a cache without slots."""
    say("append outside", interleaved, rot)
    for c in (append_case(1, 20, 4, 2, 64, rot, 2, by_axis=True), append_case(2, 20, 4, 2, 64, rot, 1, by_axis=True)):
        check_append(M, c, interleaved=interleaved)
    c = append_case(3, 20, 4, 2, 64, rot)
    check_append(M, dict(c, cos_sin=c["cos_sin"][:0]), interleaved=interleaved)
    check_append(M, dict(c, kp=c["kp"][:0], ks=c["ks"][:0], vp=c["vp"][:0], vs=c["vs"][:0]), interleaved=interleaved)
    empty = device(append_case(4, 0, 4, 2, 64, rot))
    assert call_append(M, empty, interleaved=interleaved).shape == (0, 4, 64)


def test_append_at_position_zero_is_the_paged_write(M):
    """Angles of zero: the cache's bytes are those of nvfp4_quantize_paged, but for
    the signs of zeros, which a sum with +0 may lose."""
    c = append_case(5, 50, 4, 2, 128, 128)
    c["qkv"][c["qkv"] == 0] = 1.0
    c["positions"].zero_()
    c["cos_sin"][:, :64], c["cos_sin"][:, 64:] = 1.0, 0.0
    dev = device(c)
    say("append at zero")
    q = call_append(M, dev, gs=(0.3, 0.7))
    assert torch.equal(host(q), parts(c)[0])
    for i, (p, s, gs) in enumerate((("kp", "ks", 0.3), ("vp", "vs", 0.7))):
        packed, scales = c[p].cuda(), c[s].cuda()
        M.nvfp4_quantize_paged(parts(dev)[1 + i].flatten(1).contiguous(), dev["slots"], packed, scales,
                               torch.tensor([gs]).cuda())
        assert torch.equal(packed, dev[p]) and torch.equal(scales, dev[s])


def test_append_saturated_and_tiny_blocks(M):
    """Blocks whose scale saturates or is zero, values of subnormal size."""
    c = append_case(6, 30, 2, 2, 64, 32)
    c["qkv"][::3] = (c["qkv"][::3].float() * 2.0 ** 40).to(torch.bfloat16)
    c["qkv"][1::3] = (c["qkv"][1::3].float() * 2.0 ** -120).to(torch.bfloat16)
    say("append saturated")
    for gs in ((None, None), (2.0 ** -20, 1.3), (0.7, 2.0 ** 30)):
        check_append(M, c, gs=gs)
        check_append(M, c, gs=gs, interleaved=True)


def test_append_pitched_rows_and_streams(M):
    c = append_case(7, 37, 4, 2, 128, 96)
    dev = device(c)
    want = host(call_append(M, dev)).clone()
    caches = {n: host(dev[n]).clone() for n in ("kp", "ks", "vp", "vs")}
    dev = device(c)
    wide = torch.full((37, 8, 136), 9.0, dtype=torch.bfloat16).cuda()
    rows = wide.view(37, 8 * 136)
    rows[:, 8:8 + 8 * 128] = dev["qkv"].flatten(1)
    dev["qkv"] = rows[:, 8:8 + 8 * 128].unflatten(1, (8, 128))
    out = torch.full((37, 4 * 128 + 24), 5.0, dtype=torch.bfloat16).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("append pitched, side stream")
    call_append(M, dev, q_out=out[:, 8:8 + 512].unflatten(1, (4, 128)), stream=side)
    side.synchronize()
    assert torch.equal(host(out[:, 8:520]).reshape(37, 4, 128), want)
    assert bool((host(out)[:, :8] == 5.0).all()) and bool((host(out)[:, 520:] == 5.0).all())
    for n, w in caches.items():
        assert torch.equal(host(dev[n]), w), n
    with pytest.raises(M.Nvfp4Error):
        call_append(M, dev, q_out=parts(dev)[0])          # over q


# ---- requests --------------------------------------------------------------------
def request_case(seed, kv, dim, page, totals, news, hide=(), pad=0, width=None, heads=None, spare=3):
    """Random caches and keys, pages in random order; `hide`: (request, column,
    entry) replacements in the table; `pad` rows of q before and after."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-max(t, 0) // page) for t in totals]
    width = max(need + [1]) + 1 if width is None else width
    pages = sum(need) + spare
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table, used = torch.full((len(totals), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :min(n, width)] = order[used:used + n][:width]
        used += n
    for b, col, entry in hide:
        table[b, col] = entry
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(news)]) + pad, dtype=torch.int32)
    c = dict(table=table, lens=torch.tensor(totals, dtype=torch.int32), offsets=offsets, page=page, scale=0.3 / math.sqrt(dim),
             most=max(list(news) + [0]))
    c["kp"], c["ks"] = R.random_nvfp4(g, pages * page, kv * dim)
    c["vp"], c["vs"] = R.random_nvfp4(g, pages * page, kv * dim)
    c["keys"] = torch.randint(-127, 128, (pages, kv, dim), generator=g, dtype=torch.int8)
    c["exponents"] = torch.randint(0, 6, (pages, kv), generator=g, dtype=torch.int8)
    if heads:
        c["q"] = torch.randn(int(offsets[-1]) + pad, heads, dim, generator=g).to(torch.bfloat16)
    return c


# ---- page keys -------------------------------------------------------------------
def check_keys(M, c, hint=None):
    dev = device(c)
    got = M.nvfp4_page_keys(dev["kp"], dev["ks"], dev["table"], dev["lens"], dev["offsets"], dev["keys"], dev["exponents"],
                            page_size=c["page"], max_query_len=c["most"] if hint is None else hint)
    assert got[0] is dev["keys"] and got[1] is dev["exponents"]
    keys, exponents, other = S.page_keys(c["kp"], c["ks"], c["table"], c["lens"], c["offsets"], c["keys"], c["exponents"],
                                         c["page"])
    assert torch.equal(host(got[1]), exponents)
    assert bool(((host(got[0]) == keys) | (host(got[0]) == other)).all())


@pytest.mark.parametrize("kv,dim,page", [(1, 64, 16), (2, 128, 16), (8, 128, 64), (3, 256, 24), (5, 64, 1), (20, 64, 7),
                                         (1, 256, 130), (9, 128, 33), (40, 128, 5)])
def test_page_keys(M, kv, dim, page):
    """Steps that complete no page, one, several; whole prompts; ragged ends."""
    totals = [page, page - 1, 3 * page, 3 * page + 1, 0, 2 * page, 5 * page - 1, 1]
    news = [1, 1, 1, 2, 0, 2 * page, 4 * page, 1]
    say("page keys", kv, dim, page)
    check_keys(M, request_case(kv + page, kv, dim, page, totals, news))


def test_page_keys_hints_hidden_pages_and_odd_requests(M):
    """Hints below and far above the new tokens; hidden pages; negative and too
    long lengths; more new tokens than the length; rows in front of the first request."""
    c = request_case(3, 2, 64, 8, [64, 50, -4, 24, 30], [64, 20, 3, 40, 5], hide=[(0, 2, -1), (0, 5, 10 ** 9), (1, 4, -2 ** 31)],
                     pad=4, width=7)
    for hint in (0, 1, 9, 64, 10 ** 6, 2 ** 62):
        say("page keys hint", hint)
        check_keys(M, c, hint)
    say("page keys without cache, table or request")
    none = request_case(4, 2, 64, 8, [], [])
    check_keys(M, none, 1)
    check_keys(M, dict(c, table=c["table"][:, :0]), 1)


def test_page_keys_extremes(M):
    """The largest and smallest values in every place, sums that cancel, zeros."""
    page = 64
    c = request_case(5, 2, 128, page, [4 * page], [4 * page], spare=0)
    kp, ks = c["kp"].view(4, page, -1), c["ks"].view(4, page, -1)
    kp[0], ks[0] = 0x77, 0x7e                # all 6 * 448
    kp[1], ks[1] = 0x11, 0x01                # all 0.5 / 512: the smallest value
    kp[2, ::2], kp[2, 1::2], ks[2] = 0x7f, 0xf7, 0x7e       # +6 and -6 in turn: zero sums but for none
    kp[3], ks[3] = 0x77, 0x7e
    kp[3, 0, 0], ks[3, 0, 0] = 0x17, 0x7d
    say("page keys extremes")
    check_keys(M, c)


# ---- selection -------------------------------------------------------------------
def check_select(M, c, top, first, local, **more):
    dev = device(c)
    out = torch.full((c["q"].shape[0], c["keys"].shape[1], first + top + local), -7, dtype=torch.int32).cuda()
    got = M.nvfp4_select_pages(dev["q"], dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"],
                               page_size=c["page"], top_k=top, first=first, local=local, pages=out, **more)
    want = S.select_pages(c["q"], c["keys"], c["exponents"], c["table"], c["lens"], c["offsets"], c["page"], top, first, local)
    assert got is out and torch.equal(host(out), want), (host(out) != want).nonzero()[:5]


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (3, 3, 64, 4), (12, 1, 256, 8), (14, 2, 64, 1), (96, 1, 128, 2),
                                               (20, 5, 128, 3), (64, 8, 128, 16)])
def test_select(M, heads, kv, dim, page):
    """Contexts from one token to hundreds of pages, several tokens a request, lists
    longer and shorter than the pages there are."""
    totals = [1, page, page + 1, 5 * page, 17 * page + 1, 70 * page - 1, 300 * page]
    news = [1, 1, 2, 1, 3, 1, 2]
    c = request_case(heads + dim, kv, dim, page, totals, news, heads=heads, pad=2)
    for top, first, local in ((4, 1, 2), (0, 0, 1), (16, 0, 1), (7, 3, 4), (100, 1, 1), (1, 0, 1), (64, 2, 3)):
        say("select", heads, kv, dim, page, top, first, local)
        check_select(M, c, top, first, local)


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (3, 3, 64, 4), (12, 1, 256, 8), (14, 2, 64, 1), (40, 1, 128, 2),
                                               (20, 4, 256, 3), (64, 1, 64, 5), (200, 1, 128, 4)])
def test_select_tokens_of_a_chunk(M, heads, kv, dim, page):
    """Chunks of tokens, which a workgroup takes some of at a time; requests that end
    inside them."""
    totals, news = [200 * page, 9 * page + 3, 5, 70 * page + 1], [37, 6, 5, 21]
    c = request_case(heads + dim, kv, dim, page, totals, news, heads=heads, pad=3)
    for top, first, local in ((4, 1, 2), (0, 0, 1), (30, 2, 3), (300, 0, 1)):
        say("select chunk", heads, kv, dim, page, top, first, local)
        check_select(M, c, top, first, local)


@pytest.mark.parametrize("news", [1, 9])
@pytest.mark.parametrize("octaves", [0, 30, 64])
def test_select_scores_of_any_spread(M, news, octaves):
    """Exponents up to the largest, one score far above the others, long lists."""
    c = request_case(11, 2, 64, 2, [1400, 900], [news, news], heads=4)
    c["exponents"] = torch.randint(0, octaves + 1, c["exponents"].shape, dtype=torch.int8, generator=torch.Generator().manual_seed(1))
    c["keys"][5:9], c["exponents"][5:9] = 127, 64
    for top in (1, 7, 120, 600):
        say("select spread", news, octaves, top)
        check_select(M, c, top, 1, 2)


@pytest.mark.parametrize("news", [[1, 1], [2, 1], [9, 11]])
@pytest.mark.parametrize("spread", ["one value", "few values", "zero queries"])
def test_select_ties_go_to_the_lower_page(M, spread, news):
    c = request_case(7, 2, 64, 4, [1200, 900], news, heads=4)
    g = torch.Generator().manual_seed(1)
    if spread == "one value":
        c["keys"][:], c["exponents"][:] = 3, 1
    elif spread == "few values":
        c["keys"][:] = 0
        c["keys"][..., 0] = torch.randint(-1, 2, c["keys"].shape[:2], generator=g, dtype=torch.int8)
        c["exponents"][:] = 0
    else:
        c["q"][:] = 0
    say("select ties", spread)
    for top, first, local in ((10, 1, 2), (200, 0, 1), (33, 0, 5)):
        check_select(M, c, top, first, local)


def test_select_rows_and_pages_that_do_not_count(M):
    """Empty contexts, negative lengths, queries before the context, hidden pages, a
    request all of whose pages are hidden, a table narrower than the length."""
    totals, news = [0, -5, 3, 400, 80, 33], [1, 2, 6, 3, 1, 33]
    hide = [(3, j, -1) for j in range(0, 50, 3)] + [(3, 4, 10 ** 9), (3, 7, -2 ** 31)] + [(4, j, -1) for j in range(10)]
    c = request_case(8, 2, 128, 8, totals, news, hide=hide, heads=4, pad=1)
    say("select hidden")
    for top, first, local in ((5, 1, 2), (40, 0, 1), (100, 4, 4)):
        check_select(M, c, top, first, local)
    c["table"] = c["table"][:, :20].contiguous()
    say("select narrow table")
    check_select(M, c, 5, 1, 2)
    say("select without cache or table")
    for d in (dict(c, keys=c["keys"][:0], exponents=c["exponents"][:0]), dict(c, table=c["table"][:, :0])):
        check_select(M, d, 5, 1, 2)


@pytest.mark.parametrize("power", [100, -126, -40])
def test_select_queries_of_any_size(M, power):
    """q near both ends of BF16's range: its scale is a power of two and exact."""
    c = request_case(9, 2, 64, 4, [300, 40], [1, 2], heads=6)
    c["q"] = (c["q"].double() * 2.0 ** power).to(torch.bfloat16)
    say("select sizes", power)
    check_select(M, c, 9, 1, 1)


def test_select_the_longest_table(M):
    """32768 pages a request, the most that is taken."""
    n = 32768
    c = request_case(10, 1, 64, 1, [n, 20000], [1, 1], heads=1, width=n)
    say("select longest table")
    check_select(M, c, 50, 1, 2)
    check_select(M, c, 2045, 1, 2)


def test_select_the_longest_table_for_many_tokens(M):
    """As many tokens as go to workgroups that keep all scores in LDS, with tables of
    the most pages and queries of the largest head."""
    n = 32768
    c = request_case(10, 8, 256, 1, [n, 60], [2, 98], heads=8, width=n)
    say("select longest table, many tokens")
    assert M.sparse.raw().nvfp4_select_pages_workspace(100, 8, 8, 2, n) == 0
    check_select(M, c, 50, 1, 2)


@pytest.mark.parametrize("news", [[1, 1, 1], [40, 30, 2]])
def test_select_queries_that_are_not_finite(M, news):
    """A token with such a query gets a valid list; the others' are what they were."""
    c = request_case(17, 2, 128, 4, [600, 333, 90], news, heads=8)
    top, first, local = 20, 1, 2
    bad = c["offsets"][1].item()
    q = c["q"].clone()
    q[bad, 1, 3], q[bad, 6, 100] = math.nan, -math.inf
    say("select not finite", news)

    def run(q):
        dev = device(dict(c, q=q))
        return host(M.nvfp4_select_pages(dev["q"], dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"],
                                         page_size=4, top_k=top, first=first, local=local))
    want, got = run(c["q"]), run(q)
    others = torch.arange(len(q)) != bad
    assert torch.equal(got[others], want[others])
    own = (333 - news[1]) // 4
    for h in range(2):
        p = got[bad, h]
        n = int((p >= 0).sum())
        assert bool((p[n:] == -1).all()) and bool((p[1:n] > p[:n - 1]).all()) and p[n - 1] == own
        assert p[0] == 0 and p[n - 2] == own - 1 and n <= top + first + local


# ---- attention -------------------------------------------------------------------
def lists(c, kv, n, seed, wild=False):
    """Random pages for each token and head, some repeated, some that show nothing."""
    g = torch.Generator().manual_seed(seed)
    tokens, width = c["q"].shape[0], c["table"].shape[1]
    p = torch.randint(0, max(width, 1), (tokens, kv, n), generator=g, dtype=torch.int32)
    p[torch.rand(p.shape, generator=g) < 0.15] = -1
    if wild:
        p[torch.rand(p.shape, generator=g) < 0.1] = width
        p[torch.rand(p.shape, generator=g) < 0.05] = 2 ** 31 - 1
        p[torch.rand(p.shape, generator=g) < 0.05] = -2 ** 31
    for t, b, pos in S.requests(tokens, c["table"], c["lens"], c["offsets"], c["page"]):
        if n and t % 3 and pos >= 0:
            p[t, :, n // 2] = pos // c["page"]        # the token's own page, in part
    return p


def call_sparse(M, c, dev, pages, out=None, lse=True, **more):
    return M.nvfp4_sparse_attention(dev["q"], dev["kp"], dev["ks"], dev["vp"], dev["vs"], dev["table"], dev["lens"],
                                    dev["offsets"], pages, page_size=c["page"], scale=c["scale"], out=out, lse=lse, **more)


def check_sparse(M, c, pages, gs=None, **more):
    dev = device(c)
    k_gs, v_gs = (1.0, 1.0) if gs is None else gs
    scalar = lambda v: None if gs is None else torch.tensor([v], dtype=torch.float32).cuda()  # noqa: E731
    out = torch.full_like(dev["q"], 7.0)
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    call_sparse(M, c, dev, pages.cuda(), out, lse, k_gs=scalar(k_gs), v_gs=scalar(v_gs), **more)
    ref, ref_lse, tol, lse_tol = S.sparse_attention(c["q"], c["kp"], c["ks"], c["vp"], c["vs"], c["table"], c["lens"],
                                                    c["offsets"], pages, c["page"], c["scale"], k_gs, v_gs)
    got, got_lse = host(out).double(), host(lse).double()
    mine = ~torch.isnan(ref_lse[:, 0])
    assert bool((got[~mine] == 7.0).all()) and bool((got_lse[~mine] == 7.0).all())       # rows of no request
    empty = mine[:, None] & torch.isinf(ref_lse)
    assert torch.equal(torch.isinf(got_lse), torch.isinf(ref_lse)) and bool((got[empty] == 0).all())
    seen = mine[:, None] & ~torch.isinf(ref_lse)
    worst = ((got - ref).abs() - tol)[seen]
    assert worst.numel() == 0 or worst.max() <= 0, (worst.max(), (got - ref).abs()[seen].max())
    z = ((got_lse - ref_lse).abs() - lse_tol)[seen]
    assert z.numel() == 0 or z.max() <= 0, z.max()


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (4, 4, 64, 32), (14, 2, 64, 7), (48, 1, 128, 1), (12, 4, 256, 24),
                                               (7, 7, 128, 5), (40, 1, 256, 16), (20, 1, 128, 16), (60, 1, 64, 48),
                                               (100, 1, 128, 16), (20, 5, 256, 64)])
def test_sparse_attention(M, heads, kv, dim, page):
    totals, news = [1, 2, page, 3 * page + 5, 20 * page, 11 * page - 1], [1, 2, 1, 3, 1, 2]
    c = request_case(heads + dim + page, kv, dim, page, totals, news, heads=heads, pad=2)
    for n in (1, 5, 40):
        say("sparse", heads, kv, dim, page, n)
        check_sparse(M, c, lists(c, kv, n, n), gs=(0.7, 1.9))
        check_sparse(M, c, lists(c, kv, n, n + 1, wild=True))


@pytest.mark.parametrize("heads,kv,dim,page,n", [(8, 2, 128, 16, 300), (4, 1, 64, 64, 70), (4, 2, 256, 24, 100), (2, 1, 128, 1, 2048)])
def test_sparse_attention_split(M, heads, kv, dim, page, n):
    """Few tokens with long lists: a list is split over workgroups."""
    c = request_case(dim, kv, dim, page, [20 * page + 3, 9], [1, 1], heads=heads)
    say("sparse split", heads, kv, dim, page, n)
    check_sparse(M, c, lists(c, kv, n, 5))


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 128, 16), (4, 4, 64, 32), (8, 8, 128, 6), (16, 2, 128, 32), (15, 3, 256, 16),
                                               (5, 5, 256, 7), (12, 1, 64, 64), (3, 1, 64, 1)])
@pytest.mark.parametrize("n", [3, 20])
def test_sparse_attention_tokens_that_share_pages(M, heads, kv, dim, page, n):
    """Chunks of tokens, whose lists are joined: pages that some, all or one of them
    list, in any order; requests that end inside a group of tokens; lists with a
    page listed twice among the others; entries that show nothing."""
    totals, news = [40 * page, 9 * page + 3, 5, 25 * page + 1], [37, 6, 5, 21]
    c = request_case(heads + dim + page, kv, dim, page, totals, news, heads=heads, pad=3)
    g = torch.Generator().manual_seed(n)
    tokens, width = c["q"].shape[0], c["table"].shape[1]
    common = torch.rand(1, kv, width, generator=g)
    p = (common + 0.5 * torch.rand(tokens, kv, width, generator=g)).argsort(-1)[..., :n].int().contiguous()
    p[torch.rand(p.shape, generator=g) < 0.1] = -1
    say("sparse chunks", heads, kv, dim, page, n)
    check_sparse(M, c, p, gs=(0.7, 1.9))
    p[9, :, 1], p[20, 0, 2], p[50, -1, 0] = p[9, :, 0], p[20, 0, 0], p[50, -1, 1]
    p[30:33] = lists(c, kv, n, 4, wild=True)[30:33]
    check_sparse(M, c, p)


@pytest.mark.parametrize("heads,dim,page", [(40, 64, 16), (64, 64, 5), (70, 64, 32), (40, 128, 16)])
def test_sparse_attention_many_tokens_with_many_rows(M, heads, dim, page):
    """Enough tokens of more than 32 heads on one that a workgroup takes all of them."""
    c = request_case(heads + dim + page, 1, dim, page, [20 * page, 400, 140], [200, 300, 40], heads=heads, pad=1)
    say("sparse many rows", heads, dim, page)
    check_sparse(M, c, lists(c, 1, 5, 1), gs=(0.7, 1.9))
    check_sparse(M, c, lists(c, 1, 9, 2, wild=True))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sparse_attention_rows_that_see_nothing(M, dim):
    """Empty contexts, queries before the context, hidden pages, empty lists, lists of
    later pages alone, a list without room."""
    totals, news = [0, -5, 3, 40, 80, 33], [1, 2, 6, 1, 3, 4]
    hide = [(3, 1, -1), (4, 0, 10 ** 9), (4, 2, -2 ** 31), (5, 0, -1), (5, 1, 2 ** 31 - 1), (5, 2, 500)]
    c = request_case(dim, 2, dim, 16, totals, news, hide=hide, heads=8, pad=1)
    p = lists(c, 2, 7, 3)
    p[10], p[11, 0], p[12, 1] = -1, 4, -1
    say("sparse hidden", dim)
    check_sparse(M, c, p)
    check_sparse(M, c, p[..., :0].contiguous())
    say("sparse without cache or table", dim)
    none = {k: c[k][:0] for k in ("kp", "ks", "vp", "vs")}
    for d in (dict(c, **none), dict(c, table=c["table"][:, :0])):
        out, lse = call_sparse(M, d, device(d), p.cuda())
        assert bool((host(out)[1:-1] == 0).all()) and bool((host(lse)[1:-1] == -math.inf).all())


def test_sparse_attention_over_all_pages_is_attention(M):
    """A list of all pages in order: the results of nvfp4_paged_attention, within
    both calls' bounds."""
    c = request_case(2, 2, 128, 16, [300, 41, 1], [2, 1, 1], heads=8)
    every = torch.arange(c["table"].shape[1], dtype=torch.int32).expand(4, 2, -1).contiguous()
    dev = device(c)
    say("sparse over everything")
    out, lse = call_sparse(M, c, dev, every.cuda())
    want, want_lse = M.nvfp4_paged_attention(dev["q"], dev["kp"], dev["ks"], dev["vp"], dev["vs"], dev["table"], dev["lens"],
                                             dev["offsets"], kv_heads=2, page_size=16, max_query_len=2, scale=c["scale"], lse=True)
    _, _, tol, lse_tol = S.sparse_attention(c["q"], c["kp"], c["ks"], c["vp"], c["vs"], c["table"], c["lens"], c["offsets"],
                                            every, 16, c["scale"])
    assert bool(((host(out).double() - host(want).double()).abs() <= 2 * tol).all())
    assert bool(((host(lse).double() - host(want_lse).double()).abs() <= 2 * lse_tol).all())


@pytest.mark.parametrize("page", [16, 10])
def test_sparse_attention_unseen_slots_may_hold_anything(M, page):
    """Slots behind the token, of hidden pages and of pages not listed: NaN scales
    and any code there change no byte of the result."""
    c = request_case(15, 2, 128, page, [200, 37, 111], [1, 1, 2], hide=[(0, 1, -1), (2, 0, 10 ** 7)], heads=8)
    p = lists(c, 2, 6, 2)
    say("sparse unseen slots", page)
    want = [host(x).clone() for x in call_sparse(M, c, device(c), p.cuda())]
    mine = torch.zeros(c["kp"].shape[0], dtype=torch.bool)
    for t, b, pos in S.requests(4, c["table"], c["lens"], c["offsets"], page):
        for j in set(p[t].flatten().tolist()):
            entry = int(c["table"][b, j]) if j >= 0 else -1
            if 0 <= entry < len(mine) // page:
                mine[entry * page: entry * page + max(0, min(page, pos + 1 - j * page))] = True
    for k, v in (("kp", 0xff), ("ks", 0x7f), ("vp", 0x77), ("vs", 0xff)):
        c[k] = c[k].clone()
        c[k][~mine] = v
    got = call_sparse(M, c, device(c), p.cuda())
    assert torch.equal(host(got[0]), want[0]) and torch.equal(host(got[1]), want[1])


@pytest.mark.parametrize("news", [[1, 1], [6, 5]])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (256, 32), (64, 3), (128, 10), (256, 9)])
def test_sparse_attention_nan_is_not_hidden(M, dim, page, news):
    """A NaN in a query, or in a key or value that a row sees, reaches that row's
    output; rows that do not see it keep their bytes."""
    c = request_case(16, 2, dim, page, [20 * page, 7 * page + 3], news, heads=4)
    tokens = sum(news)
    p = torch.arange(5, dtype=torch.int32).expand(tokens, 2, 5).contiguous()
    p[0, :, 2] = 9                                    # the only one that lists page 9 of request 0, and not 2
    dev = device(c)
    say("sparse NaN", dim, page, news)
    want, want_lse = [host(x).clone() for x in call_sparse(M, c, dev, p.cuda())]
    assert not bool(torch.isnan(want.float()).any())
    q = c["q"].clone()
    q[1, 3, 47] = math.nan
    out, lse = [host(x) for x in call_sparse(M, c, device(dict(c, q=q)), p.cuda())]
    hit = torch.zeros(tokens, 4, dtype=torch.bool)
    hit[1, 3] = True
    assert bool(torch.isnan(out[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    slot = int(c["table"][0, 9]) * page + page - 1
    hit = torch.zeros(tokens, 4, dtype=torch.bool)
    hit[0, :2] = True                                 # key/value head 0's
    d = device(c)
    d["ks"][slot, 2] = 0xff
    out, lse = [host(x) for x in call_sparse(M, c, d, p.cuda())]
    assert bool(torch.isnan(out[hit].float()).all()) and bool(torch.isnan(lse[hit]).all())
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])
    for block in range(dim // 16):                    # 16 dimensions of the value: those alone
        d = device(c)
        d["vs"][slot, block] = 0x7f if block % 2 else 0xff
        out, lse = [host(x) for x in call_sparse(M, c, d, p.cuda())]
        nan = torch.zeros(out.shape, dtype=torch.bool)
        nan[0, :2, 16 * block:16 * block + 16] = True
        assert torch.equal(torch.isnan(out.float()), nan), block
        assert torch.equal(out[~nan], want[~nan]) and torch.equal(lse, want_lse), block


# ---- together --------------------------------------------------------------------
@pytest.mark.parametrize("page", [2, 16])
def test_pages_far_into_a_large_cache(M, page):
    """The last pages of caches of 5 GB (offsets beyond 32 bits) give what the same
    pages give in a small cache."""
    kv, dim, heads, slots = 32, 256, 32, 1200 * 1024
    c = request_case(18, kv, dim, page, [40 * page + 1, 9 * page], [1, 3], heads=heads)
    small = c["kp"].shape[0] // page
    shift = slots // page - small
    far = dict(c, table=torch.where(c["table"] >= 0, c["table"] + shift, c["table"]))
    a, b = device(c), device(far)
    say("far pages", page)
    for n in ("kp", "ks", "vp", "vs", "keys", "exponents"):
        rows = slots if n in ("kp", "ks", "vp", "vs") else slots // page
        big = torch.zeros((rows, *c[n].shape[1:]), dtype=c[n].dtype, device="cuda")
        big[rows - c[n].shape[0]:] = a[n]
        b[n] = big
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(4, kv, dim, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    positions = torch.tensor([5, 1, 2, 3], dtype=torch.int32).cuda()
    cos_sin = torch.randn(8, dim, generator=g).cuda()
    got = []
    for d, base in ((a, 0), (b, shift * page)):
        own = torch.tensor([int(c["table"][0, 40]) * page] + [int(c["table"][1, i // page]) * page + i % page
                                                              for i in range(9 * page - 3, 9 * page)]) + base
        q = M.nvfp4_rope_append(d["q"], k, v, positions, cos_sin, own.cuda(), d["kp"], d["ks"], d["vp"], d["vs"])
        M.nvfp4_page_keys(d["kp"], d["ks"], d["table"], d["lens"], torch.tensor([0, 40 * page, 49 * page], dtype=torch.int32).cuda(),
                          d["keys"], d["exponents"], page_size=page, max_query_len=40 * page)
        pages = M.nvfp4_select_pages(q, d["keys"], d["exponents"], d["table"], d["lens"], d["offsets"], page_size=page, top_k=6)
        out, lse = M.nvfp4_sparse_attention(q, d["kp"], d["ks"], d["vp"], d["vs"], d["table"], d["lens"], d["offsets"], pages,
                                            page_size=page, scale=c["scale"], lse=True)
        tail = [d[n][len(d[n]) - len(c[n]):] for n in ("kp", "ks", "vp", "vs", "keys", "exponents")]
        got.append([host(x).clone() for x in (q, pages, out, lse, *tail)])
        if base:
            assert not bool(d["kp"][:base].any()) and not bool(d["keys"][:shift].any())
    for i, (x, y) in enumerate(zip(*got)):
        assert torch.equal(x, y), i


def test_steps_on_two_streams(M):
    """Two steps that may run at the same time, with caches and workspaces of their own."""
    want = []
    for seed in (3, 4):
        s = step_state(seed)
        first_keys(M, s)
        want.append({k: host(v).clone() for k, v in one_step(M, s).items()})
    states = [step_state(seed) for seed in (3, 4)]
    for s in states:
        first_keys(M, s)
    torch.cuda.synchronize()
    say("two streams")
    streams, got = [torch.cuda.Stream() for _ in states], [None, None]
    for _ in range(3):
        for i, s in enumerate(states):
            with torch.cuda.stream(streams[i]):
                s["table"].copy_(step_state(3 + i)["table"])
                got[i] = one_step(M, s)
    torch.cuda.synchronize()
    for i in range(2):
        for k, v in got[i].items():
            assert torch.equal(host(v), want[i][k]), (i, k)


def test_sparse_refusals(M):
    """What the binding and the library refuse, with tensors of every operator; nothing
    is launched, nothing written."""
    c = request_case(19, 2, 128, 16, [70, 33], [1, 2], heads=8)
    d = device(c)
    pages = torch.zeros(3, 2, 4, dtype=torch.int32).cuda()
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16).cuda()
    positions, slots = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(3, dtype=torch.int64).cuda()
    cos_sin = torch.zeros(9, 128).cuda()
    before = {n: host(v).clone() for n, v in d.items() if isinstance(v, torch.Tensor)}
    refused = (TypeError, ValueError, M.Nvfp4Error)

    def append(q=d["q"], k=k, v=k, p=positions, t=cos_sin, s=slots, kp=d["kp"], ks=d["ks"], vp=d["vp"], vs=d["vs"], **more):
        M.nvfp4_rope_append(q, k, v, p, t, s, kp, ks, vp, vs, **more)

    def keys(kp=d["kp"], ks=d["ks"], t=d["table"], n=d["lens"], o=d["offsets"], keys=d["keys"], e=d["exponents"], page=16, most=2):
        M.nvfp4_page_keys(kp, ks, t, n, o, keys, e, page_size=page, max_query_len=most)

    def select(q=d["q"], keys=d["keys"], e=d["exponents"], t=d["table"], n=d["lens"], o=d["offsets"], page=16, top=4, **more):
        M.nvfp4_select_pages(q, keys, e, t, n, o, page_size=page, top_k=top, **more)

    def sparse(q=d["q"], kp=d["kp"], ks=d["ks"], vp=d["vp"], vs=d["vs"], t=d["table"], n=d["lens"], o=d["offsets"], p=pages,
               page=16, **more):
        M.nvfp4_sparse_attention(q, kp, ks, vp, vs, t, n, o, p, page_size=page, **more)

    wide = torch.zeros(3, 8, 256, dtype=torch.bfloat16).cuda()
    bad = [(append, x) for x in (
        dict(q=d["q"].float()), dict(q=d["q"].cpu()), dict(q=d["q"][:2]), dict(q=d["q"][:, :0]), dict(q=wide[:, :, ::2]), dict(k=k.cpu()),
        dict(k=k[0]), dict(v=k[:, :1]), dict(p=positions.long()), dict(p=positions[:2]), dict(p=positions.cpu()),
        dict(p=torch.zeros(3, 2, dtype=torch.int32).cuda().t()), dict(p=torch.zeros(3, dtype=torch.int32).cuda().expand(2, 3)),
        dict(t=cos_sin.double()), dict(t=cos_sin[:, :127]), dict(t=cos_sin[:, :64]), dict(t=torch.zeros(9, 256).cuda()),
        dict(t=cos_sin[0]), dict(s=slots.int()), dict(s=slots[:2]), dict(kp=d["kp"][:, :64]), dict(ks=d["ks"][:9]),
        dict(vp=d["vp"].view(torch.int8)), dict(vs=d["ks"].cpu()), dict(vp=d["kp"]), dict(vs=d["ks"]),
        dict(pair_axis=torch.zeros(63, dtype=torch.int32).cuda()), dict(pair_axis=torch.zeros(64).cuda()),
        dict(k_gs=torch.zeros(2).cuda()), dict(v_gs=torch.ones(1)), dict(q_out=d["q"]), dict(q_out=d["q"][:2]),
        dict(q=None, q_out=d["q"]), dict(q=wide[:, :, :128]), dict(p=torch.zeros(17, 3, dtype=torch.int32).cuda()),
        dict(kp=d["kp"][0], ks=d["ks"][0]))]
    bad += [(keys, x) for x in (
        dict(kp=d["kp"].cpu()), dict(kp=d["kp"][:32]), dict(ks=d["ks"].float()), dict(t=d["table"].long()), dict(t=d["table"][:1]),
        dict(t=d["table"].t()), dict(n=d["lens"].long()), dict(o=d["offsets"][:2]), dict(keys=d["keys"].float()),
        dict(keys=d["keys"][:, :, :64]), dict(keys=d["keys"][:1]), dict(e=d["exponents"][:, :1]), dict(e=d["exponents"].int()),
        dict(page=0), dict(page=8), dict(page=-16), dict(page=2 ** 31), dict(page=2 ** 63), dict(most=-1), dict(page=16.0),
        dict(n=d["lens"].cpu()), dict(o=d["offsets"].cpu()))]
    bad += [(select, x) for x in (
        dict(q=d["q"].half()), dict(q=d["q"][0]), dict(q=d["q"][:, :7]), dict(q=d["q"][:, :, :64]), dict(keys=d["keys"].cpu()),
        dict(e=d["exponents"].float()), dict(t=d["table"].float()), dict(n=d["lens"][:1]), dict(o=d["offsets"].long()), dict(page=0),
        dict(top=-1), dict(top=2046), dict(top=2 ** 40), dict(first=-1), dict(first=2 ** 64), dict(local=0), dict(local=2047),
        dict(pages=pages), dict(pages=torch.zeros(3, 2, 7).cuda()), dict(top=4.0), dict(q=wide[:, :, ::2]),
        dict(workspace=torch.empty(8, dtype=torch.uint8).cuda()), dict(t=torch.zeros(2, 32769, dtype=torch.int32).cuda()),
        dict(page=2 ** 29))]
    bad += [(sparse, x) for x in (
        dict(q=d["q"].float()), dict(q=d["q"][:2]), dict(q=d["q"][:, :7]), dict(q=wide[:, :, ::2]), dict(p=pages.long()), dict(p=pages[:2]),
        dict(p=pages[0]), dict(p=pages[:, :1]), dict(p=pages.cpu()), dict(p=pages[:, :, ::2]),
        dict(p=torch.zeros(3, 2, 2049, dtype=torch.int32).cuda()), dict(page=0), dict(page=7), dict(page=2 ** 31), dict(page=2 ** 40),
        dict(t=d["table"].cpu()), dict(n=d["lens"].float()), dict(o=d["offsets"][1:]), dict(kp=d["kp"][:, :8]), dict(vs=d["vs"][1:]),
        dict(ks=d["ks"].int()), dict(scale=math.nan), dict(scale=math.inf), dict(k_gs=torch.zeros(3).cuda()), dict(out=d["q"][:2]),
        dict(out=d["q"].float()), dict(lse=torch.zeros(3, 7).cuda()), dict(lse=torch.zeros(3, 8).half().cuda()),
        dict(p=pages[:, :0]),
        dict(p=torch.zeros(3, 2, 400, dtype=torch.int32).cuda(), workspace=torch.empty(64, dtype=torch.uint8).cuda()))]
    for call in (append, keys, select, sparse):           # what the others change is all that is wrong
        say("taken", call.__name__)
        if call is not append:
            call()
    for name in before:
        d[name].copy_(before[name])
    for call, change in bad:
        say("refused", call.__name__, {n: tuple(v.shape) if isinstance(v, torch.Tensor) else v for n, v in change.items()})
        with pytest.raises((*refused, C.ArgumentError)):
            call(**change)
    for n, v in before.items():
        assert torch.equal(host(d[n]), v), n


@pytest.mark.parametrize("offsets", [[0, 30, 12, 40], [5, 5, 5, 5], [40, 30, 20, 10], [-7, 10 ** 9, 20, 2 ** 31 - 1], [0, -2 ** 31, 40, 3]])
def test_offsets_that_fall(M, offsets):
    """Such offsets are no requests; what they give is not specified, but every call
    ends and writes lists of valid pages."""
    c = request_case(20, 2, 64, 16, [100, 300, 555], [10, 20, 10], heads=8)
    dev = device(dict(c, offsets=torch.tensor(offsets, dtype=torch.int32)))
    say("falling offsets", offsets)
    M.nvfp4_page_keys(dev["kp"], dev["ks"], dev["table"], dev["lens"], dev["offsets"], dev["keys"], dev["exponents"], page_size=16,
                      max_query_len=20)
    for n in (40, 3):
        q = dev["q"][:n]
        pages = torch.full((n, 2, 12), -1, dtype=torch.int32).cuda()
        M.nvfp4_select_pages(q, dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"], page_size=16, top_k=9,
                             pages=pages)
        got = host(pages)
        assert bool(((got >= -1) & (got < c["table"].shape[1])).all())
        call_sparse(M, c, dict(dev, q=q), pages)
        torch.cuda.synchronize()


def step_state(seed=3):
    """Six requests over pages of 16, 8/2 heads of 128: caches with pages' keys."""
    g = torch.Generator().manual_seed(seed)
    context, query = [40, 0, 17, 63, 400, 31], [1, 5, 1, 2, 0, 1]
    s = dict(context=torch.tensor(context, dtype=torch.int32).cuda(), query=torch.tensor(query, dtype=torch.int32).cuda())
    table, used = torch.full((6, 30), -1, dtype=torch.int32), 0
    order = torch.randperm(80, generator=g).to(torch.int32)
    for b, n in enumerate(context):
        n = -(-n // 16)
        table[b, :n] = order[used:used + n]
        used += n
    s["table"], s["free"] = table.cuda(), order[used:].contiguous().cuda()
    for n in ("k", "v"):
        p, sc = R.random_nvfp4(g, 80 * 16, 256)
        s[n], s[n + "s"] = p.cuda(), sc.cuda()
    s["keys"] = torch.zeros(80, 2, 128, dtype=torch.int8).cuda()
    s["exponents"] = torch.zeros(80, 2, dtype=torch.int8).cuda()
    s["qkv"] = torch.randn(12, 12, 128, generator=g).to(torch.bfloat16).cuda()
    angle = torch.arange(512).double()[:, None] * 1e4 ** (-torch.arange(64).double() / 64)
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    positions = sum([list(range(c, c + n)) for c, n in zip(context, query)], [])
    s["positions"] = torch.tensor(positions + [0, 0], dtype=torch.int32).cuda()
    return s


def first_keys(M, s):
    """Keys of the pages that the contexts hold."""
    n = s["context"]
    offsets = torch.cat([n.new_zeros(1), torch.cumsum(n, 0).to(torch.int32)])
    M.nvfp4_page_keys(s["k"], s["ks"], s["table"], n, offsets, s["keys"], s["exponents"], page_size=16, max_query_len=400)


def one_step(M, s):
    slots, offsets, lens, end = M.kv_block_tables(s["context"], s["query"], s["table"], 16, 12, free_pages=s["free"])
    qkv = s["qkv"]
    q = M.nvfp4_rope_append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], s["positions"], s["cos_sin"], slots, s["k"], s["ks"], s["v"],
                            s["vs"])
    M.nvfp4_page_keys(s["k"], s["ks"], s["table"], lens, offsets, s["keys"], s["exponents"], page_size=16, max_query_len=5)
    pages = M.nvfp4_select_pages(q, s["keys"], s["exponents"], s["table"], lens, offsets, page_size=16, top_k=5, first=1, local=2)
    o, lse = M.nvfp4_sparse_attention(q, s["k"], s["ks"], s["v"], s["vs"], s["table"], lens, offsets, pages, page_size=16, lse=True)
    return dict(slots=slots, offsets=offsets, lens=lens, end=end, table=s["table"], q=q, k=s["k"], ks=s["ks"], v=s["v"], vs=s["vs"],
                keys=s["keys"], exponents=s["exponents"], pages=pages[:10], o=o[:10], lse=lse[:10])


def test_one_sparse_decoding_step(M):
    """Pages, rotated append, page keys, selection and attention one after the other,
    each against its definition on what the one before left."""
    s = step_state()
    say("one sparse step")
    first_keys(M, s)
    before = {n: host(s[n]).clone() for n in ("k", "ks", "v", "vs", "keys", "exponents")}
    r = {k: host(v).clone() for k, v in one_step(M, s).items()}
    assert r["lens"].tolist() == [41, 5, 18, 65, 400, 32]
    qkv = host(s["qkv"])
    q, caches = S.rope_append(qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], host(s["positions"])[None], host(s["cos_sin"]), r["slots"],
                              [before[n].numpy() for n in ("k", "ks", "v", "vs")])
    assert torch.equal(r["q"], q)
    for n, w in zip(("k", "ks", "v", "vs"), caches):
        assert np.array_equal(r[n].numpy(), w), n
    keys, exponents, other = S.page_keys(r["k"], r["ks"], r["table"], r["lens"], r["offsets"], before["keys"],
                                         before["exponents"], 16)
    assert bool(((r["keys"] == keys) | (r["keys"] == other)).all()) and torch.equal(r["exponents"], exponents)
    pages = S.select_pages(q, r["keys"], exponents, r["table"], r["lens"], r["offsets"], 16, 5, 1, 2)
    assert torch.equal(r["pages"], pages[:10])
    ref, ref_lse, tol, lse_tol = S.sparse_attention(q[:10], r["k"], r["ks"], r["v"], r["vs"], r["table"], r["lens"], r["offsets"],
                                                    r["pages"], 16, 1 / math.sqrt(128))
    assert bool(((r["o"].double() - ref).abs() <= tol).all())
    assert bool(((r["lse"].double() - ref_lse).abs() <= lse_tol).all())


def test_sparse_graph_replays_match_eager(M):
    """The whole step captured into a graph and replayed, with eager steps
    (their own workspaces) and synchronizations in between."""
    s = step_state()
    first_keys(M, s)
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
    state = ("table", "k", "ks", "v", "vs", "keys", "exponents")
    for r in range(4):
        for k, v in captured.items():
            if k not in state:
                v.zero_()
        if r % 2:
            one_step(M, s)
        torch.cuda.synchronize()
        say("sparse graph replay", r)
        graph.replay()
        for k, v in captured.items():
            assert torch.equal(host(v), want[k]), (r, k)


def test_sparse_same_inputs_same_bytes(M):
    c = request_case(12, 2, 128, 16, [3000, 1500, 40], [1, 1, 2], heads=16)
    dev = device(c)
    say("sparse same bytes")

    def both():
        pages = M.nvfp4_select_pages(dev["q"], dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"],
                                     page_size=16, top_k=40)
        return [pages.clone()] + [x.clone() for x in call_sparse(M, c, dev, pages)]
    a = both()
    for r in range(5):
        assert all(torch.equal(x, y) for x, y in zip(a, both())), r
