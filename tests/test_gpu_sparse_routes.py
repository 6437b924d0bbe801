"""The sparse-attention operators on the GPU, path by path: what a workspace held
before a call does not change its result, whatever the offsets; the paths that many
tokens and many requests take, bit for bit; page keys half way between two numbers."""
import numpy as np
import pytest
import torch

import sparse_many_ref as P
from test_gpu_sparse import M, append_case, call_sparse, check_append, device, host, lists, request_case, say  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- what the workspace held -----------------------------------------------------
FALLING = [[0, 30, 12, 40], [40, 30, 20, 10], [-7, 10 ** 9, 20, 2 ** 31 - 1], [0, -2 ** 31, 40, 3], [3, 9, 5, 38]]


def filled(size, kind):
    """A workspace of these bytes: zeros, infinities, NaN, the largest numbers, any bits."""
    words = {"zero": 0, "infinity": 0x7f800000, "nan": 0x7fc00000, "-nan": 0xffc00000, "largest": 0x7f7fffff}
    g = np.random.default_rng(size)
    w = (g.integers(0, 2 ** 32, size // 4, dtype=np.uint64) if kind == "any" else np.full(size // 4, words[kind], np.uint64))
    return torch.from_numpy(w.astype(np.uint32).view(np.uint8)).cuda()


@pytest.mark.parametrize("offsets", [[0, 10, 30, 40]] + FALLING)
def test_select_does_not_read_what_the_workspace_held(M, offsets):
    """Every score that a list is made from was written by the same call."""
    c = request_case(20, 2, 64, 16, [100, 300, 555], [10, 20, 10], heads=8)
    dev = device(dict(c, offsets=torch.tensor(offsets, dtype=torch.int32)))
    say("select, workspaces", offsets)
    for n in (40, 33, 3):
        size = M.sparse.raw().nvfp4_select_pages_workspace(n, 8, 2, 3, c["table"].shape[1])
        assert size > 0
        got = []
        for kind in ("zero", "infinity", "nan", "-nan", "largest", "any"):
            say("select, workspace", n, kind)
            pages = torch.full((n + 2, 2, 12), -7, dtype=torch.int32).cuda()
            M.nvfp4_select_pages(dev["q"][:n], dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"],
                                 page_size=16, top_k=9, pages=pages[1:n + 1], workspace=filled(size, kind))
            got.append(host(pages).clone())
        for p in got[1:]:
            assert torch.equal(p, got[0])
        assert bool((got[0][0] == -7).all()) and bool((got[0][-1] == -7).all())
        assert bool(((got[0] >= -1) & (got[0] < c["table"].shape[1]) | (got[0] == -7)).all())


@pytest.mark.parametrize("offsets", [[0, 10, 30, 40], [2, 10, 30, 37], [0, 30, 10, 35, 40]] + FALLING)
@pytest.mark.parametrize("heads", [8, 80])
def test_sparse_attention_does_not_read_what_the_workspace_held(M, offsets, heads):
    """Every part that a row is joined from was written by the same call; a row whose
    token no workgroup has found a request for keeps its values."""
    more = len(offsets) - 4                     # tokens 10 to 29 of five such offsets are no request's
    c = request_case(20, 2, 64, 16, [100, 300, 555, 60][:3 + more], [10, 20, 5, 5] if more else [10, 20, 10], heads=heads)
    dev = device(dict(c, offsets=torch.tensor(offsets, dtype=torch.int32)))
    say("sparse, workspaces", offsets, heads)
    for n in (40, 33, 3):
        size = M.sparse.raw().nvfp4_sparse_attention_workspace(n, heads, 2, 64, 16, 3 + more, 30)
        assert size > 0
        p = lists(dict(c, q=c["q"][:n]), 2, 30, 5).cuda()
        got = []
        for kind in ("zero", "infinity", "nan", "-nan", "largest", "any"):
            say("sparse, workspace", n, kind)
            out = torch.full((n + 2, heads, 64), 7.0, dtype=torch.bfloat16).cuda()
            lse = torch.full((n + 2, heads), 7.0).cuda()
            call_sparse(M, c, dict(dev, q=dev["q"][:n]), p, out[1:n + 1], lse[1:n + 1], workspace=filled(size, kind))
            got.append((host(out).clone(), host(lse).clone()))
        for out, lse in got:
            assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
            assert not bool(torch.isnan(out.float()).any()) and bool((out[[0, -1]] == 7.0).all()) and bool((lse[[0, -1]] == 7.0).all())
        if more and n > 30:
            none = slice(13, 31)                # 10 and 11 may be taken with 8 and 9
            assert bool((got[0][0][none] == 7.0).all()) and bool((got[0][1][none] == 7.0).all())
            assert not bool((got[0][1][1:11] == 7.0).any())


# ---- many tokens of the rotated append ---------------------------------------------
@pytest.mark.parametrize("heads,kv,dim,rot,inter,layout,together", [
    (16, 8, 128, 128, False, "whole", 1), (32, 8, 128, 128, False, "whole", 2), (28, 4, 128, 128, False, "whole", 4),
    (12, 2, 128, 64, False, "halves of 8", 1), (28, 4, 128, 64, False, "halves of 8", 2), (9, 4, 128, 96, False, "halves of 8", 4),
    (12, 2, 128, 24, False, "halves", 1), (28, 4, 128, 70, False, "halves", 2), (9, 4, 128, 120, False, "halves", 4),
    (12, 2, 128, 128, True, "neighbours", 1), (28, 4, 128, 64, True, "neighbours", 2), (9, 4, 128, 22, True, "neighbours", 4),
    (13, 2, 80, 80, False, "halves of 8", 4), (0, 6, 64, 64, False, "whole", 4), (0, 9, 256, 256, True, "neighbours", 2)])
def test_append_many_tokens(M, heads, kv, dim, rot, inter, layout, together):
    """Threads that take several heads, and heads of several tokens: each pair layout
    with 1, 2 and 4 tokens a workgroup and a last group that is not full; unknown
    axes, positions outside the table and slots outside the cache all over."""
    tokens = 4099
    assert P.append_plan(tokens, heads, kv, dim, rot, inter) == (layout, 1, together)
    say("append many", heads, kv, dim, rot, inter)
    for axes in (1, 3):
        c = append_case(heads + rot + axes, tokens, heads, kv, dim, rot, axes, by_axis=axes > 1)
        g = torch.Generator().manual_seed(axes)
        c["slots"][torch.rand(tokens, generator=g) < 0.1] = -1
        c["positions"][torch.rand(c["positions"].shape, generator=g) < 0.1] = 500
        check_append(M, c, with_q=heads > 0, interleaved=inter, gs=(0.013, 3.7))


# ---- many tokens and many requests of the selection --------------------------------
def pages_case(seed, heads, kv, dim, page, totals, news, pad=0, width=None, ties=False):
    """Requests whose pages have keys alone, in random order, some of them hidden."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-t // page) for t in totals]
    width = max(need) + 1 if width is None else width
    count = sum(need) + 3
    order = torch.randperm(count, generator=g).to(torch.int32)
    table, used = torch.full((len(totals), width), -1, dtype=torch.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = order[used:used + n]
        used += n
    hide = torch.rand(table.shape, generator=g) < 0.05
    table[hide] = torch.tensor([-1, count, 2 ** 31 - 1, -2 ** 31])[torch.randint(0, 4, (int(hide.sum()),), generator=g)].int()
    c = dict(table=table, lens=torch.tensor(totals, dtype=torch.int32), page=page,
             offsets=torch.tensor(np.concatenate([[0], np.cumsum(news)]) + pad, dtype=torch.int32),
             keys=torch.randint(-127, 128, (count, kv, dim), generator=g, dtype=torch.int8),
             exponents=torch.randint(0, 6, (count, kv), generator=g, dtype=torch.int8),
             q=torch.randn(sum(news) + 2 * pad, heads, dim, generator=g).to(torch.bfloat16))
    if ties:
        c["keys"][:] = 0
        c["keys"][..., 0] = torch.randint(-1, 2, (count, kv), generator=g, dtype=torch.int8)
        c["exponents"][:] = 0
    return c


def check_lists(M, c, top, first, local):
    dev = device(c)
    out = torch.full((c["q"].shape[0], c["keys"].shape[1], first + top + local), -7, dtype=torch.int32).cuda()
    M.nvfp4_select_pages(dev["q"], dev["keys"], dev["exponents"], dev["table"], dev["lens"], dev["offsets"], page_size=c["page"],
                         top_k=top, first=first, local=local, pages=out)
    want = P.select_pages(c["q"], c["keys"], c["exponents"], c["table"], c["lens"], c["offsets"], c["page"], top, first, local)
    assert torch.equal(host(out), want), (host(out) != want).nonzero()[:5]


def route(M, c):
    """Tokens of a workgroup, workgroups over a token's pages (0: a workgroup keeps all
    scores), rounds of the longest token's."""
    (tokens, heads, _), kv, (seqs, width) = c["q"].shape, c["keys"].shape[1], c["table"].shape
    together, chunks, size = P.select_plan(tokens, heads, kv, seqs, width)
    assert M.sparse.raw().nvfp4_select_pages_workspace(tokens, heads, kv, seqs, width) == size
    return together, chunks, -(-width // 256) / chunks if chunks else 0


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("heads,kv,dim,page,longest,news,together", [
    (8, 8, 64, 4, 200, [700, 1, 230, 402, 300], 16), (32, 8, 128, 16, 400, [600, 5, 171, 260], 10),
    (28, 4, 128, 3, 60, [900, 2, 333, 517, 40], 9), (16, 8, 256, 2, 500, [450, 260, 99], 8), (64, 8, 64, 1, 1000, [1, 300, 200], 4),
    (6, 3, 128, 5, 256, [3000, 17, 1100, 33], 15)])
def test_select_many_tokens(M, heads, kv, dim, page, longest, news, together, ties):
    """Workgroups that keep the scores of several tokens: requests that end among them,
    tokens in front of the first and behind the last request, hidden pages, ties."""
    totals = [longest * page - 1, 3] + [max(n, longest * page * (i + 2) // 6 + i) for i, n in enumerate(news[2:])]
    totals = [max(t, 1) for t in totals[:len(news)]]
    totals = [min(t, longest * page) for t in totals]
    c = pages_case(heads + dim, heads, kv, dim, page, totals, news, pad=3, ties=ties)
    assert route(M, c) == (together, 0, 0)
    for top, first, local in ((28, 1, 3), (0, 2, 1), (longest, 0, 1), (1, 0, 2)):
        say("select many", heads, kv, dim, page, top, first, local, ties)
        check_lists(M, c, top, first, local)


@pytest.mark.parametrize("heads,kv,dim,news", [(200, 2, 64, [150, 1, 240]), (65, 1, 128, [300, 500]), (1024, 8, 64, [60, 50])])
def test_select_many_tokens_with_many_heads(M, heads, kv, dim, news):
    """More than 64 query rows for a token: the largest score of several rounds of rows."""
    c = pages_case(heads, heads, kv, dim, 4, [280, 5, 190][:len(news)], news, pad=1)
    assert route(M, c) == (1, 0, 0)
    for top, first, local in ((9, 1, 2), (70, 0, 1)):
        say("select many heads", heads, kv, dim, top, first, local)
        check_lists(M, c, top, first, local)


@pytest.mark.parametrize("heads,kv,dim,seqs,longest,news,expected", [
    (64, 8, 128, 64, 1000, 1, (1, 2, 2)), (800, 8, 64, 64, 900, 1, (1, 2, 2)), (8, 8, 64, 60, 4200, 1, (1, 2, 8.5)),
    (40, 8, 64, 30, 1030, 3, (3, 4, 1.25)), (4, 4, 256, 180, 700, 1, (1, 1, 3))])
def test_select_rounds_of_pages(M, heads, kv, dim, seqs, longest, news, expected):
    """Fewer workgroups than parts of 256 pages: each scores several, one after the other."""
    g = np.random.default_rng(seqs)
    totals = [longest] + [int(x) for x in np.exp(g.uniform(np.log(news), np.log(longest), seqs - 1))]
    totals = [max(t, news) for t in totals[:1] + ([longest - 1, longest // 2] + totals[1:])[:seqs - 1]]
    if longest > 4096:
        totals[2:] = [min(t, 600) for t in totals[2:]]
    c = pages_case(heads, heads, kv, dim, 1, totals, [news] * seqs, pad=1 if seqs < 60 else 0, width=longest)
    assert route(M, c) == expected
    for top, first, local in ((57, 1, 6), (1500, 0, 1)):
        say("select rounds", heads, kv, dim, seqs, top, first, local)
        check_lists(M, c, top, first, local)


# ---- page keys half way between two numbers ------------------------------------------
@pytest.mark.parametrize("page", [1, 2, 4, 7, 64])
def test_page_keys_half_way(M, page):
    """One result for each sum: with the device's binary64 2^-e, which is an ulp low for
    some e, a sum half way between two numbers goes to the one nearer 0, else to the
    even one (a product in binary64, rounded half to even, as the plain form has it)."""
    kv, dim, pages = 4, 128, 600 if page < 64 else 200
    g = torch.Generator().manual_seed(page)
    c = request_case(page, kv, dim, page, [pages * page], [pages * page], spare=0)
    # scales of one page and head within an octave or so: its largest sum is not far above the others
    octave = torch.randint(1, 14, (pages, 1, kv, 1), generator=g)
    within = torch.randint(0, 8, (pages, page, kv, dim // 16), generator=g)
    c["ks"] = (8 * octave + within).to(torch.uint8).reshape(pages * page, -1)
    dev = device(c)
    say("page keys half way", page)
    M.nvfp4_page_keys(dev["kp"], dev["ks"], dev["table"], dev["lens"], dev["offsets"], dev["keys"], dev["exponents"], page_size=page,
                      max_query_len=page)
    sums = P.page_sums(c["kp"], c["ks"], torch.arange(pages), kv, dim, page)
    e = P.key_exponents(sums)
    power = host(torch.pow(2.0, -torch.arange(64, dtype=torch.float64, device="cuda")))
    off = (power * torch.ldexp(torch.ones(64, dtype=torch.float64), torch.arange(64)) - 1).abs()
    assert float(off.max()) <= 2.0 ** -52                   # an ulp at most, or the header's two neighbours would not do
    want = (sums.double() * power[e][..., None]).round().clamp(-127, 127)
    assert torch.equal(host(dev["exponents"]).long(), e.long())
    assert torch.equal(host(dev["keys"]).double(), want)
    ties = (e > 0)[..., None] & (sums.abs() % (2 ** e[..., None].long()) == 2 ** (e[..., None].long() - 1).clamp(min=0))
    say("sums half way", int(ties.sum()), "exponents", sorted(set(e[ties.any(-1)].flatten().tolist())))
    assert int(ties.sum()) > 100


# ---- tables with columns that no request needs ---------------------------------------
@pytest.mark.parametrize("news", [[1, 1, 2], [70, 30, 41], [1000, 500, 333]])
def test_tables_wider_than_the_requests(M, news):
    """A wide table, and the columns of it that the longest request needs (rows with a
    pitch), give the same keys, lists and rows as a table without others."""
    kv, dim, page = 2, 64, 4
    c = request_case(31, kv, dim, page, [1203, 900, 350], news, heads=8)
    dev, need = device(c), 301
    assert c["table"].shape[1] == need + 1
    wide = torch.full((3, 5000), -1, dtype=torch.int32).cuda()
    wide[:, :need + 1] = dev["table"]
    wide[:, need:] = 2 ** 31 - 1                 # nobody's
    say("wide tables", news)
    got = []
    for table in (dev["table"][:, :need].contiguous(), wide[:, :need], wide):
        keys, exponents = dev["keys"].clone(), dev["exponents"].clone()
        M.nvfp4_page_keys(dev["kp"], dev["ks"], table, dev["lens"], dev["offsets"], keys, exponents, page_size=page,
                          max_query_len=max(news))
        pages = M.nvfp4_select_pages(dev["q"], keys, exponents, table, dev["lens"], dev["offsets"], page_size=page, top_k=20)
        out, lse = call_sparse(M, c, dict(dev, table=table), pages)
        got.append([host(x).clone() for x in (keys, exponents, pages, out, lse)])
    for other in got[1:]:
        assert all(torch.equal(x, y) for x, y in zip(got[0], other))
    c.update(keys=got[0][0], exponents=got[0][1])
    assert torch.equal(got[0][2], P.select_pages(c["q"], c["keys"], c["exponents"], c["table"], c["lens"], c["offsets"], page, 20, 1, 2))
