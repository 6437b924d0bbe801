"""The decoding-step operators (include/nvfp4_serving.h) on the GPU at the ends
of what their calls take, against the definitions of tests/serving_ref.py."""
import math

import pytest
import torch

import serving_ref as R
import test_gpu_serving as S
from test_gpu_serving import M, attn_case, call_attention, check_attention, device, host, say  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- hints and positions up to the types' ends ----------------------------------
HINTS = (2 ** 30, 2 ** 31 - 301, 2 ** 31 - 1, 2 ** 62)


@pytest.mark.parametrize("hint", HINTS)
def test_attention_prompt_with_the_largest_length_hints(M, hint):
    """Many row blocks (by the hint) leave one split, whose share of the tokens
    is the whole of what the hint promises."""
    c = attn_case(21, 8, 2, 128, 16, [700, 90], [300, 90])
    say("attention prompt, length hint", hint)
    check_attention(M, c, max_query_len=20000, max_seq_len=hint)
    check_attention(M, c, max_query_len=20000, max_seq_len=hint, window=150)
    check_attention(M, c, max_query_len=2 ** 62, max_seq_len=hint, causal=False)
    check_attention(M, c, max_seq_len=hint)          # split


@pytest.mark.parametrize("hint", HINTS)
def test_attention_most_requests_with_the_largest_length_hints(M, hint):
    """So many requests that one split is all a launch takes."""
    n = 65535
    c = attn_case(22, 64, 64, 64, 16, [300, 40], [1, 2])
    dev = device(c)
    offsets = torch.full((n + 1,), 3, dtype=torch.int32)
    offsets[:n - 1] = 0
    offsets[n - 1] = 1
    lens = torch.zeros(n, dtype=torch.int32)
    lens[n - 2:] = c["lens"]
    table = torch.full((n, c["table"].shape[1]), -1, dtype=torch.int32)
    table[n - 2:] = c["table"]
    dev.update(offsets=offsets.cuda(), lens=lens.cuda(), table=table.cuda())
    for window in (0, 130):
        say("attention most requests, length hint", hint, window)
        out, lse = call_attention(M, c, dev, max_query_len=1, max_seq_len=hint, window=window)
        ref, ref_lse, tol, lse_tol = R.paged_attention(
            c["q"], c["kp"], c["ks"], c["vp"], c["vs"], c["table"], c["lens"], c["offsets"], 64, 16, c["scale"], True, window)
        assert bool(((host(out).double() - ref).abs() <= tol).all())
        assert bool(((host(lse).double() - ref_lse).abs() <= lse_tol).all())


@pytest.mark.parametrize("news", [1, 40])
@pytest.mark.parametrize("page", [1 << 16, 65533])
def test_attention_window_at_the_end_of_the_longest_table(M, page, news):
    """A table of nearly 2^30 tokens (two pages, over and over), of which a window
    shows the last ones: the same as a short context that ends with them."""
    width = (1 << 30) // page
    g = torch.Generator().manual_seed(23)
    kp, ks = R.random_nvfp4(g, 2 * page, 64)
    vp, vs = R.random_nvfp4(g, 2 * page, 64)
    length = width * page - 77
    table = (torch.arange(width) % 2).to(torch.int32)[None]
    c = dict(q=torch.randn(news, 4, 64, generator=g).to(torch.bfloat16), kp=kp, ks=ks, vp=vp, vs=vs, table=table,
             lens=torch.tensor([length], dtype=torch.int32), offsets=torch.tensor([0, news], dtype=torch.int32),
             kv_heads=1, page=page, scale=0.04)
    short = dict(c, table=table[:, -2:], lens=torch.tensor([2 * page - 77], dtype=torch.int32))
    for hint in (1000, 1 << 30, 2 ** 31 - 1, 2 ** 62):
        for window in (200, 3000):
            say("attention deep window", page, news, hint, window)
            out, lse = call_attention(M, c, device(c), max_seq_len=hint, window=window)
            ref, ref_lse, tol, lse_tol = R.paged_attention(
                short["q"], kp, ks, vp, vs, short["table"], short["lens"], short["offsets"], 1, page, 0.04, True, window)
            assert bool(((host(out).double() - ref).abs() <= tol).all())
            assert bool(((host(lse).double() - ref_lse).abs() <= lse_tol).all())


# ---- one token that takes nearly all the weight ------------------------------------
@pytest.mark.parametrize("octaves", [23.4, 25.2, 30.0])
@pytest.mark.parametrize("dim,page,news,hint", [
    (128, 16, 1, 100), (128, 16, 1, 65536), (64, 16, 40, 100), (64, 24, 3, 100), (256, 16, 2, 100), (256, 64, 50, 65536),
    (128, 16, 300, 100), (64, 32, 129, 65536), (256, 16, 60, 100), (128, 24, 130, 100)])
def test_attention_tail_behind_dominant_tokens(M, octaves, dim, page, news, hint):
    """Four tokens with values of zero take the weight, one of each of a
    workgroup's four waves (tokens 0, 32, 64, 96), and 65000 others stand `octaves`
    powers of two below: the result is the others' share alone.

    Bound: a probability is a hardware exponential (d, as in serving_ref), rounded
    to FP16 relative to a reference at least 2^11 below the row's largest: off by 2^-11
    relative or, where that is more, by 2^-25 of the reference, 2^-36 of the largest.
    Sums run in FP32 over n tokens; BF16 rounds by 2^-8."""
    heads, kv_heads, n = 4, 2, 65000
    pages = -(-n // page)
    g = torch.Generator().manual_seed(24)
    cols = kv_heads * dim
    sinks = torch.tensor([0, 32, 64, 96])
    kp, vp = torch.zeros(pages * page, cols // 2, dtype=torch.uint8), torch.randint(0, 256, (pages * page, cols // 2), generator=g)
    vp = (vp & 0x77).to(torch.uint8)                                # no negative values, so nothing cancels
    kp[sinks], vp[sinks] = 0x22, 0                                  # keys of ones, values of zero
    ks = torch.full((pages * page, cols // 16), 0x38, dtype=torch.uint8)       # scales of 1
    c = dict(q=torch.ones(news, heads, dim, dtype=torch.bfloat16), kp=kp, ks=ks, vp=vp, vs=ks, kv_heads=kv_heads, page=page,
             table=torch.arange(pages, dtype=torch.int32)[None], lens=torch.tensor([n], dtype=torch.int32),
             offsets=torch.tensor([0, news], dtype=torch.int32), scale=octaves * math.log(2) / dim)
    say("attention tail", octaves, dim, page, news, hint)
    out, lse = call_attention(M, c, device(c), max_seq_len=hint)
    v = R.nvfp4_values(vp[:n], ks[:n]).view(n, kv_heads, dim).cumsum(0)[n - news:].repeat_interleave(heads // kv_heads, 1)
    seen = torch.arange(n - news + 1, n + 1).double().view(-1, 1, 1)          # tokens that each row sees
    small = 2.0 ** -octaves
    total = 4 + (seen - 4) * small
    want = v * small / total
    d = (dim + 8) * 2.0 ** -24 * octaves * math.log(2) + 2.0 ** -21
    tol = want * (2.0 ** -8 + 2.0 ** -11 + 2 * d + (seen + 8) * 2.0 ** -24) + seen * 2.0 ** -36 * 6 / total
    worst = ((host(out).double() - want).abs() / tol).max()
    assert worst <= 1, worst
    exact = octaves * math.log(2) + torch.log(total[..., 0])
    assert bool(((host(lse).double() - exact).abs() <= d + (seen[..., 0] + 8) * 2.0 ** -24 + 2.0 ** -22 * (1 + exact)).all())


# ---- memory side by side -------------------------------------------------------------
def test_block_tables_in_one_buffer(M):
    """Every array in one allocation, one right behind the other, and the free
    list's end in a gap between two rows of the table: no overlap, not refused."""
    context, query, table, free = S.table_case(31, 7, 200, 16, "prompts")
    n, width, total = len(query), len(table[0]), sum(max(q, 0) for q in query)
    buf = torch.full((2 * (total + 3) + 4 * n + 2 + len(free) + n * (width + 3),), -9, dtype=torch.int32).cuda()
    at = [0]

    def take(count):
        at[0] += count
        return buf[at[0] - count:at[0]]

    slots = take(2 * (total + 3)).view(torch.int64)
    c, q, lens, offsets, f, begin = take(n), take(n), take(n), take(n + 1), take(len(free)), take(1)
    rows = take(n * (width + 3)).view(n, width + 3)
    c.copy_(torch.tensor(context))
    q.copy_(torch.tensor(query))
    f.copy_(torch.tensor(free))
    begin.fill_(2)
    rows[:, :width] = torch.tensor(table, dtype=torch.int32)
    end = rows[2, width + 1:width + 2]
    say("block tables in one buffer")
    M.kv_block_tables(c, q, rows[:, :width], 16, total + 3, free_pages=f, free_begin=begin, slots=slots, query_offsets=offsets,
                      seq_lens=lens, free_end=end)
    want = [list(r) for r in table]
    want_slots, want_offsets, want_lens, want_end = R.kv_block_tables(context, query, want, 16, total + 3, free, 2)
    assert host(slots).tolist() == want_slots and host(offsets).tolist() == want_offsets
    assert host(lens).tolist() == want_lens and host(end).tolist() == [want_end]
    gap = torch.full((n, 3), -9, dtype=torch.int32)
    gap[2, 1] = want_end
    assert torch.equal(host(rows), torch.cat([torch.tensor(want, dtype=torch.int32), gap], 1))


def test_block_tables_refuses_shared_memory(M):
    """From Python: views that overlap, and the pairs that start together."""
    n = 5
    buf = torch.zeros(4 * n, dtype=torch.int32).cuda()
    table = torch.zeros(n, 4, dtype=torch.int32).cuda()
    free = torch.arange(9, dtype=torch.int32).cuda()
    lens, query = buf[:n], buf[n:2 * n]
    say("block tables, shared memory")
    for more in (dict(query_offsets=buf[:n + 1]), dict(query_offsets=buf[2 * n - 1:3 * n]), dict(seq_lens=buf[1:n + 1]),
                 dict(free_end=buf[3:4]), dict(free_end=table[1, 1:2]), dict(free_end=free[8:]), dict(seq_lens=table.view(-1)[:n]),
                 dict(query_offsets=buf[2 * n:3 * n + 1], seq_lens=buf[3 * n:])):
        with pytest.raises(M.Nvfp4Error):
            M.kv_block_tables(lens, query, table, 4, 8, free_pages=free, **more)
    with pytest.raises(ValueError):
        M.kv_block_tables(lens, query, table, 4, 8, free_pages=free, seq_lens=lens)
    assert bool((host(buf) == 0).all())


# ---- what a layer must not read ---------------------------------------------------------
@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("tokens", [1, 20])
@pytest.mark.parametrize("hidden,inter", [(32, 32), (96, 64), (256, 128), (288, 160), (512, 256), (544, 288), (768, 384)])
def test_moe_unreached_experts_and_padding_may_hold_anything(M, kind, tokens, hidden, inter):
    """NaN in all weights of the experts that no token reaches, right behind the
    reached ones' last rows, and between the rows of a pitched x; summed axes of one
    to three chunks, whole and ragged."""
    c = S.moe_case(tokens + hidden, kind, tokens, hidden, inter, 4)
    c["logits"][:, 1::2] = -5.0 - c["logits"][:, 1::2].abs()
    c["logits"][:, 0::2] += 8.0
    nan8, nan16 = 0x7f, math.nan
    for n in ("w1", "w2"):
        c[n][1::2] = 0xff if kind == "nvfp4" else nan16
    if kind == "nvfp4":
        for n in ("s1", "s2"):
            c[n][1::2] = nan8
        for n in ("gs1", "gs2"):
            c[n][1::2] = math.nan
    dev = device(c)
    wide = torch.full((tokens, hidden + 24), math.nan, dtype=torch.bfloat16).cuda()
    wide[:, :hidden] = dev["x"]
    say("moe unread", kind, tokens, hidden, inter)
    for top_k in (1, 2):
        out, ids, _ = S.call_moe(M, c, dict(dev, x=wide[:, :hidden]), top_k)
        ref, tol, want, _ = R.moe_layer(c["x"], c["logits"], c["w1d"], c["w2d"], top_k, True,
                                        2.0 ** -17 if kind == "bf16" else 2.0 ** -11)
        assert host(ids).tolist() == want.tolist()
        d = (host(out).double() - ref).abs() - tol
        assert bool((d <= 0).all()), d.max()


# ---- Python integers past the C types ---------------------------------------------------
def test_integers_past_the_c_types(M):
    """Sizes that would wrap are refused; hints and windows past 64 bits mean the
    same as the largest that fit."""
    c = attn_case(41, 8, 2, 64, 16, [90, 33], [1, 3])
    dev = device(c)
    lens = torch.tensor([5, 6], dtype=torch.int32).cuda()
    table = torch.zeros(2, 4, dtype=torch.int32).cuda()
    say("integers past the C types")
    for page in (2 ** 32 + 16, 2 ** 31, -2 ** 32 + 16, 2 ** 64 + 16):
        with pytest.raises(ValueError):
            M.kv_block_tables(None, lens, table, page, 11)
        with pytest.raises(ValueError):
            call_attention(M, dict(c, page=page), dev)
    want = call_attention(M, c, dev, max_query_len=2 ** 63 - 1, max_seq_len=2 ** 63 - 1, window=2 ** 63 - 1)
    for big in (2 ** 63, 2 ** 64 + 5, 2 ** 70):
        got = call_attention(M, c, dev, max_query_len=big, max_seq_len=big, window=big)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), big
        for name in ("max_query_len", "max_seq_len", "window"):
            with pytest.raises(ValueError):
                call_attention(M, c, dev, **{name: -big - 1})
    with pytest.raises(M.Nvfp4Error):
        call_attention(M, c, dev, window=-1)
    for tokens in (0, 2):
        w = S.moe_case(42, "bf16", tokens, 64, 32, 4)
        for top_k in (2 ** 32 + 1, -2 ** 32 + 1):
            with pytest.raises(ValueError):
                S.call_moe(M, w, device(w), top_k)


# ---- every form of the prompt kernel ------------------------------------------------------
@pytest.mark.parametrize("heads,kv_heads,dim,page,totals,news", [
    (4, 1, 256, 24, [300, 65], [130, 65]), (8, 2, 256, 1, [150, 40], [60, 40]), (4, 2, 256, 7, [700], [200]),
    (2, 2, 256, 100, [260, 1, 90], [257, 1, 33]), (3, 1, 64, 40, [600], [300])])
def test_attention_prompts_with_other_pages(M, heads, kv_heads, dim, page, totals, news):
    c = attn_case(dim + heads + page, heads, kv_heads, dim, page, totals, news, pad=2)
    say("attention prompts, other pages", heads, kv_heads, dim, page, totals, news)
    check_attention(M, c, gs=(0.9, 1.1))
    check_attention(M, c, window=50)
    check_attention(M, c, causal=False)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 24, 1])
def test_attention_split_prompts(M, dim, page):
    """Ranges of several thousand tokens for few requests: the prompt kernel's
    splits and their join, with windows that empty the first splits."""
    c = attn_case(dim + page, 8, 2, dim, page, [4097, 1500, 60], [70, 40, 33])
    say("attention split prompts", dim, page)
    need = M.serving.raw().nvfp4_paged_attention_workspace(143, 8, 2, dim, 3, 70, 4097, 0)
    assert need > 0
    check_attention(M, c)
    check_attention(M, c, window=1200)
    check_attention(M, c, window=3000, causal=False)


# ---- small values beside large ones -------------------------------------------------------
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("news", [1, 40, 200])
@pytest.mark.parametrize("power", [20, 31, 35])
def test_attention_small_components_of_a_query(M, dim, news, power):
    """One component of q meets keys of 0 and is 2^power times the others, which alone
    make the scores. Down to 2^-31 of the largest they are exact in FP16; below they are
    off by at most 2^-39 of it."""
    c = attn_case(51, 4, 2, dim, 16, [230], [news], scale=0.05 * 2.0 ** power)
    g = torch.Generator().manual_seed(power + dim)
    q = (1 + torch.randint(0, 128, c["q"].shape, generator=g) / 128) * torch.where(torch.rand(c["q"].shape, generator=g) < 0.5, -1.0, 1.0)
    q *= 2.0 ** -power
    q[:, :, 3] = 1.0
    c["q"] = q.to(torch.bfloat16)
    assert torch.equal(c["q"].float(), q)
    kp = c["kp"].view(-1, 2, dim // 2)
    kp[:, :, 1] &= 0x0f                                # element 3 of each head's keys: 0
    c["ks"] = (c["ks"].int() & 7 | 0x38).to(torch.uint8)         # scales of 1 to 2
    say("attention small components", dim, news, power)
    out, lse = call_attention(M, c, device(c))
    ref, ref_lse, tol, lse_tol = R.paged_attention(*[c[k] for k in ("q", "kp", "ks", "vp", "vs", "table", "lens", "offsets")], 2,
                                                   16, c["scale"])
    d = 0.0 if power <= 31 else 2.0 ** -39 * dim * 12 * c["scale"]      # keys are at most 6 x 1.875
    v = R.nvfp4_values(c["vp"], c["vs"]).abs().max()
    assert bool(((host(lse).double() - ref_lse).abs() <= lse_tol + d).all())
    assert bool(((host(out).double() - ref).abs() <= tol + 2 * d * v).all())


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("tokens", [1, 18])
@pytest.mark.parametrize("inter", [96, 512])
@pytest.mark.parametrize("power", [10, 18, 22])
def test_moe_small_activations_beside_a_large_one(M, kind, tokens, inter, power):
    """h[0] is about 2^(power + 11) times the others and meets weights of 0, so the others
    alone make the result: h is rounded by 2^-11 relative or, where that is more, by 2^-39
    of the largest of its run of 256 (NVFP4 weights), by 2^-17 relative (BF16 weights)."""
    hidden, experts = 64, 2
    g = torch.Generator().manual_seed(power)
    c = S.moe_case(52, kind, tokens, hidden, inter, experts)
    x = torch.zeros(tokens, hidden)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -power, 1.0
    c["x"] = x.to(torch.bfloat16)
    j = torch.arange(inter)
    gate, up = 16 * (j // 8) + j % 8, 16 * (j // 8) + 8 + j % 8
    w1 = torch.zeros(experts, 2 * inter, hidden, dtype=torch.float64)
    w1[:, gate, 0] = 4.0                                                 # gates: 4
    w1[:, up, 1] = torch.randint(1, 5, (experts, inter), generator=g).double() / 2      # ups: 2^-power times 0.5 to 2
    w1[:, 8, 1], w1[:, 8, 2] = 0.0, 6.0                                  # the first up: 6, times 256 by its block's scale
    w1[:, 8] *= 256
    w2 = torch.randint(1, 5, (experts, hidden, inter), generator=g).double() / 2
    w2[:, :, 0] = 0.0
    if kind == "bf16":
        c["w1"], c["w2"] = w1.to(torch.bfloat16), w2.to(torch.bfloat16)
        assert torch.equal(c["w1"].double(), w1)
    else:
        for name, w in (("1", w1), ("2", w2)):
            scale = torch.ones(w.shape[0], w.shape[1], w.shape[2] // 16, dtype=torch.float64)
            if name == "1":
                scale[:, 8] = 256.0
            code = (torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]).double() ==
                    (w / scale.repeat_interleave(16, -1))[..., None]).double().argmax(-1).to(torch.uint8)
            c["w" + name] = code[..., 0::2] | code[..., 1::2] << 4
            c["s" + name] = torch.where(scale == 256.0, 0x78, 0x38).to(torch.uint8)
            c["gs" + name] = torch.ones(experts)
            assert torch.equal(R.nvfp4_values(c["w" + name], c["s" + name]), w)
    say("moe small activations", kind, tokens, inter, power)
    out, ids, weights = S.call_moe(M, c, device(c), 1)
    ids = host(ids)[:, 0].long()
    acc = torch.matmul(w1, c["x"][0].double())                           # every token is the same
    h = acc[:, gate] * torch.sigmoid(acc[:, gate]) * acc[:, up]
    want = torch.matmul(w2, h[:, :, None])[:, :, 0][ids]
    if kind == "bf16":
        dh = 2.0 ** -17 * h.abs()
    else:
        run = torch.nn.functional.pad(h.abs(), (0, -inter % 256)).view(experts, -1, 256).amax(2).repeat_interleave(256, 1)[:, :inter]
        dh = torch.maximum(2.0 ** -11 * h.abs(), 2.0 ** -39 * run)
    dh = dh + 2.0 ** -19 * h.abs()
    tol = torch.matmul(w2, dh[:, :, None])[:, :, 0][ids] + want.abs() * (2.0 ** -8 + (inter + 16) * 2.0 ** -24 + 2.0 ** -20)
    worst = ((host(out).double() - want).abs() / tol).max()
    assert worst <= 1, worst


# ---- NaN -------------------------------------------------------------------------------
@pytest.mark.parametrize("dim,news,hint", [(64, 1, 100), (128, 1, 4000), (256, 2, 100), (128, 40, 100), (64, 200, 4000),
                                           (256, 100, 100)])
def test_attention_nan_is_not_hidden(M, dim, news, hint):
    """A global scale of keys that is NaN, and a query with a NaN: the results of the rows
    it reaches are NaN, no number; the other rows' stay in their bounds."""
    c = attn_case(61, 8, 2, dim, 16, [3000, 500], [news, 1], scale=0.02)
    dev = device(c)
    say("attention nan", dim, news, hint)
    nan = torch.tensor([math.nan]).cuda()
    for more in (dict(k_gs=nan), dict(k_gs=nan, window=600)):
        out, lse = call_attention(M, c, dev, max_seq_len=hint, **more)
        assert bool(torch.isnan(host(out)).all()) and bool(torch.isnan(host(lse)).all())
    c["q"][0, 2, 5] = math.nan
    out, lse = call_attention(M, c, device(c), max_seq_len=hint)
    out, lse = host(out), host(lse)
    assert bool(torch.isnan(out[0, 2]).all()) and bool(torch.isnan(lse[0, 2]))
    c["q"][0, 2, 5] = 0
    ref, ref_lse, tol, lse_tol = R.paged_attention(*[c[k] for k in ("q", "kp", "ks", "vp", "vs", "table", "lens", "offsets")], 2,
                                                   16, c["scale"])
    rest = torch.ones(news + 1, 8, dtype=torch.bool)
    rest[0, 2] = False
    assert bool(((out.double() - ref).abs() <= tol)[rest].all()) and bool(((lse.double() - ref_lse).abs() <= lse_tol)[rest].all())


# ---- a cache past 4 GiB -----------------------------------------------------------------
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("news", [1, 70])
def test_attention_far_in_a_large_cache(M, page, news):
    """Codes of 4.6 GB each for keys and values: pages behind 4 GiB give what the same
    pages in a small cache give."""
    c = attn_case(71, 16, 8, 256, page, [400, 90], [news, 1])
    dev = device(c)
    say("attention large cache", page, news)
    want = call_attention(M, c, dev)
    used = c["kp"].shape[0]
    slots = 4500000 // page * page
    first = slots // page - used // page
    big = dict(dev)
    for k in ("kp", "ks", "vp", "vs"):
        big[k] = torch.zeros(slots, c[k].shape[1], dtype=torch.uint8, device="cuda")
        big[k][slots - used:] = dev[k]
    assert big["kp"].numel() > 2 ** 32
    big["table"] = torch.where(dev["table"] >= 0, dev["table"] + first, dev["table"])
    got = call_attention(M, c, big)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ---- rows far apart, the largest layers ---------------------------------------------------
def spread(t, pitch, fill):
    """A view with t's values and rows `pitch` elements apart, and its buffer."""
    buf = torch.full(((t.shape[0] - 1) * pitch + t[0].numel(),), fill, dtype=t.dtype, device="cuda")
    view = buf.as_strided(t.shape, (pitch,) + t.stride()[1:])
    view.copy_(t)
    return view


@pytest.mark.parametrize("news,page", [([1, 2, 1], 16), ([70, 3, 1], 16), ([1, 40, 2], 24)])
def test_attention_rows_and_tables_far_apart(M, news, page):
    """Rows of q, out and the block table whose byte offsets pass 32 bits."""
    c = attn_case(81, 8, 2, 64, page, [2500, 90, 40], news)
    dev = device(c)
    say("attention far rows", news, page)
    want, want_lse = call_attention(M, c, dev)
    rows = c["q"].shape[0]
    pitch = (5 << 30) // 2 // (rows - 1) // 8 * 8
    far = dict(dev, q=spread(dev["q"], pitch, 3.0), table=spread(dev["table"], (5 << 30) // 8, -1))
    out = spread(torch.zeros_like(dev["q"]), pitch, 5.0)
    _, lse = call_attention(M, c, far, out=out)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    del far, out


def test_block_tables_rows_far_apart(M):
    context, query, table, free = S.table_case(82, 3, 300, 16, "prompts")
    total, width = sum(max(q, 0) for q in query), len(table[0])
    far = spread(torch.tensor(table, dtype=torch.int32).cuda(), (5 << 30) // 8, -9)
    say("block tables far rows")
    got = M.kv_block_tables(S.ints(context), S.ints(query), far, 16, total, free_pages=S.ints(free))
    want = R.kv_block_tables(context, query, table, 16, total, free)
    for a, b in zip(got, want):
        assert host(a).tolist() == (b if isinstance(b, list) else [b])
    assert host(far).tolist() == table


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
def test_moe_rows_far_apart(M, kind):
    """x over the most bytes that a call takes, out over more than 4 GiB."""
    c = S.moe_case(83, kind, 64, 64, 32, 6)
    dev = device(c)
    say("moe far rows", kind)
    want = S.call_moe(M, c, dev, 2)
    pitch = (2 ** 31 - 4096 - 1) // 2 - 64
    x = spread(dev["x"], pitch // 63 // 8 * 8, math.nan)
    out = spread(torch.zeros_like(dev["x"]), (5 << 30) // 2 // 63 // 8 * 8, 5.0)
    got = S.call_moe(M, c, dict(dev, x=x), 2, out=out)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(M.Nvfp4Error):
        S.call_moe(M, c, dict(dev, x=spread(dev["x"], 2 ** 30 // 63 // 8 * 8 + 8, 0.0)), 2)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("hidden,inter", [(2 ** 20, 32), (32, 2 ** 20)])
def test_moe_largest_layers(M, kind, hidden, inter):
    c = S.moe_case(84, kind, 2, hidden, inter, 2)
    say("moe largest", kind, hidden, inter)
    S.check_moe(M, c, 1, True)


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
def test_moe_most_workspace(M, kind):
    """64 tokens whose values of h fill nearly 2^31 bytes: the last tokens' results are
    those of a call with these tokens alone."""
    hidden, inter, experts, top_k = 32, 2 ** 20, 8, 7
    g = torch.Generator(device="cuda").manual_seed(85)
    x = torch.randn(64, hidden, generator=g, device="cuda").to(torch.bfloat16)
    dev = dict(x=x, logits=torch.randn(64, experts, generator=g, device="cuda"))
    shapes = (("1", (experts, 2 * inter, hidden)), ("2", (experts, hidden, inter)))
    for n, (e, rows, cols) in shapes:
        if kind == "bf16":
            dev["w" + n] = torch.empty(e, rows, cols, dtype=torch.bfloat16, device="cuda").normal_(0, cols ** -0.5, generator=g)
        else:
            dev["w" + n] = torch.randint(0, 256, (e, rows, cols // 2), generator=g, device="cuda", dtype=torch.uint8)
            dev["s" + n] = torch.randint(0x20, 0x41, (e, rows, cols // 16), generator=g, device="cuda", dtype=torch.uint8)
            dev["gs" + n] = torch.full((e,), (8 * cols) ** -0.5, device="cuda")
    c = dict(kind=kind)
    say("moe most workspace", kind)
    out, ids, weights = S.call_moe(M, c, dev, top_k)
    for first in (0, 30, 61):
        few, few_ids, few_weights = S.call_moe(M, c, dict(dev, x=x[first:first + 3].contiguous(), logits=dev["logits"][first:first + 3]), top_k)
        assert torch.equal(ids[first:first + 3], few_ids) and torch.equal(weights[first:first + 3], few_weights)
        # the same FP32 sums, cut into other runs: two BF16 roundings, and some 2^10 roundings
        # of random sign (2^20 terms) of 2^-24 of the largest sums
        a, b = out[first:first + 3].double(), few.double()
        assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -10 * b.abs().amax()).all())


@pytest.mark.parametrize("kind", ["nvfp4", "bf16"])
@pytest.mark.parametrize("tokens", [2, 16, 40])
def test_moe_rows_of_a_padded_batch_leave_the_others_alone(M, kind, tokens):
    """Rows of x with NaN and infinities, and of logits with NaN, as a padded batch may
    hold: the other rows' results keep every byte."""
    c = S.moe_case(91, kind, tokens, 288, 96, 6)
    dev = device(c)
    say("moe padded rows", kind, tokens)
    for top_k in (1, 3):
        want = S.call_moe(M, c, dev, top_k)
        for bad, logits in ((math.nan, False), (math.inf, False), (math.nan, True)):
            rest = torch.arange(tokens) % 5 != 1
            x, z = c["x"].clone(), c["logits"].clone()
            x[~rest] = bad
            x[~rest, ::3] = -bad
            if logits:
                z[~rest] = math.nan
            got = S.call_moe(M, c, dict(dev, x=x.cuda(), logits=z.cuda()), top_k)
            for a, b in zip(got, want):
                assert torch.equal(host(a)[rest], host(b)[rest]), (top_k, bad, logits)
            out = host(got[0])[~rest]
            assert bool((out == 0).all() if logits else (~torch.isfinite(out)).any())
