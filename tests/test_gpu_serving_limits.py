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
