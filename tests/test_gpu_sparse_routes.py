"""The sparse-attention operators on the GPU: what a workspace held before a call
does not change its result, whatever the offsets."""
import numpy as np
import pytest
import torch

from test_gpu_sparse import M, call_sparse, device, host, lists, request_case, say  # noqa: F401

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
