"""tests/sparse_many_ref.py against tests/sparse_ref.py on small cases, and its copy
of the selection's plan against the library's workspace query. CPU only."""
import itertools

import pytest
import torch

import sparse_many_ref as P
import sparse_ref as S
from test_gpu_sparse import request_case
from test_sparse_host import lib  # noqa: F401


@pytest.mark.parametrize("heads,kv,dim,page", [(8, 2, 64, 4), (3, 3, 64, 1), (14, 2, 128, 3)])
def test_selection(heads, kv, dim, page):
    totals, news = [0, -5, 3, 30 * page + 1, 9 * page, page], [1, 2, 6, 5, 1, page]
    hide = [(3, j, -1) for j in range(0, 20, 3)] + [(3, 4, 10 ** 9), (3, 7, -2 ** 31)] + [(4, j, -1) for j in range(9)]
    c = request_case(heads, kv, dim, page, totals, news, hide=hide, heads=heads, pad=2)
    c["keys"][:, 0, 1:] = 0                       # ties
    c["q"][3] = 0
    args = (c["q"], c["keys"], c["exponents"], c["table"], c["lens"], c["offsets"], page)
    for top, first, local in ((4, 1, 2), (0, 0, 1), (100, 3, 2), (7, 0, 40)):
        assert torch.equal(P.select_pages(*args, top, first, local), S.select_pages(*args, top, first, local))


def test_page_keys():
    c = request_case(3, 3, 64, 4, [100], [100])
    entries = c["table"][0, :25].long()
    sums = P.page_sums(c["kp"], c["ks"], entries, 3, 64, 4)
    e = P.key_exponents(sums)
    keys, exponents, other = S.page_keys(c["kp"], c["ks"], c["table"], c["lens"], c["offsets"], c["keys"], c["exponents"], 4)
    assert torch.equal(exponents[entries].long(), e.long())
    exact = (sums.double() * torch.pow(2.0, -e.double())[..., None]).round().clamp(-127, 127)
    assert torch.equal(keys[entries].double(), exact)
    assert P.key_exponents(torch.tensor([[[0, 0]], [[127, -1]], [[-128, 5]], [[0, 255]], [[-256, 0]]])).flatten().tolist() \
        == [0, 0, 1, 1, 2]


def test_plan_of_the_selection(lib):  # noqa: F811
    for tokens, (heads, kv), seqs, width in itertools.product(
            (1, 3, 64, 90, 100, 500, 1000, 2048), ((8, 8), (32, 8), (28, 4), (200, 2), (1, 1)), (0, 1, 3, 64, 500),
            (0, 1, 60, 400, 2049, 32768)):
        assert P.select_plan(tokens, heads, kv, seqs, width)[2] == lib.nvfp4_select_pages_workspace(tokens, heads, kv, seqs, width)
