"""Limits of the sparse-attention operators on the host, no GPU needed: the workspace
queries refuse what the calls refuse."""
import pytest

from test_sparse_host import INVALID, MISALIGNED, SHAPE, lib, select, sparse  # noqa: F401


@pytest.mark.parametrize("tokens,heads,kv,seqs,refused", [
    (4, 8, 2, 65535, False), (4, 8, 2, 65536, True), (4, 64, 64, 65535, False), (4, 65, 65, 65535, True),
    (4, 1024, 1024, 4096, False), (4, 1024, 1024, 4097, True), (0, 8, 2, 65536, True), (4, 8, 2, 2 ** 40, True),
    (4, 8, 2, 2 ** 62, True), (2 ** 20, 8, 2, 4, False), (2 ** 20 + 1, 8, 2, 4, True)])
def test_sparse_workspace_refuses_what_the_call_refuses(lib, tokens, heads, kv, seqs, refused):  # noqa: F811
    size = lib.nvfp4_sparse_attention_workspace(tokens, heads, kv, 128, 16, seqs, 20)
    assert (size == -1) == refused and (refused or size >= 0)
    ld = heads * 128
    # no launch is reached: sizes that are taken are refused for q's alignment
    got = sparse(lib, q=0x10008, tokens=tokens, heads=heads, kv=kv, n=seqs, ld_q=ld, ld_o=ld)
    # (a table of 2^62 rows is refused before its number of requests, as it passes 2^63 bytes)
    assert got == (MISALIGNED if not refused and tokens else INVALID if seqs == 2 ** 62 else SHAPE), got


@pytest.mark.parametrize("tokens,heads,kv,seqs,pages,refused", [
    (4, 8, 2, 65535, 8, False), (4, 8, 2, 65536, 8, True), (4, 8, 2, 2, 32768, False), (4, 8, 2, 2, 32769, True),
    (2 ** 20, 8, 2, 2, 8, False), (2 ** 20 + 1, 8, 2, 2, 8, True), (4, 1024, 1024, 2, 8, False), (4, 1025, 1, 2, 8, True)])
def test_select_workspace_refuses_what_the_call_refuses(lib, tokens, heads, kv, seqs, pages, refused):  # noqa: F811
    size = lib.nvfp4_select_pages_workspace(tokens, heads, kv, seqs, pages)
    assert (size == -1) == refused and (refused or size >= 0)
    got = select(lib, q=0x10008, tokens=tokens, heads=heads, kv=kv, n=seqs, mp=pages, ld=pages, ld_q=heads * 128)
    assert got == (SHAPE if refused else MISALIGNED), got
