"""The sparse-attention operators on the host, no GPU needed: the header and the
exports agree, bad arguments are refused with the documented status before any
HIP call, the workspace sizes, and the plain definitions of the GPU tests against
hand-worked values."""
import math
import os
import re
import subprocess

import numpy as np
import pytest
import torch

import sparse_ref as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_sparse.h")
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
A = 0x10000      # a fake aligned "device" address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from moe_swiglu_epilogue_amd import binding, build, sparse
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return sparse.raw()


def test_header_and_exports_agree(lib):
    import moe_swiglu_epilogue_amd as M
    from moe_swiglu_epilogue_amd import binding, sparse
    names = set(re.findall(r"^(?:nvfp4_status_t|int64_t)\s+(\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(sparse.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(l.split()[-1] for l in out.splitlines() if " T " in l)
    assert {n for n in names if not n.endswith("_workspace")} <= set(M.__all__)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "nvfp4_sparse.h"\nint main(void){return (int)NVFP4_SUCCESS;}\n')
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def append(lib, q=A, tokens=4, ld_q=1024, heads=8, k=A + 0x10000, ld_k=256, v=A + 0x20000, ld_v=256, kv=2, dim=128,
           pos=A, ld_pos=4, axes=1, axis=None, cs=A, most=100, rot=128, inter=0, kg=None, vg=None, slots=A, ns=160,
           kp=A + 0x100000, ks=A + 0x200000, vp=A + 0x300000, vs=A + 0x400000, out=A + 0x500000, ld_o=1024):
    return lib.nvfp4_rope_append(q, tokens, ld_q, heads, k, ld_k, v, ld_v, kv, dim, pos, ld_pos, axes, axis, cs, most, rot, inter,
                                 kg, vg, slots, ns, kp, ks, vp, vs, out, ld_o, None)


def test_append_validation(lib):
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=-8), dict(kv=0), dict(dim=0), dict(axes=0), dict(most=-1), dict(rot=-2),
                dict(rot=130), dict(ns=-1), dict(ld_q=1016), dict(ld_o=1016), dict(ld_k=248), dict(ld_v=248), dict(ld_q=2 ** 62),
                dict(ld_k=2 ** 62), dict(axes=2, ld_pos=3), dict(axes=3, ld_pos=2 ** 62), dict(k=None), dict(v=None),
                dict(slots=None), dict(out=None), dict(pos=None), dict(cs=None), dict(kp=None), dict(ks=None), dict(vp=None),
                dict(vs=None), dict(ns=2 ** 62)):
        assert append(lib, **bad) == INVALID, bad
    for bad in (dict(dim=120, rot=64), dict(dim=528, ld_k=2048, ld_v=2048, ld_q=8192, ld_o=8192), dict(rot=127), dict(axes=17, ld_pos=9),
                dict(heads=1025, ld_q=2 ** 18, ld_o=2 ** 18), dict(kv=1025, ld_k=2 ** 18, ld_v=2 ** 18), dict(tokens=2 ** 31),
                dict(most=2 ** 31)):
        assert append(lib, **bad) == SHAPE, bad
    for bad in (dict(q=A + 8), dict(k=A + 8), dict(v=A + 8), dict(out=A + 8), dict(cs=A + 4), dict(slots=A + 4), dict(kp=A + 4),
                dict(vp=A + 4), dict(pos=A + 2), dict(axis=A + 2), dict(kg=A + 2), dict(vg=A + 2), dict(ld_q=1028), dict(ld_o=1028),
                dict(ld_k=260), dict(ld_v=260)):
        assert append(lib, **bad) == MISALIGNED, bad
    assert append(lib, tokens=0) == OK


def test_append_refuses_shared_memory(lib):
    """The rotated q over q, k or v (4 rows of 1024 and 256 values of 2 bytes), at
    either end; the caches over each other (160 rows)."""
    for name, at, size in (("q", 0x800000, 8192), ("k", 0x900000, 2048), ("v", 0xa00000, 2048)):
        for out in (at, at + size - 16, at - 8192 + 16):
            assert append(lib, **{name: at, "out": out}) == INVALID, (name, out - at)
    for a, b, n in (("kp", "vp", 160 * 128), ("ks", "vs", 160 * 16)):
        for at in (0x800000, 0x800000 + n - 8, 0x800000 - n + 8):
            assert append(lib, **{a: 0x800000, b: at}) == INVALID, (a, at)


def keys(lib, kp=A, ks=A, ns=160, kv=2, dim=128, page=16, table=A, ld=8, mp=8, lens=A, off=A, n=2, mq=2, keys=A, e=A):
    return lib.nvfp4_page_keys(kp, ks, ns, kv, dim, page, table, ld, mp, lens, off, n, mq, keys, e, None)


def test_page_keys_validation(lib):
    for bad in (dict(ns=-16), dict(ns=161), dict(kv=0), dict(page=0), dict(mp=-1), dict(ld=7), dict(n=-1), dict(mq=-1),
                dict(ld=2 ** 62), dict(kp=None), dict(ks=None), dict(table=None), dict(lens=None), dict(off=None), dict(keys=None),
                dict(e=None)):
        assert keys(lib, **bad) == INVALID, bad
    for bad in (dict(dim=96), dict(dim=512), dict(kv=1025), dict(n=65536), dict(ns=2 ** 31), dict(mp=2 ** 26 + 1, ld=2 ** 27)):
        assert keys(lib, **bad) == SHAPE, bad
    for bad in (dict(kp=A + 4), dict(keys=A + 8), dict(table=A + 2), dict(lens=A + 2), dict(off=A + 2)):
        assert keys(lib, **bad) == MISALIGNED, bad
    for empty in (dict(n=0), dict(ns=0), dict(mp=0, ld=0)):
        assert keys(lib, **empty) == OK


def select(lib, q=A, tokens=4, ld_q=1024, heads=8, kv=2, dim=128, keys=A, e=A, ns=160, page=16, table=A, ld=8, mp=8, lens=A, off=A,
           n=2, top=4, first=1, local=2, pages=A, ws=A, wb=2 ** 40):
    return lib.nvfp4_select_pages(q, tokens, ld_q, heads, kv, dim, keys, e, ns, page, table, ld, mp, lens, off, n, top, first, local,
                                  pages, ws, wb, None)


def test_select_validation(lib):
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=7), dict(kv=0), dict(top=-1), dict(first=-1), dict(local=0), dict(ld_q=1016),
                dict(ld_q=2 ** 62), dict(ns=-16), dict(ns=161), dict(page=0), dict(mp=-1), dict(ld=7), dict(n=-1), dict(q=None),
                dict(keys=None), dict(e=None), dict(table=None), dict(lens=None), dict(off=None), dict(pages=None), dict(wb=-1),
                dict(wb=0), dict(ws=None)):
        assert select(lib, **bad) == INVALID, bad
    for bad in (dict(dim=96, ld_q=2048), dict(heads=2048, ld_q=2 ** 19), dict(n=65536), dict(tokens=2 ** 28), dict(ns=2 ** 31),
                dict(mp=32769, ld=2 ** 16), dict(mp=2 ** 14, ld=2 ** 16, page=2 ** 17, ns=2 ** 18), dict(top=2046),
                dict(first=2043), dict(local=2044), dict(top=2 ** 31 - 1), dict(top=2 ** 31 - 1, first=2 ** 31 - 1, local=2 ** 31 - 1)):
        assert select(lib, **bad) == SHAPE, bad
    for bad in (dict(q=A + 8), dict(keys=A + 8), dict(ld_q=1028), dict(table=A + 2), dict(lens=A + 2), dict(off=A + 2),
                dict(pages=A + 2), dict(ws=A + 8)):
        assert select(lib, **bad) == MISALIGNED, bad
    for empty in (dict(tokens=0), dict(n=0)):
        assert select(lib, **empty) == OK


def test_select_workspace(lib):
    """Scores of all pages for few tokens; none for many, and where they would be large."""
    size = lib.nvfp4_select_pages_workspace
    assert size(1, 32, 8, 1, 2049) == 8 * 2052 * 4 and size(64, 64, 8, 64, 1024) == 64 * 8 * 1024 * 4
    assert size(4096, 32, 8, 1, 500) == 0 and size(4096, 32, 8, 4096, 500) == 0 and size(0, 8, 8, 0, 9) == 0
    assert size(5, 8, 2, 2, 30) == 5 * 2 * 32 * 4 and size(600, 4, 4, 1, 32768) == 0
    for bad in ((-1, 8, 8, 1, 4), (1, 8, 3, 1, 4), (1, 8, 8, -1, 4), (1, 8, 8, 1, -4), (1, 8, 8, 1, 32769), (1, 2048, 8, 1, 4),
                (1, 8, 8, 65536, 4), (2 ** 21, 8, 8, 1, 4)):
        assert size(*bad) == -1, bad


def sparse(lib, q=A, tokens=4, ld_q=1024, heads=8, kv=2, dim=128, kp=A, ks=A, vp=A, vs=A, ns=160, page=16, table=A, ld=8, mp=8, lens=A,
           off=A, n=2, pages=A, listed=20, scale=0.1, kg=None, vg=None, out=A, ld_o=1024, lse=None, ws=A, wb=2 ** 40):
    return lib.nvfp4_sparse_attention(q, tokens, ld_q, heads, kv, dim, kp, ks, vp, vs, ns, page, table, ld, mp, lens, off, n, pages,
                                      listed, scale, kg, vg, out, ld_o, lse, ws, wb, None)


def test_sparse_attention_validation(lib):
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=7), dict(kv=0), dict(ns=-16), dict(ns=161), dict(page=0), dict(mp=-1),
                dict(ld=7), dict(ld=2 ** 62), dict(n=-1), dict(listed=-1), dict(scale=math.nan), dict(scale=math.inf),
                dict(ld_q=1016), dict(ld_o=1016), dict(ld_q=2 ** 62), dict(ld_o=2 ** 62), dict(q=None), dict(out=None),
                dict(lens=None), dict(off=None), dict(table=None), dict(kp=None), dict(ks=None), dict(vp=None), dict(vs=None),
                dict(pages=None), dict(wb=-1), dict(wb=0, listed=2000), dict(ws=None, listed=2000)):
        assert sparse(lib, **bad) == INVALID, bad
    for bad in (dict(dim=96, ld_q=2048, ld_o=2048), dict(heads=2048, ld_q=2 ** 19, ld_o=2 ** 19), dict(n=65536), dict(tokens=2 ** 28),
                dict(ns=2 ** 31), dict(mp=2 ** 26 + 1, ld=2 ** 27), dict(listed=2049), dict(listed=2 ** 40),
                dict(listed=1025, page=2 ** 20, ns=2 ** 20)):
        assert sparse(lib, **bad) == SHAPE, bad
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(ld_q=1028), dict(ld_o=1028), dict(kp=A + 8), dict(vp=A + 8), dict(ks=A + 4),
                dict(vs=A + 4), dict(table=A + 2), dict(lens=A + 2), dict(off=A + 2), dict(pages=A + 2), dict(kg=A + 2),
                dict(vg=A + 2), dict(lse=A + 2), dict(ws=A + 8)):
        assert sparse(lib, **bad) == MISALIGNED, bad
    for empty in (dict(tokens=0), dict(n=0)):
        assert sparse(lib, **empty) == OK


def test_sparse_workspace(lib):
    """None for many tokens; for few an output row, a reference and a sum a split, and
    a count a row."""
    size = lib.nvfp4_sparse_attention_workspace
    assert size(4096, 32, 8, 128, 64, 1, 32) == 0 and size(0, 32, 8, 128, 64, 2, 32) >= 0 and size(1, 8, 8, 128, 16, 1, 0) == 0
    n = size(1, 32, 8, 128, 64, 1, 1000)
    assert n > 0 and (n // 4 // 32 - 1) % 130 == 0
    for bad in ((-1, 8, 8, 128, 16, 1, 4), (1, 8, 3, 128, 16, 1, 4), (1, 8, 8, 96, 16, 1, 4), (1, 8, 8, 128, 0, 1, 4),
                (1, 8, 8, 128, 16, 1, 2049), (1, 8, 8, 128, 2 ** 20, 1, 1025), (2 ** 28, 8, 8, 128, 16, 1, 4),
                (1, 8, 8, 128, 16, -1, 4)):
        assert size(*bad) == -1, bad
    for page, listed in ((2 ** 30, 1), (2 ** 19, 2048), (1, 2048), (524287, 2048)):
        for tokens in (1, 3, 100):
            for seqs in (0, 1, 50):
                assert size(tokens, 8, 1, 64, page, seqs, listed) >= 0


# ---- the definitions -------------------------------------------------------------
def test_rotation_by_hand():
    """A quarter turn and a half turn; a position behind the table; the second pair on
    the other axis."""
    x = torch.tensor([[[1.0, 2.0, 3.0, 4.0, 5.0]]]).to(torch.bfloat16)
    table = torch.tensor([[1.0, 1.0, 0.0, 0.0], [0.0, 0.0, 1.0, 1.0], [-1.0, -1.0, 0.0, 0.0]])
    turn = lambda *p, **m: S.rotate(x, torch.tensor(p, dtype=torch.int32)[:, None], table, **m)[0, 0].tolist()  # noqa: E731
    assert turn(0) == [1, 2, 3, 4, 5]
    assert turn(1) == [-3, -4, 1, 2, 5] and turn(2) == [-1, -2, -3, -4, 5] and turn(3) == [1, 2, 3, 4, 5]
    assert turn(1, interleaved=True) == [-2, 1, -4, 3, 5]
    assert turn(1, 2, pair_axis=[0, 1]) == [-3, -2, 1, -4, 5] and turn(1, 2, pair_axis=[2, 1]) == [1, -2, 3, -4, 5]


def test_page_keys_by_hand():
    """Two tokens of 64 values: 6 * 2 and 0.5 * 1 in one, 4 * 2 in the other."""
    packed, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.full((4, 4), 0x38, dtype=torch.uint8)
    scales[2:, 0] = 0x40
    packed[2, 0], packed[2, 8], packed[3, 0] = 0x07, 0x19, 0x06        # 6; -0.5, 0.5 of the second block; 4
    k, e = torch.full((2, 1, 64), 99, dtype=torch.int8), torch.full((2, 1), 99, dtype=torch.int8)
    k, e, other = S.page_keys(packed, scales, torch.tensor([[1, 0]]), [3], [0, 3], k, e, 2)
    assert torch.equal(k, other)
    # sums 20 and +-0.5, in units of 2^-10: 20480 (15 bits), 512; e = 8: 80, 2
    assert e.tolist() == [[99], [8]] and k[1, 0, 0] == 80 and k[1, 0, 16] == -2 and k[1, 0, 17] == 2 and k[1].abs().sum() == 84
    assert k[0].eq(99).all()


def test_selection_by_hand():
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    q[:, 0, 0], q[:, 1, 0] = 1.0, -1.0
    keys, e = torch.zeros(8, 1, 64, dtype=torch.int8), torch.zeros(8, 1, dtype=torch.int8)
    keys[:, 0, 0] = torch.tensor([5, -9, 9, 3, 7, 0, 1, 1])
    e[3] = 1                     # 3 * 2 = 6
    assert S.q8(q[0]) == [[64] + [0] * 63, [-64] + [0] * 63]
    table = torch.tensor([[0, 1, 2, 3, 4, 5, 6, 7]])
    # positions 27, 28 of 29 with pages of 4: own pages 6 and 7; scores |5| 9 9 6 7 0 1
    got = S.select_pages(q, keys, e, table, [29], [0, 2], 4, 3, 0, 1)
    assert got.tolist() == [[[1, 2, 4, 6]], [[1, 2, 4, 7]]]
    got = S.select_pages(q, keys, e, table, [29], [0, 2], 4, 1, 2, 2)
    assert got.tolist() == [[[0, 1, 2, 5, 6]], [[0, 1, 2, 6, 7]]]
    table[0, 1], table[0, 2] = -1, 8                      # hidden: 4, 3, 0 are left
    assert S.select_pages(q, keys, e, table, [29], [0, 2], 4, 3, 0, 1).tolist() == [[[0, 3, 4, 6]], [[0, 3, 4, 7]]]


def test_attention_by_hand():
    """One key and value a page: weights 1 : 2 for scores 0 and ln 2; a page twice."""
    packed, scales = torch.zeros(3, 32, dtype=torch.uint8), torch.full((3, 4), 0x38, dtype=torch.uint8)
    kp, vp = packed.clone(), packed.clone()
    kp[1, 0], vp[0, 0], vp[1, 0] = 0x02, 0x02, 0x04        # key 1; values 1 and 2
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    q[0, 0, 0] = 1.0
    run = lambda *p: S.sparse_attention(q, kp, scales, vp, scales, torch.tensor([[0, 1, 2]]), [2], [0, 1],  # noqa: E731
                                        torch.tensor([[p]]).view(1, 1, -1), 1, math.log(2))
    out, lse, _, _ = run(0, 1, 2, -1)
    assert math.isclose(out[0, 0, 0], 5 / 3) and math.isclose(lse[0, 0], math.log(3))
    out, lse, _, _ = run(1, 0, 0)
    assert math.isclose(out[0, 0, 0], 1.5) and math.isclose(lse[0, 0], math.log(4))
    out, lse, _, _ = run(2, 7)
    assert out.abs().sum() == 0 and lse[0, 0] == -math.inf
    assert np.isfinite(run(0)[2].numpy()).all()
