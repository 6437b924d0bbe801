"""The decoding-step operators on the host, no GPU needed: the header and the
exports agree, bad arguments are refused with the documented status before
any HIP call, the workspace sizes, and the plain definitions of the GPU tests
against hand-worked values."""
import math
import os
import re
import subprocess

import pytest
import torch

import serving_ref as R

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "nvfp4_serving.h")
OK, INVALID, SHAPE, MISALIGNED = 0, 1, 2, 3
A = 0x10000      # a fake aligned "device" address, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from moe_swiglu_epilogue_amd import binding, build, serving
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return serving.raw()


def test_header_and_exports_agree(lib):
    from moe_swiglu_epilogue_amd import binding, serving
    names = set(re.findall(r"^(?:nvfp4_status_t|int64_t)\s+(\w+)\s*\(", open(HEADER).read(), re.M))
    assert names == set(serving.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(l.split()[-1] for l in out.splitlines() if " T " in l)


def test_header_compiles_as_c(tmp_path):
    src = tmp_path / "t.c"
    src.write_text('#include "nvfp4_serving.h"\nint main(void){return (int)NVFP4_SUCCESS;}\n')
    subprocess.run(["gcc", "-std=c11", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", "-c", str(src), "-o", str(tmp_path / "t.o")], check=True)


def bt(lib, c=A, q=A, n=4, page=16, free=A, nf=8, begin=None, table=A, ld=8, mp=8, off=A, lens=A, slots=A, mt=9, end=A):
    return lib.kv_block_tables(c, q, n, page, free, nf, begin, table, ld, mp, off, lens, slots, mt, end, None)


def test_block_tables_validation(lib):
    for bad in (dict(n=-1), dict(page=0), dict(page=-4), dict(nf=-2), dict(mp=-1, ld=0), dict(mt=-1), dict(ld=7),
                dict(q=None), dict(table=None), dict(off=None), dict(lens=None), dict(slots=None), dict(end=None),
                dict(free=None), dict(ld=2 ** 62)):
        assert bt(lib, **bad) == INVALID, bad
    for bad in (dict(n=4097), dict(nf=2 ** 31), dict(mp=2 ** 31, ld=2 ** 31), dict(mt=2 ** 31)):
        assert bt(lib, **bad) == SHAPE, bad
    for name in ("c", "q", "free", "begin", "table", "off", "lens", "end"):
        assert bt(lib, **{name: A + 2}) == MISALIGNED, name
    assert bt(lib, slots=A + 4) == MISALIGNED


def at(lib, q=A, tokens=4, ld_q=1024, heads=8, kv=2, dim=128, kp=A, ks=A, vp=A, vs=A, ns=160, page=16, table=A, ld_t=8,
       mp=8, lens=A, off=A, n=2, mq=2, ms=100, scale=0.1, causal=1, window=0, kg=None, vg=None, out=A, ld_o=1024, lse=None,
       ws=A, wb=2 ** 40):
    return lib.nvfp4_paged_attention(q, tokens, ld_q, heads, kv, dim, kp, ks, vp, vs, ns, page, table, ld_t, mp, lens, off,
                                     n, mq, ms, scale, causal, window, kg, vg, out, ld_o, lse, ws, wb, None)


def test_attention_validation(lib):
    for bad in (dict(tokens=-1), dict(heads=0), dict(heads=7), dict(kv=0), dict(kv=-2), dict(ns=-16), dict(ns=161),
                dict(page=0), dict(mp=-1), dict(ld_t=7), dict(n=-1), dict(mq=-1), dict(ms=-1), dict(window=-1),
                dict(scale=math.nan), dict(ld_q=1016), dict(ld_o=1016), dict(ld_q=2 ** 62), dict(ld_o=2 ** 62),
                dict(ld_t=2 ** 62), dict(q=None), dict(out=None), dict(lens=None), dict(off=None), dict(table=None),
                dict(kp=None), dict(ks=None), dict(vp=None), dict(vs=None), dict(wb=-1), dict(scale=math.inf),
                dict(n=1, ms=2 ** 20, mq=1, tokens=1, wb=0), dict(n=1, ms=2 ** 20, mq=1, tokens=1, ws=None)):
        assert at(lib, **bad) == INVALID, bad
    for bad in (dict(dim=96, ld_q=2048, ld_o=2048), dict(dim=512, ld_q=8192, ld_o=8192), dict(dim=0),
                dict(heads=2048, kv=1, ld_q=2 ** 19, ld_o=2 ** 19), dict(n=65536), dict(tokens=2 ** 31), dict(ns=2 ** 31),
                dict(tokens=2 ** 27 + 1),
                dict(mp=2 ** 30 // 16 + 1, ld_t=2 ** 31)):
        assert at(lib, **bad) == SHAPE, bad
    for bad in (dict(q=A + 8), dict(out=A + 8), dict(ld_q=1028), dict(ld_o=1028), dict(kp=A + 8), dict(vp=A + 8),
                dict(ks=A + 4), dict(vs=A + 4), dict(table=A + 2), dict(lens=A + 2), dict(off=A + 2), dict(kg=A + 2),
                dict(vg=A + 2), dict(lse=A + 2), dict(ws=A + 8)):
        assert at(lib, **bad) == MISALIGNED, bad
    # nothing to do succeeds without a launch
    assert at(lib, tokens=0, q=None, out=None) == OK
    assert at(lib, n=0, lens=None, off=None, table=None) == OK


def test_attention_workspace(lib):
    f = lib.nvfp4_paged_attention_workspace
    assert f(-1, 8, 2, 128, 1, 1, 1, 0) == -1 and f(1, 8, 3, 128, 1, 1, 1, 0) == -1 and f(1, 8, 2, 96, 1, 1, 1, 0) == -1
    assert f(0, 8, 2, 128, 0, 0, 0, 0) == 0
    long = f(1, 32, 8, 128, 1, 1, 131072, 0)
    assert 0 < long < 2 ** 28                  # a split context needs room
    assert f(1, 32, 8, 128, 1, 1, 131072, 100) <= long
    assert f(8192, 32, 8, 128, 4, 2048, 2048, 0) < 2 ** 31
    # the largest window and hints stand for no limit
    assert f(1, 32, 8, 128, 1, 2 ** 62, 131072, 2 ** 63 - 1) == f(1, 32, 8, 128, 1, 2 ** 62, 131072, 0)
    assert f(1, 32, 8, 128, 1, 1, 131072, 2 ** 63 - 1) == long


def mo(lib, fp4, x=A, tokens=4, ld_x=128, logits=A, w1=A, s1=A, g1=None, w2=A, s2=A, g2=None, hidden=128, inter=64, e=8,
       k=2, out=A, ld_o=128, ids=A, w=A, ws=A, wb=2 ** 40):
    if fp4:
        return lib.moe_layer_nvfp4(x, tokens, ld_x, logits, w1, s1, g1, w2, s2, g2, hidden, inter, e, k, 1, out, ld_o, ids,
                                   w, ws, wb, None)
    return lib.moe_layer_bf16(x, tokens, ld_x, logits, w1, w2, hidden, inter, e, k, 1, out, ld_o, ids, w, ws, wb, None)


@pytest.mark.parametrize("fp4", [True, False])
def test_moe_validation(lib, fp4):
    for bad in (dict(tokens=-1), dict(hidden=-32), dict(inter=-32), dict(e=0), dict(k=0), dict(k=9), dict(ld_x=120),
                dict(ld_o=120), dict(ld_x=2 ** 62), dict(x=None), dict(logits=None), dict(w1=None), dict(w2=None),
                dict(out=None), dict(ids=None), dict(w=None), dict(ws=None), dict(wb=15)):
        assert mo(lib, fp4, **bad) == INVALID, bad
    for bad in (dict(tokens=65), dict(hidden=0), dict(inter=0), dict(hidden=48), dict(inter=48), dict(e=513),
                dict(e=100, k=33), dict(hidden=2 ** 21, ld_x=2 ** 21, ld_o=2 ** 21), dict(inter=2 ** 21)):
        assert mo(lib, fp4, **bad) == SHAPE, bad
    for bad in (dict(x=A + 8), dict(out=A + 8), dict(ld_x=132), dict(ld_o=132), dict(w1=A + 8), dict(w2=A + 8),
                dict(logits=A + 2), dict(ids=A + 2), dict(w=A + 2), dict(ws=A + 8)):
        assert mo(lib, fp4, **bad) == MISALIGNED, bad
    if fp4:
        assert mo(lib, fp4, s1=None) == INVALID and mo(lib, fp4, s2=None) == INVALID
        for name in ("s1", "s2"):
            assert mo(lib, fp4, **{name: A + 1}) == MISALIGNED
        for name in ("g1", "g2"):
            assert mo(lib, fp4, **{name: A + 2}) == MISALIGNED
    assert mo(lib, fp4, tokens=0, x=None, logits=None, out=None) == OK


def test_moe_workspace(lib):
    f = lib.moe_layer_workspace
    assert f(65, 128, 64, 8, 2) == -1 and f(1, 128, 64, 8, 9) == -1 and f(1, 40, 64, 8, 1) == -1
    assert f(0, 128, 64, 8, 2) >= 0
    assert 0 < f(1, 128, 64, 8, 2) <= f(64, 128, 64, 8, 2) < 2 ** 28


def test_binding_rejects_host_tensors_and_wrong_types():
    import moe_swiglu_epilogue_amd as M
    i = torch.zeros(2, dtype=torch.int32)
    u = torch.zeros(32, 128, dtype=torch.uint8)
    with pytest.raises(TypeError):
        M.kv_block_tables(i, i, torch.zeros(2, 4, dtype=torch.int32), 16, 8)
    with pytest.raises(TypeError):
        M.nvfp4_paged_attention(torch.zeros(2, 4, 128, dtype=torch.bfloat16), u, u, u, u, torch.zeros(2, 4, dtype=torch.int32),
                                i, torch.zeros(3, dtype=torch.int32), kv_heads=2, page_size=16, max_query_len=1)
    x, z = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(2, 4)
    with pytest.raises(TypeError):
        M.moe_layer_bf16(x, z, torch.zeros(4, 128, 64, dtype=torch.bfloat16), torch.zeros(4, 64, 64, dtype=torch.bfloat16), 2)
    with pytest.raises(TypeError):
        M.moe_layer_nvfp4(x, z, u, u, u, u, 2)


# ---- the plain definitions, against hand-worked values --------------------------------
def test_reference_block_tables():
    table = [[5, -1, -1], [-1, -1, -1]]
    got = R.kv_block_tables([3, 0], [2, 5], table, 4, 9, [7, 8, 9])
    assert table == [[5, 7, -1], [8, 9, -1]]
    assert got == ([23, 28, 32, 33, 34, 35, 36, -1, -1], [0, 2, 7], [5, 5], 3)


def test_reference_attention_against_a_library_product():
    g = torch.Generator().manual_seed(1)
    kp, ks = R.random_nvfp4(g, 16, 128)
    vp, vs = R.random_nvfp4(g, 16, 128)
    q = torch.randn(3, 4, 64, generator=g).to(torch.bfloat16)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    lens, offsets = torch.tensor([11]), torch.tensor([0, 3])
    out, lse, tol, _ = R.paged_attention(q, kp, ks, vp, vs, table, lens, offsets, 2, 4, 0.1)
    slot = torch.tensor([8, 9, 10, 11, 0, 1, 2, 3, 4, 5, 6])
    k = R.nvfp4_values(kp[slot], ks[slot]).view(11, 2, 64).repeat_interleave(2, 1).transpose(0, 1)
    v = R.nvfp4_values(vp[slot], vs[slot]).view(11, 2, 64).repeat_interleave(2, 1).transpose(0, 1)
    mask = torch.ones(3, 11, dtype=torch.bool).tril(8)
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), k, v, mask, scale=0.1)
    assert torch.allclose(out, want.transpose(0, 1), rtol=1e-12, atol=1e-12)
    assert (tol > 2.0 ** -9 * out.abs()).all() and (tol < 0.02 * v.abs().max()).all()


def test_reference_route_and_layer():
    ids, w = R.route(torch.tensor([[1.0, 3.0, 3.0, math.nan], [-math.inf, 0.0, -math.inf, -math.inf]]), 2, True)
    assert ids.tolist() == [[1, 2], [1, -1]] and w.tolist() == [[0.5, 0.5], [1.0, 0.0]]
    x = torch.tensor([[1.0, 2.0] + [0.0] * 30]).to(torch.bfloat16)
    w1 = torch.zeros(1, 16, 32, dtype=torch.float64)
    w1[0, 0, 0], w1[0, 8, 1] = 1.0, 1.5            # gate 0 = 1, up 0 = 3
    w2 = torch.zeros(1, 32, 8, dtype=torch.float64)
    w2[0, 5, 0] = 2.0
    out, tol, _, _ = R.moe_layer(x, torch.zeros(1, 1), w1, w2, 1, True, 0.0)
    assert abs(float(out[0, 5]) - 6.0 / (1 + math.exp(-1))) < 1e-12 and float(out.abs().sum()) == float(out[0, 5])
    assert float(tol[0, 5]) < 2.0 ** -7 * float(out[0, 5])
