"""Code generation checks on the gfx950 ISA of the decoding-step operators (CPU
only, as tests/test_codegen.py): matrix results are never read too early on
any path, no scalar memory writes, no packed FP32, and the walk that finds early
reads finds planted ones."""
import re

import pytest

import mfma_hazard as H
from test_codegen import _kernels


@pytest.fixture(scope="module")
def isa(tmp_path_factory):
    from moe_swiglu_epilogue_amd import build as B
    out = {}
    for src in (B.GEMM_SRC, *B.SERVING_SRCS):
        f = tmp_path_factory.mktemp("isa") / "k.s"
        B.asm(str(f), src)
        out[src] = f.read_text()
    return out


def test_matrix_results_are_not_read_early(isa):
    kernels = {n: b for text in isa.values() for n, b in _kernels(text).items()}
    assert sum(any(l.startswith("v_mfma") for l in b) for b in kernels.values()) >= 20
    bad = {n: H.early_uses(b)[:2] for n, b in kernels.items() if H.early_uses(b)}
    assert not bad, bad


def test_the_walk_finds_an_early_read_on_a_taken_branch():
    body = ["v_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]", "s_cbranch_scc1 .LBB0_1",
            "s_nop 7", "s_nop 7", ".LBB0_1:", "v_accvgpr_read_b32 v9, a2", "s_endpgm"]
    (mfma, use, waited), = H.early_uses(body)
    assert use[0] == "v_accvgpr_read_b32" and waited == 1
    body[1] = "s_nop 5"
    assert len(H.early_uses(body[:2] + body[4:])) == 1
    body[1] = "s_nop 6"
    assert H.early_uses(body[:2] + body[4:]) == []
    # the next instruction's accumulator is forwarded, its operand is not
    assert H.early_uses([body[0], body[0], "s_endpgm"]) == []
    assert len(H.early_uses([body[0], "v_mfma_f32_16x16x32_f16 a[4:7], a[0:3], v[4:7], 0", "s_endpgm"])) == 1


def test_no_scalar_memory_writes_and_no_packed_fp32(isa):
    for src, text in isa.items():
        assert not re.findall(r"\bs_(?:store|atomic|buffer_store|buffer_atomic|dcache_wb|scratch_store)\w*", text), src
        assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32", text), src
