"""Code generation checks on the gfx950 ISA of the sparse-attention operators (CPU
only, as tests/test_serving_codegen.py): matrix results are never read earlier
than straight-line code reads them, no scalar memory writes, no packed FP32."""
import re

import pytest

import mfma_hazard as H
from test_codegen import _kernels


@pytest.fixture(scope="module")
def isa(tmp_path_factory):
    from moe_swiglu_epilogue_amd import build as B
    out = {}
    for src in B.SPARSE_SRCS:
        f = tmp_path_factory.mktemp("isa") / "k.s"
        B.asm(str(f), src)
        out[src] = f.read_text()
    return out


def test_matrix_results_are_not_read_early(isa):
    count = 0
    for text in isa.values():
        for name, body in _kernels(text).items():
            matrix = [l.split()[0] for l in body if l.startswith("v_mfma")]
            assert all(any(s in op for s in H.KEPT) for op in matrix), (name, set(matrix))
            assert not H.early_uses(body, H.KEPT), name
            count += len(matrix)
    assert count > 100


def test_no_scalar_memory_writes_and_no_packed_fp32(isa):
    for src, text in isa.items():
        assert not re.findall(r"\bs_(?:store|atomic|buffer_store|buffer_atomic|dcache_wb|scratch_store)\w*", text), src
        assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32", text), src
