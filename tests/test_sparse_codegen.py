"""Code generation checks on the gfx950 ISA of the sparse-attention operators (CPU
only, as tests/test_serving_codegen.py): matrix results are never read earlier
than straight-line code reads them, no scalar memory writes, no packed FP32."""
import re

import pytest

import mfma_hazard as H
from test_codegen import _kernels

# wait states behind the 8-bit products, as straight-line code keeps them (counted below)
KEPT = dict(H.KEPT, **{"16x16x64": 8})

PROBE = r"""
#include <hip/hip_runtime.h>
typedef int i4 __attribute__((ext_vector_type(4)));
__global__ void small_i8(const i4* a, const i4* b, int* out)
{
    const i4 c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[threadIdx.x], b[threadIdx.x], i4{}, 0, 0, 0);
    out[threadIdx.x] = c[0] + c[1];
}
"""


@pytest.fixture(scope="module")
def isa(tmp_path_factory):
    from moe_swiglu_epilogue_amd import build as B
    out = {}
    for src in B.SPARSE_SRCS:
        f = tmp_path_factory.mktemp("isa") / "k.s"
        B.asm(str(f), src)
        out[src] = f.read_text()
    return out


def test_wait_states_of_straight_line_code(tmp_path):
    from moe_swiglu_epilogue_amd import build as B
    src, out = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(PROBE)
    B.asm(str(out), str(src))
    (body,) = _kernels(out.read_text()).values()
    code = [l.split(";")[0].split() for l in body]
    code = [c for c in code if c and not c[0].startswith(".")]
    at = next(i for i, c in enumerate(code) if c[0].startswith("v_mfma"))
    result, waited = H._registers(code[at][1].rstrip(",")), 0
    for op, *rest in code[at + 1:]:
        if H._registers(" ".join(rest)) & result:
            break
        waited += 1 + int(rest[0]) if op == "s_nop" else 1
    assert "16x16x64" in code[at][0] and waited == KEPT["16x16x64"], waited


def test_matrix_results_are_not_read_early(isa):
    count = 0
    for text in isa.values():
        for name, body in _kernels(text).items():
            matrix = [l.split()[0] for l in body if l.startswith("v_mfma")]
            assert all(any(s in op for s in KEPT) for op in matrix), (name, set(matrix))
            assert not H.early_uses(body, KEPT), name
            count += len(matrix)
    assert count > 100


def test_no_scalar_memory_writes_and_no_packed_fp32(isa):
    for src, text in isa.items():
        assert not re.findall(r"\bs_(?:store|atomic|buffer_store|buffer_atomic|dcache_wb|scratch_store)\w*", text), src
        assert not re.findall(r"\bv_pk_(?:add|mul|fma)_f32", text), src
