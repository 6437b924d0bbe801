"""The wait states behind matrix instructions (tests/mfma_hazard.py) as the
compiler keeps them in straight-line code for gfx950, and the built kernels
against those (CPU only)."""
import re

import mfma_hazard as H
from test_codegen import _kernels
from test_serving_codegen import isa  # noqa: F401

PROBE = r"""
#include <hip/hip_runtime.h>
typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef float f4 __attribute__((ext_vector_type(4)));
typedef float f16 __attribute__((ext_vector_type(16)));
#define PROBE(name, A, C, mfma) \
    extern "C" __global__ void name(const A* a, const A* b, float* out) \
    { \
        const C c = __builtin_amdgcn_##mfma(a[threadIdx.x], b[threadIdx.x], C{}, 0, 0, 0); \
        out[threadIdx.x] = c[0] * c[1]; \
    }
PROBE(small_f16, half8, f4, mfma_f32_16x16x32_f16)
PROBE(small_bf16, bf8, f4, mfma_f32_16x16x32_bf16)
PROBE(large_f16, half8, f16, mfma_f32_32x32x16_f16)
PROBE(large_bf16, bf8, f16, mfma_f32_32x32x16_bf16)
"""


def test_wait_states_of_straight_line_code(tmp_path):
    from moe_swiglu_epilogue_amd import build as B
    src, out = tmp_path / "probe.hip", tmp_path / "probe.s"
    src.write_text(PROBE)
    B.asm(str(out), str(src))
    found = set()
    for body in re.findall(r"^(?:small|large)_\w+:[^\n]*\n(.*?)^\.Lfunc_end", out.read_text(), re.M | re.S):
        code = [l.split(";")[0].split() for l in body.split("\n") if l.startswith("\t") and not l.strip().startswith((".", ";"))]
        code = [c for c in code if c]
        at = next(i for i, c in enumerate(code) if c[0].startswith("v_mfma"))
        result = H._registers(code[at][1].rstrip(","))
        shape = next(s for s in H.KEPT if s in code[at][0])
        waited = 0
        for op, *rest in code[at + 1:]:
            if H._registers(" ".join(rest)) & result:
                break
            waited += 1 + int(rest[0]) if op == "s_nop" else 1
        assert waited == H.KEPT[shape], (shape, waited, body)
        found.add(code[at][0])
    assert len(found) == 4, found


def test_matrix_results_are_read_no_earlier_than_straight_line_code_does(isa):  # noqa: F811
    count = 0
    for text in isa.values():
        for name, body in _kernels(text).items():
            matrix = [l.split()[0] for l in body if l.startswith("v_mfma")]
            assert all(any(s in op for s in H.KEPT) for op in matrix), (name, set(matrix))
            assert not H.early_uses(body, H.KEPT), name
            count += len(matrix)
    assert count > 1000


def test_the_walk_finds_a_read_one_state_early():
    mfma = "v_mfma_f32_16x16x32_f16 v[0:3], v[8:11], v[12:15], v[0:3]"
    read = "v_mul_f32_e32 v9, v1, v2"
    assert len(H.early_uses([mfma, "s_nop 6", read, "s_endpgm"], H.KEPT)) == 1
    assert H.early_uses([mfma, "s_nop 7", read, "s_endpgm"], H.KEPT) == []
    mfma = "v_mfma_f32_32x32x16_f16 v[0:15], v[16:19], v[20:23], v[0:15]"
    assert len(H.early_uses([mfma, "s_nop 7", "s_nop 2", read, "s_endpgm"], H.KEPT)) == 1
    assert H.early_uses([mfma, "s_nop 7", "s_nop 3", read, "s_endpgm"], H.KEPT) == []
