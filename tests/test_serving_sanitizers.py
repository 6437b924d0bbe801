"""The host code of the decoding-step operators under AddressSanitizer and
UndefinedBehaviorSanitizer (host pass only; the device code is built as usual),
driven through the refusals and the workspace sizes of every entry point with the
types' extreme values. No call reaches a launch, so no GPU is needed."""
import os

import pytest

from test_sanitizers import ROOT, _run

DRIVER = r"""
#include <stdio.h>
#include <stdint.h>
#include "nvfp4_serving.h"
#define A ((void *)0x10000)
#define CHECK(e) do { if (!(e)) { printf("failed check at driver line %d\n", __LINE__); ++bad; } } while (0)
#define COUNT(a) ((int)(sizeof a / sizeof a[0]))
static const int64_t wide[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 17, 4096, 65535, 65536, 1 << 20, INT32_MAX - 127, INT32_MAX,
                               (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX / 4, INT64_MAX - 127, INT64_MAX};
static const int32_t narrow[] = {INT32_MIN, -1, 0, 1, 2, 16, 64, 100, 128, 256, 1024, 1 << 20, INT32_MAX};
static nvfp4_status_t attention(int64_t tokens, int32_t heads, int32_t kv, int32_t dim, int64_t slots, int32_t page, int64_t pages,
                                int64_t ld, int64_t seqs, int64_t mq, int64_t ms, int64_t window)
{
    /* a q that is never aligned: refused at the latest by that */
    return nvfp4_paged_attention((const uint16_t *)((char *)A + 2), tokens, ld, heads, kv, dim, A, A, A, A, slots, page, A, ld,
                                 pages, A, A, seqs, mq, ms, 1.0f, 1, window, NULL, NULL, A, ld, NULL, A, INT64_MAX, NULL);
}
int main(void) {
    int bad = 0;
    for (int i = 0; i < COUNT(wide); ++i)
        for (int j = 0; j < COUNT(wide); ++j) {
            for (int k = 0; k < COUNT(narrow); ++k)
                for (int l = 0; l < COUNT(narrow); ++l) {
                    int64_t n = moe_layer_workspace(wide[i], wide[j], wide[j], narrow[k], narrow[l]);
                    CHECK(n >= -1);
                    n = moe_layer_workspace(wide[i] & 63, wide[j] & ~31, 32 << (i & 15), narrow[k], narrow[l]);
                    CHECK(n >= -1);
                    n = nvfp4_paged_attention_workspace(wide[i], narrow[k], narrow[l], 128, wide[j], wide[(i + j) % COUNT(wide)],
                                                        wide[j], wide[(i + k) % COUNT(wide)]);
                    CHECK(n >= -1);
                    CHECK(attention(wide[i], narrow[k], narrow[l], 64, wide[j], narrow[(k + l) % COUNT(narrow)], wide[(i + l) % COUNT(wide)],
                                    wide[(j + k) % COUNT(wide)], wide[(i + j) % COUNT(wide)], wide[j], wide[i], wide[j])
                          != NVFP4_SUCCESS || wide[i] == 0 || wide[(i + j) % COUNT(wide)] == 0);
                    CHECK(moe_layer_bf16((const uint16_t *)((char *)A + 2), wide[i], wide[j], A, A, A, wide[(i + k) % COUNT(wide)] & ~31,
                                         wide[(j + l) % COUNT(wide)] & ~31, narrow[k], narrow[l], 1, A, wide[j], A, A, A, INT64_MAX, NULL)
                          != NVFP4_SUCCESS || wide[i] == 0);
                }
            /* hints and windows at the types' ends, for sizes that are taken */
            for (int k = 3; k < COUNT(wide); ++k)
                for (int dim = 64; dim <= 256; dim *= 2) {
                    if (wide[i] < 0 || wide[j] < 0)
                        continue;
                    CHECK(nvfp4_paged_attention_workspace(12288, 32, 8, dim, 3, wide[i], wide[j], wide[k]) >= 0);
                    CHECK(nvfp4_paged_attention_workspace(1, 32, 8, dim, 1, wide[i], wide[j], wide[k]) >= 0);
                    CHECK(nvfp4_paged_attention_workspace(1 << 20, 1024, 64, dim, 65535, wide[i], wide[j], wide[k]) >= 0);
                    CHECK(attention(70000, 64, 8, dim, 160, 16, 10, 1 << 16, 70, wide[i], wide[j], wide[k]) == NVFP4_ERROR_MISALIGNED);
                }
            for (int k = 0; k < COUNT(wide); ++k)
                for (int l = 0; l < COUNT(narrow); ++l)
                    CHECK(kv_block_tables((const int32_t *)((char *)A + 2), A, wide[i], narrow[l], A, wide[j], NULL, A, wide[k],
                                          wide[(i + k) % COUNT(wide)], A, A, A, wide[(j + k) % COUNT(wide)], A, NULL) != NVFP4_SUCCESS);
        }
    /* the comparison of memory: the table at the address space's end, lists of the largest sizes */
    char *end = (char *)(UINTPTR_MAX - 0xffff);
    CHECK(kv_block_tables(A, A, 4096, 16, (int32_t *)((char *)A + 0x100000), INT32_MAX, NULL, (int32_t *)end, 1, 1, (int32_t *)(end + 0x8000),
                          (int32_t *)((char *)A + 0x200000), A, INT32_MAX, (int32_t *)(end + 0x100), NULL) == NVFP4_ERROR_INVALID_VALUE);
    printf("serving sanitizer run: %d failures\n", bad);
    return bad != 0;
}
"""


@pytest.mark.slow
def test_serving_host_code_under_asan_ubsan(tmp_path):
    from moe_swiglu_epilogue_amd import build as B
    rocm = os.path.dirname(os.path.dirname(B.HIPCC))
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    lib = tmp_path / "libmoe_nvfp4_san.so"
    flags = [f for f in B.FLAGS if f != "-Wall"]
    host_san = [a for f in san for a in ("-Xarch_host", f)]
    _run([B.HIPCC, *flags, *host_san, "-I", os.path.join(ROOT, "include"), B.SRC, B.GEMM_SRC, *B.SERVING_SRCS, "-o", str(lib)])
    drv = tmp_path / "drv.c"
    drv.write_text(DRIVER)
    exe = tmp_path / "serving_san"
    _run([os.path.join(rocm, "llvm", "bin", "clang"), "-std=c11", *san, "-D__HIP_PLATFORM_AMD__",
          "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), str(drv), str(lib),
          "-L", os.path.join(rocm, "lib"), "-lamdhip64",
          "-Wl,-rpath," + str(tmp_path), "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", str(exe)])
    r = _run([str(exe)], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=120)
    assert "0 failures" in r.stdout
