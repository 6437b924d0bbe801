"""The host code of the sparse-attention operators under AddressSanitizer and
UndefinedBehaviorSanitizer (host pass only; the device code is built as usual),
driven through the refusals and the workspace sizes of every entry point with the
types' extreme values. No call reaches a launch, so no GPU is needed."""
import os

import pytest

from test_sanitizers import ROOT, _run

DRIVER = r"""
#include <stdio.h>
#include <stdint.h>
#include "nvfp4_sparse.h"
#define A ((void *)0x10000)
#define U ((const uint16_t *)((char *)A + 2))      /* never aligned: refused at the latest by that */
#define CHECK(e) do { if (!(e)) { printf("failed check at driver line %d\n", __LINE__); ++bad; } } while (0)
#define COUNT(a) ((int)(sizeof a / sizeof a[0]))
static const int64_t wide[] = {INT64_MIN, INT64_MIN + 1, -1, 0, 1, 17, 4096, 65535, 65536, 1 << 20, INT32_MAX - 127, INT32_MAX,
                               (int64_t)INT32_MAX + 1, (int64_t)1 << 40, INT64_MAX / 4, INT64_MAX - 127, INT64_MAX};
static const int32_t narrow[] = {INT32_MIN, -1, 0, 1, 2, 16, 64, 100, 128, 256, 1024, 1 << 20, INT32_MAX};
#define W(x) wide[(x) % COUNT(wide)]
#define N(x) narrow[(x) % COUNT(narrow)]
int main(void) {
    int bad = 0;
    for (int i = 0; i < COUNT(wide); ++i)
        for (int j = 0; j < COUNT(wide); ++j)
            for (int k = 0; k < COUNT(narrow); ++k)
                for (int l = 0; l < COUNT(narrow); ++l) {
                    CHECK(nvfp4_select_pages_workspace(W(i), N(k), N(l), W(j), W(i + j + k)) >= -1);
                    CHECK(nvfp4_select_pages_workspace(W(i) & 4095, 64, 8, W(j) & 1023, W(k + l) & 32767) >= 0);
                    CHECK(nvfp4_sparse_attention_workspace(W(i), N(k), N(l), 128, N(i + j), W(j), W(j + l)) >= -1);
                    CHECK(nvfp4_sparse_attention_workspace(W(i) & 4095, 32, 8, 64 << (k % 3), N(l) & 0x7ffff, W(j) & 1023, W(k + l) & 2047) >= -1);
                    CHECK(nvfp4_rope_append(U, W(i), W(j), N(k), A, W(j + l), A, W(k), N(l), N(k + l + 1), A, W(i + k), N(i), A, A, W(l),
                                            N(j), k & 1, NULL, NULL, A, W(j + k), A, A, A, A, A, W(j), NULL)
                          != NVFP4_SUCCESS || W(i) == 0);
                    CHECK(nvfp4_rope_append(U, W(i), W(j) & ~7, 32, A, W(j) & ~7, A, W(j) & ~7, 8, 128, A, W(l), 1 + (k & 15), A, A, W(k), 128, 0,
                                            NULL, NULL, A, W(i + j), A, A, A, A, A, W(j) & ~7, NULL)
                          != NVFP4_SUCCESS || W(i) == 0);
                    CHECK(nvfp4_page_keys((const uint8_t *)U, A, W(i), N(k), 64 << (l % 4), N(l), A, W(j), W(i + l), A, A, W(j + k), W(k), A, A, NULL)
                          != NVFP4_SUCCESS || W(i) == 0 || W(i + l) == 0 || W(j + k) == 0);
                    CHECK(nvfp4_page_keys((const uint8_t *)U, A, 4096, 8, 128, 16, A, W(j), W(i), A, A, W(k + l), W(l), A, A, NULL)
                          != NVFP4_SUCCESS || W(i) == 0 || W(k + l) == 0);
                    CHECK(nvfp4_select_pages(U, W(i), W(j), N(k), N(l), 64 << (k % 4), A, A, W(i + k), N(i + l), A, W(j + l), W(l), A, A, W(k),
                                             N(i), N(j), N(i + j), A, A, W(i + j), NULL)
                          != NVFP4_SUCCESS || W(i) == 0 || W(k) == 0);
                    CHECK(nvfp4_select_pages(U, 1 + (W(i) & 1023), 4096, 32, 8, 128, A, A, 4096, 16, A, 4096, W(j) & 4095, A, A, 1 + (W(k) & 255),
                                             N(k), N(l), N(k + l), A, A, W(l), NULL) != NVFP4_SUCCESS);
                    CHECK(nvfp4_sparse_attention(U, W(i), W(j), N(k), N(l), 64 << (k % 4), A, A, A, A, W(i + k), N(i + l), A, W(j + l), W(l), A,
                                                 A, W(k), A, W(j + k), 1.0f, NULL, NULL, A, W(j), NULL, A, W(i + j), NULL)
                          != NVFP4_SUCCESS || W(i) == 0 || W(k) == 0);
                    CHECK(nvfp4_sparse_attention(U, 1 + (W(i) & 1023), 4096, 32, 8, 128, A, A, A, A, 4096, 16, A, 4096, W(j) & 4095, A, A,
                                                 1 + (W(k) & 255), A, W(l) & 2047, 1.0f, NULL, NULL, A, 4096, NULL, A, W(k + l), NULL)
                          != NVFP4_SUCCESS);
                }
    /* the comparison of memory at the address space's end */
    char *end = (char *)(UINTPTR_MAX - 0xffff);
    CHECK(nvfp4_rope_append(A, 4, 4096, 32, A, 4096, A, 4096, 8, 128, A, 4, 1, NULL, A, 8, 128, 0, NULL, NULL, A, INT32_MAX,
                            (uint8_t *)end, A, (uint8_t *)end, A, (uint16_t *)(end + 0x8000), 4096, NULL) == NVFP4_ERROR_INVALID_VALUE);
    printf("sparse sanitizer run: %d failures\n", bad);
    return bad != 0;
}
"""


@pytest.mark.slow
def test_sparse_host_code_under_asan_ubsan(tmp_path):
    from moe_swiglu_epilogue_amd import build as B
    rocm = os.path.dirname(os.path.dirname(B.HIPCC))
    san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    lib = tmp_path / "libmoe_nvfp4_san.so"
    flags = [f for f in B.FLAGS if f != "-Wall"]
    host_san = [a for f in san for a in ("-Xarch_host", f)]
    _run([B.HIPCC, *flags, *host_san, "-I", os.path.join(ROOT, "include"), B.SRC, B.GEMM_SRC, *B.SERVING_SRCS, *B.SPARSE_SRCS,
          "-o", str(lib)])
    drv = tmp_path / "drv.c"
    drv.write_text(DRIVER)
    exe = tmp_path / "sparse_san"
    _run([os.path.join(rocm, "llvm", "bin", "clang"), "-std=c11", *san, "-D__HIP_PLATFORM_AMD__",
          "-I", os.path.join(rocm, "include"), "-I", os.path.join(ROOT, "include"), str(drv), str(lib),
          "-L", os.path.join(rocm, "lib"), "-lamdhip64",
          "-Wl,-rpath," + str(tmp_path), "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", str(exe)])
    r = _run([str(exe)], env=dict(os.environ, ASAN_OPTIONS="detect_leaks=0"), timeout=120)
    assert "0 failures" in r.stdout
