"""How nvfp4_paged_attention cuts its work (csrc/attention_plan.hpp), on the
CPU: for every size and hint that the call takes, up to the types' largest, the
plan has at least one split, the splits of any range of tokens cover it
exactly once, no integer overflows (compiled with the undefined-behaviour
checks on) and the grids stay inside what a launch takes."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <stdio.h>
#include "attention_plan.hpp"
#define CHECK(e) do { if (!(e)) { printf("%s: tokens %lld heads %d/%d x %d seqs %lld hints %lld %lld window %lld: " \
    "splits %d chunk %d\n", #e, (long long)t, h[0], h[1], d, (long long)n, (long long)mq, (long long)ms, (long long)w, \
    p.splits, p.chunk); if (++bad > 20) return 1; } } while (0)

int main()
{
    const int64_t hints[] = {0, 1, 100, 2048, 131072, 8400000, (1 << 30) - 1, 1 << 30, (1 << 30) + 1, 2147483647LL - 300,
                             2147483647LL - 127, 2147483647LL, 1LL << 31, 1LL << 62, INT64_MAX};
    const int heads[][2] = {{1, 1}, {32, 8}, {64, 1}, {1024, 1024}, {96, 2}};
    const int64_t seqs[] = {0, 1, 3, 64, 4095, 65535}, calls[] = {0, 1, 70, 12288, 70000, 1 << 20};
    const int64_t queries[] = {0, 1, 5, 33, 4096, 1LL << 62}, windows[] = {0, 1, 1500, (1 << 30) - 1, 2147483647LL, INT64_MAX};
    const int begins[] = {0, 32, 160, 8388608, 8400000, (1 << 30) - 64, (1 << 30) - 32, 1 << 30};
    const int lengths[] = {0, 1, 127, 5000, 8400000, (1 << 29) + 77, 1 << 30};
    int bad = 0;
    long long plans = 0, ranges = 0;
    for (const auto& h : heads)
        for (int d : {64, 128, 256})
            for (int64_t n : seqs)
                for (int64_t t : calls)
                    for (int64_t mq : queries)
                        for (int64_t ms : hints)
                            for (int64_t w : windows) {
                                if (n * h[1] > (1 << 22) || t * h[0] > (1 << 30))
                                    continue;
                                const attention::Plan p = attention::make_plan(t, h[0], h[1], d, n, mq, ms, w);
                                ++plans;
                                CHECK(p.splits >= 1 && p.splits <= 256);
                                CHECK(p.chunk >= 128 && p.chunk % 128 == 0);
                                CHECK(p.row_blocks >= 1);
                                if (p.splits < 1 || p.chunk < 1)
                                    continue;
                                const int64_t work = n * p.row_blocks * p.splits;
                                CHECK((work + 7) / 8 * 8 * h[1] <= 1 << 23);
                                if (n != 1 && n != 65535)
                                    continue;
                                for (int begin : begins)
                                    for (int length : lengths) {
                                        if ((int64_t)begin + length > 1 << 30)
                                            continue;
                                        const int end = begin + length, chunk = attention::chunk_of(p.chunk, p.splits, length);
                                        int at = begin;
                                        for (int split = 0; split < p.splits; ++split) {
                                            const int first = begin + split * chunk;
                                            const int last = attention::last_of(first, chunk, end);
                                            if (first >= last)
                                                continue;
                                            CHECK(first == at && last > first);
                                            at = last;
                                        }
                                        CHECK(at == end);
                                        ++ranges;
                                    }
                            }
    printf("%lld plans, %lld ranges\n", plans, ranges);
    return bad != 0;
}
"""


def test_plans_cover_every_range(tmp_path):
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(ROOT, "moe_swiglu_epilogue_amd", "csrc"), "-I", os.path.join(ROOT, "include"),
                    "-I", "/opt/rocm/include", str(src), "-o", str(exe), "-L", "/opt/rocm/lib", "-lamdhip64",
                    "-Wl,-rpath,/opt/rocm/lib"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert int(r.stdout.split()[0]) > 10000, r.stdout
