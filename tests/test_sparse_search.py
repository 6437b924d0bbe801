"""The search for the score that ends a list of pages (find_limit of
csrc/page_select.hip), compiled for the CPU from the kernel's own source: the lanes
of a workgroup are coroutines that take turns at every exchange and barrier. It has
to end, and to choose at most top_k pages, for any 32 bits in the place of a score,
and to choose the right ones for the scores that the kernels write."""
import os
import struct
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "moe_swiglu_epilogue_amd", "csrc", "page_select.hip")

DRIVER = r"""
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <ucontext.h>
#include <vector>
#define __device__
#define __forceinline__
static const int kMostLanes = 256;
static ucontext_t lanes[kMostLanes], home;
static char stacks[kMostLanes][1 << 16];
static int threads, now, left;
static long turns, most_turns;
static struct { unsigned x; } threadIdx;
static bool ends;

// every lane gets here before one goes on
static void sync()
{
    const int me = now;
    if (++turns > most_turns) {                 // the search does not end
        ends = false;
        swapcontext(&lanes[me], &home);
    }
    now = (me + 1) % threads;
    threadIdx.x = now;
    if (now != me)
        swapcontext(&lanes[me], &lanes[now]);
}
static uint32_t said[kMostLanes];
template <class F> static uint32_t over_wave(uint32_t v, F f)
{
    said[now] = v;
    sync();
    const uint32_t r = f(said + now / 64 * 64, now % 64);
    sync();
    return r;
}
static uint32_t sums_up_to_lane(uint32_t v)
{
    return over_wave(v, [](const uint32_t* x, int lane) { uint32_t s = 0; for (int i = 0; i <= lane; ++i) s += x[i]; return s; });
}
static uint32_t read_lane(uint32_t v, int of) { return over_wave(v, [=](const uint32_t* x, int) { return x[of & 63]; }); }
static uint32_t last_lane(uint32_t v) { return read_lane(v, 63); }
static uint32_t largest_of(uint32_t v)
{
    return over_wave(v, [](const uint32_t* x, int) { uint32_t s = 0; for (int i = 0; i < 64; ++i) s = x[i] > s ? x[i] : s; return s; });
}
static uint32_t smallest_of(uint32_t v)
{
    return over_wave(v, [](const uint32_t* x, int) { uint32_t s = ~0u; for (int i = 0; i < 64; ++i) s = x[i] < s ? x[i] : s; return s; });
}
static uint64_t __ballot(bool b)
{
    const uint32_t low = over_wave(b, [](const uint32_t* x, int) { uint32_t s = 0; for (int i = 0; i < 32; ++i) s |= x[i] << i; return s; });
    return low | (uint64_t)over_wave(b, [](const uint32_t* x, int) { uint32_t s = 0; for (int i = 0; i < 32; ++i) s |= x[32 + i] << i; return s; }) << 32;
}
static int __ffsll(long long v) { return __builtin_ffsll(v); }
#define __builtin_amdgcn_readlane(v, l) ((int)read_lane((uint32_t)(v), l))
#define __syncthreads sync
template <class T> static T min(T a, T b) { return b < a ? b : a; }
template <class T> static T max(T a, T b) { return a < b ? b : a; }
static uint32_t min(uint32_t a, unsigned long b) { return b < a ? (uint32_t)b : a; }
static uint32_t max(uint32_t a, int b) { return max(a, (uint32_t)b); }
static void atomicAdd(uint32_t* p, uint32_t v) { *p += v; }
static void atomicMin(uint32_t* p, uint32_t v) { *p = v < *p ? v : *p; }
static void atomicMax(uint32_t* p, uint32_t v) { *p = v > *p ? v : *p; }
static uint32_t __float_as_uint(float v) { uint32_t b; memcpy(&b, &v, 4); return b; }
static float __uint_as_float(uint32_t b) { float v; memcpy(&v, &b, 4); return v; }
// as the card converts: NaN is 0, the rest saturates
struct Whole {
    int v;
    Whole(float x) : v(x != x ? 0 : x >= 2147483648.0f ? INT32_MAX : x < -2147483648.0f ? INT32_MIN : (int)x) {}
    Whole(uint32_t x) : v((int)x) {}
    Whole(int x) : v(x) {}
    operator int() const { return v; }
};
typedef uint32_t uint4v __attribute__((ext_vector_type(4)));
//SOURCE
static std::vector<float> score;
static int first_page, top_k, wide;
static Limit got[kMostLanes];
alignas(16) static SelectShared<1> lds1[1];
alignas(16) static SelectShared<4> lds4;
template <int W, class Shared> static void lane(Shared& lds)
{
    const int me = now;
    got[me] = find_limit<W>(lds, score.data(), first_page, (int)score.size(), top_k);
    // a lane that is done waits here until all are
    ++left;
    while (left < threads)
        sync();
    swapcontext(&lanes[me], &home);
}
static void run1() { lane<1>(lds1[0]); }
static void run4() { lane<4>(lds4); }

// reads: lanes, first, top, count, the scores' bits; writes: ends, the limit's bits, ties
int main()
{
    int32_t head[4];
    while (fread(head, 4, 4, stdin) == 4) {
        threads = head[0];
        first_page = head[1];
        top_k = head[2];
        score.resize(head[3]);
        if (head[3] && fread(score.data(), 4, head[3], stdin) != (size_t)head[3])
            return 1;
        memset(&lds1, 0, sizeof lds1);
        memset(&lds4, 0, sizeof lds4);
        lds4.lo[0] = ~0u;
        now = left = 0;
        turns = 0;
        most_turns = 20000L * threads;
        ends = true;
        threadIdx.x = 0;
        for (int i = 0; i < threads; ++i) {
            getcontext(&lanes[i]);
            lanes[i].uc_stack.ss_sp = stacks[i];
            lanes[i].uc_stack.ss_size = sizeof stacks[i];
            lanes[i].uc_link = &home;
            makecontext(&lanes[i], threads == 64 ? run1 : run4, 0);
        }
        swapcontext(&home, &lanes[0]);
        uint32_t out[3] = {ends, __float_as_uint(got[0].limit), got[0].ties};
        for (int i = 1; ends && i < threads; ++i)
            if (memcmp(&got[i], &got[0], sizeof got[0]))
                out[0] = 2;                     // the lanes do not agree
        fwrite(out, 4, 3, stdout);
    }
    return 0;
}
"""


def between(text, start, end):
    at = text.index(start)
    return text[at:text.index(end, at)]


@pytest.fixture(scope="module")
def search(tmp_path_factory):
    from moe_swiglu_epilogue_amd import build as B
    text = open(SOURCE).read()
    code = (between(text, "__device__ __forceinline__ uint32_t ordered", "// op over the lanes")
            + between(text, "struct Limit {", "// Where a request's tokens stand"))
    code = code.replace('asm volatile("" ::: "memory")', "sync()").replace("#pragma unroll 1\n", "").replace("#pragma unroll\n", "")
    assert code.count("min((int)((v - lo) * scale), kBins - 1)") == 1
    code = code.replace("(int)((v - lo) * scale)", "(int)Whole((v - lo) * scale)")
    where = tmp_path_factory.mktemp("search")
    src, exe = where / "search.cpp", where / "search"
    src.write_text(DRIVER.replace("//SOURCE", code))
    clang = os.path.join(os.path.dirname(os.path.dirname(B.HIPCC)), "llvm", "bin", "clang++")
    subprocess.run([clang, "-std=c++17", "-O1", "-ffp-contract=off", "-w", str(src), "-o", str(exe)], check=True)

    def run(cases):
        """[(lanes, first, top, scores)] -> [(state, limit, ties)]."""
        text = b"".join(struct.pack("<4i", w, f, t, len(s)) + np.asarray(s, np.float32).tobytes() for w, f, t, s in cases)
        out = subprocess.run([str(exe)], input=text, stdout=subprocess.PIPE, check=True, timeout=300).stdout
        assert len(out) == 12 * len(cases)
        return [(e, struct.unpack("<f", struct.pack("<I", bits))[0], ties) for e, bits, ties in struct.iter_unpack("<3I", out)]
    return run


def chosen(scores, first, limit, ties):
    """The pages that a list takes: those above the limit, and the first ties."""
    s = np.asarray(scores, np.float32)[first:]
    same = np.flatnonzero((s == limit) & (s != -np.inf))
    return sorted(np.flatnonzero(s > limit).tolist() + same[:ties].tolist())


def test_the_scores_that_are_written(search):
    """Whole numbers times powers of two and hidden pages: the top largest, ties to the
    lower page."""
    r = np.random.default_rng(3)
    cases = []
    for _ in range(160):
        n, most, octaves = int(r.integers(1, 1500)), int(r.choice([2, 40, 10 ** 5, 127 * 127 * 256])), int(r.choice([0, 4, 64]))
        s = np.ldexp(r.integers(-most, most + 1, n).astype(np.float64), r.integers(0, octaves + 1, n)).astype(np.float32)
        s[r.random(n) < 0.1] = -np.inf
        cases.append((int(r.choice([64, 256])), int(r.integers(0, min(n, 5) + 1)), int(r.integers(0, n + 2)), s))
    for (w, first, top, s), (state, limit, ties) in zip(cases, search(cases)):
        t = s[first:]
        want = [j for j in np.argsort(-t.astype(np.float64), kind="stable") if t[j] != -np.inf][:top]
        assert state == 1 and chosen(s, first, limit, ties) == sorted(want), (w, first, top, len(s))


def special(kind, r, n):
    s = np.round(r.standard_normal(n) * 1e5).astype(np.float32)
    at = r.choice(n, min(n, 6), replace=False)
    if kind == "random bits":
        return r.integers(0, 2 ** 32, n, dtype=np.uint64).astype(np.uint32).view(np.float32)
    if kind == "tiny":
        return r.integers(0, 40, n).astype(np.uint32).view(np.float32)
    s[at] = {"one infinity": [math_inf] + s[at[1:]].tolist(), "infinities": [math_inf] * len(at),
             "far apart": [3e38, -3e38] * 3, "NaN": [math_nan, -math_nan] * 3,
             "all of them": [math_inf, -math_inf, math_nan, 3e38, -3e38, 1e-45]}[kind][:len(at)]
    return s


math_inf, math_nan = float("inf"), float("nan")


@pytest.mark.parametrize("kind", ["one infinity", "infinities", "far apart", "NaN", "all of them", "random bits", "tiny"])
def test_any_bits_end_and_stay_in_the_list(search, kind):
    r = np.random.default_rng(len(kind))
    cases = [(w, 1, top, special(kind, r, n)) for w in (64, 256) for n in (6, 70, 500, 1100) for top in (1, 7, 100, 499) if top < n]
    for (w, first, top, s), (state, limit, ties) in zip(cases, search(cases)):
        assert state == 1, (kind, w, len(s), top, "does not end" if state == 0 else "lanes differ")
        assert len(chosen(s, first, limit, ties)) <= top, (kind, w, len(s), top)
