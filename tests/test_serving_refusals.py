"""What the decoding-step operators (include/nvfp4_serving.h) refuse, on the
host: fake addresses, no call here may pass the checks."""
import os

import pytest

INVALID = 1
A = 0x100000      # fake "device" addresses, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from moe_swiglu_epilogue_amd import binding, build, serving
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return serving.raw()


SEQS, FREE, TOKENS, LD, WIDTH = 6, 40, 30, 24, 9
PLACES = dict(context=(0x0000, 4 * SEQS), query=(0x1000, 4 * SEQS), free=(0x2000, 4 * FREE), begin=(0x3000, 4),
              table=(0x4000, 4 * LD * (SEQS - 1) + 4 * WIDTH), offsets=(0x5000, 4 * SEQS + 4), lens=(0x6000, 4 * SEQS),
              slots=(0x7000, 8 * TOKENS), end=(0x8000, 4))


def call(lib, **moved):
    at = {n: A + moved.get(n, p) for n, (p, _) in PLACES.items()}
    return lib.kv_block_tables(at["context"], at["query"], SEQS, 16, at["free"], FREE, at["begin"], at["table"], LD, WIDTH,
                               at["offsets"], at["lens"], at["slots"], TOKENS, at["end"], None)


@pytest.mark.parametrize("out", ["offsets", "lens", "slots", "end", "table"])
@pytest.mark.parametrize("other", list(PLACES))
def test_block_tables_refuses_shared_memory(lib, out, other):
    """An output over an input or another output: from the same address, and by one
    element at either end."""
    if out == other:
        return
    (at, size), n = PLACES[other], PLACES[out][1]
    step = 8 if "slots" in (out, other) else 4
    for place in (at, at + size // step * step - step, at - (n // step * step - step)):
        assert call(lib, **{out: place}) == INVALID, (out, other, place - at)


def test_block_tables_refuses_outputs_over_any_row_of_the_table(lib):
    table = PLACES["table"][0]
    for row in range(SEQS):
        for col in (0, WIDTH - 1):
            assert call(lib, end=table + 4 * (row * LD + col)) == INVALID, (row, col)
    assert call(lib, slots=table + 4 * (LD - 4)) == INVALID          # begins in a gap, ends in the next row
