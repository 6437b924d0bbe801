"""Static check of gfx950 assembly: no result of a matrix instruction is touched
too early, on any path.

A matrix instruction's result may be read (other than as the accumulator of
the same shape's next instruction) or overwritten by the vector unit or a
memory instruction only a number of wait states later; the hardware does not
wait, the compiler has to put other instructions or s_nop in between. Compiled
code has been seen to get this right on the path that falls through a branch
and wrong on the one that takes it. This walks all paths behind every matrix
instruction and counts wait states (one an instruction, n + 1 for s_nop n).
"""
import re

# wait states until the vector unit may read the result
# (v_mfma_f32_16x16x32 takes 16 clocks, v_mfma_f32_32x32x16 32). WAIT is one
# state too few for the first; KEPT is what the compiler keeps in straight-line
# code (tests/test_serving_hazards.py compiles some and counts).
WAIT = {"16x16x32": 7, "32x32x16": 12}
KEPT = {"16x16x32": 8, "32x32x16": 12}


def _registers(text):
    out = set()
    for kind, a, b, one in re.findall(r"\b([va])(?:\[(\d+):(\d+)\]|(\d+)\b)", text):
        lo, hi = (int(a), int(b)) if a else (int(one), int(one))
        out.update((kind, r) for r in range(lo, hi + 1))
    return out


def _parse(body):
    """Instructions (mnemonic, operands) and the successors of each."""
    code, labels = [], {}
    for l in body:
        l = l.split(";")[0].strip()
        if not l or l.startswith("."):
            m = re.match(r"(\.LBB\w+):", l)
            if m:
                labels[m.group(1)] = len(code)
            continue
        op, _, rest = l.partition(" ")
        code.append((op, rest.strip()))
    nexts = []
    for i, (op, rest) in enumerate(code):
        if op == "s_endpgm" or op == "s_setpc_b64":
            nexts.append([])
        elif op == "s_branch":
            nexts.append([labels[rest]])
        elif op.startswith("s_cbranch"):
            nexts.append([i + 1, labels[rest]])
        else:
            nexts.append([i + 1])
    return code, [[n for n in s if n < len(code)] for s in nexts]


def early_uses(body, wait=WAIT):
    """[(matrix instruction, use, wait states between)] of the hazards in one kernel."""
    code, nexts = _parse(body)
    bad = []
    for i, (op, rest) in enumerate(code):
        shape = next((s for s in wait if op.startswith("v_mfma") and s in op), None)
        if shape is None:
            continue
        result = _registers(rest.split(",")[0])
        todo, seen = [(n, 0) for n in nexts[i]], {}
        while todo:
            at, waited = todo.pop()
            if waited >= wait[shape] or seen.get(at, 99) <= waited:
                continue
            seen[at] = waited
            o, r = code[at]
            if o.startswith("v_mfma"):
                parts = re.split(r",\s*(?![^\[]*\])", r)
                # as the accumulator in and out it is forwarded
                if _registers(parts[1] + " " + parts[2]) & result:
                    bad.append(((op, rest), (o, r), waited))
                    continue
                if _registers(parts[0]) & result:
                    continue
            elif _registers(r) & result and o.startswith(("v_", "ds_", "buffer_", "global_", "scratch_", "flat_")):
                bad.append(((op, rest), (o, r), waited))
                continue
            step = 1 + int(r.split()[0]) if o == "s_nop" else 1
            todo += [(n, waited + step) for n in nexts[at]]
    return bad
