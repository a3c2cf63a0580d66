"""The wait states between a matrix instruction and what reads or overwrites its result, in the library's own machine
code.  The hardware does not look after them, and the compiler can miss a short way there: out of a loop that ends behind
a product it counted the longer one, and the last registers were read too early, the same wrong values every time.  Needs
the disassembler that comes with hipcc, no GPU."""
from __future__ import annotations

import re

import pytest

pytest.importorskip("torch")
from test_machine_code_cpu import kernels  # noqa: E402, F401

PASSES = {"4x4x4": 2, "16x16x4": 8, "16x16x16": 4, "16x16x32": 4, "16x16x128": 8, "32x32x2": 16, "32x32x8": 8, "32x32x16": 8,
          "32x32x64": 16}


def registers(operand):
    """(file, first, last) of a vector operand, or None"""
    m = re.match(r"[-|]*([va])(?:(\d+)|\[(\d+):(\d+)\])", operand)
    return m and (m[1], int(m[2] or m[3]), int(m[2] or m[4]))


def meet(a, b):
    return a is not None and b is not None and a[0] == b[0] and a[1] <= b[2] and b[1] <= a[2]


def needed(op):
    """Wait states until a vector instruction may touch the result (3 beyond the passes and one more on this chip, products of
    fp32 values 2), and until a product may add to a part of it."""
    sizes, inputs = re.match(r"v_mfma_(?:scale_)?\w+?_(\d+x\d+x\d+)_?(\w*)", op).groups()
    p = PASSES[sizes]
    if inputs == "f32":
        return p + 2, p + 2
    return p + 3 + (p != 2), p + 1 + (p != 2)


def early(code):
    """(matrix instruction, the one that comes too early, wait states between them)"""
    place = {at: n for n, (at, _) in enumerate(code)}
    ops = [text.split(None, 1)[0] for _, text in code]
    args = [[a.strip() for a in (text.split(None, 1)[1] if " " in text else "").split(",")] for _, text in code]
    for n, op in enumerate(ops):
        if not op.startswith("v_mfma"):
            continue
        result = registers(args[n][0])
        most, part = needed(op)
        fewest, ways = {}, [(n + 1, 0)]
        while ways:
            k, states = ways.pop()
            if k >= len(code) or states >= most or fewest.get(k, most) <= states:
                continue
            fewest[k] = states
            o, a = ops[k], args[k]
            if o.startswith("v_mfma"):
                hit = any(meet(result, registers(x)) for x in a[1:3])
                c = registers(a[3])
                if c == result and not hit:
                    continue                             # the sum goes on: that one's result now
                hit |= meet(result, c) and states < part
            elif o.startswith("v_"):
                hit = any(meet(result, registers(x)) for x in a)
            elif o.startswith(("ds_", "buffer_", "global_", "scratch_", "flat_")):
                loads = ("load" in o or "read" in o) and not code[k][1].endswith(" lds")
                hit = any(meet(result, registers(x)) for x in a[loads:])
            else:
                hit = False
            if hit:
                yield code[n][1], code[k][1], states
                break
            if o == "s_endpgm":
                continue
            after = states + (int(a[0], 0) + 1 if o == "s_nop" else 1)
            if m := re.match(r"s_c?branch", o):
                words = int(a[0])
                to = place.get(code[k][0] + 4 + 4 * (words - 65536 if words >= 32768 else words))
                if to is not None:
                    ways.append((to, after))
            if o != "s_branch":
                ways.append((k + 1, after))


def test_results_of_matrix_instructions_are_not_touched_early(kernels):  # noqa: F811
    products, bad = 0, []
    for name, code in kernels.items():
        products += sum(op.startswith("v_mfma") for _, op in code)
        bad += [(name[:60], *b) for b in early(code)]
    assert products > 1000
    assert not bad, f"{len(bad)} of {products}: {bad[:3]}"


# the shape in which it was seen: behind a product a branch to the loop's end, taken after four instructions
SEEN = ["v_mfma_f32_32x32x16_bf16 v[0:15], v[68:71], v[64:67], v[0:15]", "s_mov_b32 s3, 1", "s_andn2_b64 vcc, exec, s[0:1]",
        "s_cbranch_vccz 3", "s_lshl_b32 s4, s3, 5", "s_nop 9", "s_nop 0", "v_mov_b64_e32 v[126:127], v[14:15]", "s_endpgm"]


@pytest.mark.parametrize("change,found", [({}, 1), ({1: "s_nop 8"}, 1), ({1: "s_nop 9"}, 0), ({7: "v_mov_b64_e32 v[126:127], v[16:17]"}, 0),
                                          ({7: "v_mov_b32_e32 v15, 0"}, 1), ({7: "ds_write_b32 v90, v3"}, 1),
                                          ({7: "ds_read_b32 v3, v90"}, 0), ({3: "s_nop 0"}, 0),
                                          ({1: "v_mfma_f32_32x32x16_bf16 v[0:15], v[68:71], v[64:67], v[0:15]"}, 1),
                                          ({7: "v_mfma_f32_32x32x16_bf16 v[16:31], v[8:11], v[64:67], v[16:31]"}, 1)])
def test_the_search_itself(change, found):
    text = [change.get(n, op) for n, op in enumerate(SEEN)]
    assert len(list(early([(4 * n, op) for n, op in enumerate(text)]))) == found
