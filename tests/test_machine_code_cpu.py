"""The library's own machine code, where the compiler does not look after it: the
HBM -> LDS copies are issued from inline asm, so neither the wait states that the
hardware asks for in front of them nor the waits for what they bring are the
compiler's.  Needs the disassembler that comes with hipcc, no GPU."""
from __future__ import annotations

import os
import re
import struct
import subprocess

import pytest

pytest.importorskip("torch")
import post_weight_quantization_29_amd as P  # noqa: E402
from post_weight_quantization_29_amd import _lib as M  # noqa: E402

OBJDUMP = "/opt/rocm/llvm/bin/llvm-objdump"


def code_objects(path):
    """The gfx950 code objects of a library: the entries of its offload bundles."""
    b, at = open(path, "rb").read(), 0
    while (at := b.find(b"__CLANG_OFFLOAD_BUNDLE__", at)) >= 0:
        n, = struct.unpack_from("<Q", b, at + 24)
        p = at + 32
        for _ in range(n):
            off, size, length = struct.unpack_from("<QQQ", b, p)
            if b"gfx950" in b[p + 24:p + 24 + length] and size:
                yield b[at + off:at + off + size]
            p += 24 + length
        at += 24


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{symbol: [(address, instruction)]}"""
    if not os.path.exists(OBJDUMP):
        pytest.skip("no disassembler")
    P.lib()
    out, folder = {}, tmp_path_factory.mktemp("code")
    for k, obj in enumerate(code_objects(M.LIB_PATH)):
        f = folder / f"{k}.o"
        f.write_bytes(obj)
        text = subprocess.run([OBJDUMP, "-d", "--no-show-raw-insn", "--mcpu=gfx950", str(f)], capture_output=True, text=True,
                              check=True).stdout
        name = None
        for line in text.splitlines():
            if m := re.match(r"(?:[0-9a-f]+ )?<(\S+)>:$", line):
                name = m.group(1)
            elif name and (m := re.match(r"\t(\S.*?)\s*//\s*([0-9A-F]+):", line)):
                out.setdefault(name, []).append((int(m.group(2), 16), m.group(1)))
    assert len(out) > 20
    return out


def to_lds(op):
    return op.startswith("buffer_load") and op.endswith(" lds")


def test_copies_to_lds_keep_the_required_wait_states(kernels):
    """One wait state between a write of M0 and the copy that goes to its address, five between a vector
    instruction's write of a scalar register and a memory instruction that reads it."""
    copies, bad = 0, []
    for name, code in kernels.items():
        for n, (at, op) in enumerate(code):
            if not to_lds(op):
                continue
            copies += 1
            lo, hi = map(int, re.search(r"s\[(\d+):(\d+)\]", op).groups())
            states = 0
            for _, before in reversed(code[max(0, n - 6):n]):
                if states < 1 and re.match(r"s_\S+ m0,", before):
                    bad.append((name, hex(at), before))
                if states < 5 and (m := re.match(r"v_\w+ s\[?(\d+)(?::(\d+))?", before)) and \
                        int(m.group(1)) <= hi and lo <= int(m.group(2) or m.group(1)):
                    bad.append((name, hex(at), before, states))
                states += int(before.split()[1], 0) + 1 if before.startswith("s_nop") else 1
    assert copies > 100
    assert not bad, f"{len(bad)} of {copies}: {bad[:4]}"


def is_memory(op):
    return re.match(r"(buffer|global|flat|scratch)_(load|store|atomic)", op) is not None


def test_a_stage_of_few_tokens_is_there_before_its_barrier(kernels):
    """The product of some tokens reads a stage of activations behind a barrier, which has to wait for the copies
    of all stages before the one whose own are in flight: no more operations may be outstanding than were issued
    since the barrier before it.  (A load whose value nobody uses is not issued, whatever the source counts.)"""
    barriers, bad = 0, []
    for name, code in kernels.items():
        if "w4_mid_kernel" not in name:
            continue
        issued, waits, first = 0, [], True
        for at, op in code:
            if is_memory(op):
                issued += 1
            elif m := re.match(r"s_waitcnt .*vmcnt\((\d+)\)", op):
                waits.append((int(m.group(1)), issued))
            elif op == "s_barrier":
                barriers += 1
                # the first one follows a wait for everything
                if not any(left <= (0 if first else new) for left, new in waits):
                    bad.append((name, hex(at), waits))
                issued, waits, first = 0, [], False
    assert barriers >= 12 * 4
    assert not bad, f"{len(bad)} of {barriers}: {bad[:4]}"


def test_append_reads_no_row_before_it_knows_that_the_batch_has_it(kernels):
    """Rows outside the batch are not read: what another stream does with them is its own affair.  A token's
    sequence is found by counting the starts up to it (s_bcnt1 of a ballot); rows are read by wide loads (12 or 16 bytes a lane)."""
    found = 0
    for name, code in kernels.items():
        if "kv4_append_kernel" not in name:
            continue
        ops = [op for _, op in code]
        row = next(n for n, op in enumerate(ops) if re.match(r"(global|flat)_load_dwordx[34] ", op))
        count = next(n for n, op in enumerate(ops) if op.startswith("s_bcnt1_i32_b64"))
        assert count < row, name
        found += 1
    assert found == 6
