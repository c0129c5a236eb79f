"""Wide vector stores of the kernels that hand partial sums over in memory, in
the device code as compiled: no store of more than 8 bytes is followed at once by
an instruction that overwrites a register of its data.  (The compiler takes
stores with a scalar offset as safe from that; on the card they were not.)"""
import os
import re
import subprocess

import pytest

from quantization_error_compensation_amd import build

OUT = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build")


def registers(operand):
    m = re.match(r"v\[(\d+):(\d+)\]$", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"v(\d+)$", operand)
    return {int(m[1])} if m else set()


def overwritten(lines):
    """Pairs (store, next instruction) where the second writes the first's data."""
    pairs = []
    for line, after in zip(lines, lines[1:]):
        m = re.match(r"(buffer|global|flat)_store_dwordx[34]\s+(.*)", line)
        if not m:
            continue
        operands = [o.strip() for o in m[2].split(",")]
        data = registers(operands[0 if m[1] == "buffer" else 1])
        n = re.match(r"(v_\w+)\s+([^,]+)", after)
        if n and not n[1].startswith(("v_cmp", "v_readlane", "v_readfirstlane")) and registers(n[2].strip()) & data:
            pairs.append((line, after))
    return pairs


def test_the_search_finds_such_a_pair():
    lines = ["buffer_store_dwordx4 v[82:85], v103, s[4:7], s22 offen sc1", "v_or_b32_e32 v82, s19, v102",
             "buffer_store_dwordx4 v[86:89], v82, s[4:7], 0 offen", "s_nop 0", "v_mov_b32_e32 v86, 0",
             "global_store_dwordx4 v[2:3], v[6:9], off", "v_mov_b32_e32 v2, 0"]
    assert overwritten(lines) == [(lines[0], lines[1])]


@pytest.mark.parametrize("source", ["k_q8_gemm.hip", "k_decode.hip", "k_kv_decode.hip", "k_kv_prefill.hip"])
def test_no_store_loses_its_data(source):
    os.makedirs(OUT, exist_ok=True)
    asm = os.path.join(OUT, source.replace(".hip", ".gcn"))
    subprocess.check_call([build.HIPCC, *build.CFLAGS, *build.FILE_FLAGS.get(source, []), "-S",
                           "--cuda-device-only", os.path.join(build.CSRC, source), "-o", asm],
                          stderr=subprocess.DEVNULL)
    with open(asm) as f:
        lines = [x.split(";")[0].strip() for x in f]
    lines = [x for x in lines if x and not x.startswith(".") and not x.endswith(":")]
    assert any("_store_dwordx4" in x for x in lines)
    assert not overwritten(lines)
