"""The compiled attention kernels never read a matrix product's result before it is there (CPU).

A 16x16x32 product's registers may be read by other instructions after eight wait states.
The compiler sees to that, but behind a branch that overwrites a part of the result under a mask it
has left the wait out for the other parts; the kernels wait by themselves there. This
compiles them to assembly and follows every path behind every product.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
STATES = 8


def registers(token):
    m = re.match(r"v\[(\d+):(\d+)\]$", token)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.match(r"-?\|?v(\d+)\|?$", token)
    return {int(m[1])} if m else set()


def kernels(text):
    """Instructions and labels of every kernel of an assembly listing."""
    found, name = {}, None
    for line in text.splitlines():
        line = line.split(";")[0].strip()
        m = re.match(r"(_Z\w+):$", line)
        if m:
            name = m[1]
            found[name] = []
        elif name and line and (not line.startswith(".") or line.startswith(".LBB")):
            found[name].append(line)
    return {k: v for k, v in found.items() if any(x.startswith("v_mfma") for x in v)}


def operands(line):
    p = line.split(None, 1)
    return p[0], [o.strip() for o in p[1].split(",")] if len(p) > 1 else []


def early_reads(lines):
    """(product, reader) pairs where fewer than STATES wait states lie between them on some path."""
    at = {x[:-1]: i for i, x in enumerate(lines) if x.endswith(":")}
    found = []
    for i, x in enumerate(lines):
        if not x.startswith("v_mfma"):
            continue
        todo, seen = [(i + 1, 0, frozenset(registers(operands(x)[1][0])))], set()
        while todo:
            j, passed, live = todo.pop()
            while j < len(lines) and passed < STATES and live and (j, passed, live) not in seen:
                seen.add((j, passed, live))
                y = lines[j]
                j += 1
                if y.endswith(":"):
                    continue
                op, args = operands(y)
                if op == "s_nop":
                    passed += int(args[0], 0) + 1
                    continue
                if op == "s_branch":
                    todo.append((at[args[0]], passed + 1, live))
                    break
                if op == "s_endpgm":
                    break
                if op.startswith("s_cbranch"):
                    todo.append((at[args[0]], passed + 1, live))
                elif op.startswith("v_mfma"):     # its own accumulator is chained by the unit
                    if (registers(args[1]) | registers(args[2])) & live:
                        found.append((x, y))
                    live = live - registers(args[0])
                elif op.startswith(("v_", "ds_", "global_", "buffer_")) and args:
                    reads = args[1:] if op.startswith("v_") and not op.startswith(("v_cmp", "v_permlane", "v_fmac")) else args
                    if set().union(*map(registers, reads)) & live:
                        found.append((x, y))
                        break
                    if op.startswith("v_"):
                        live = live - registers(args[0])
                passed += 1
    return found


def test_the_search_finds_an_early_read():
    product = "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]"
    read = "v_max_f32_e32 v12, v3, v3"
    assert early_reads([product, read]) and early_reads([product, "s_nop 6", read])
    assert not early_reads([product, "s_nop 7", read])
    assert not early_reads([product, "v_mov_b32_e32 v3, 0", read])
    # one side of a branch waits, the other does not
    sides = [product, "s_cbranch_vccnz .LBB0_1", "s_nop 7", "v_mov_b32_e32 v3, 0", ".LBB0_1:", read]
    assert early_reads(sides) == [(product, read)]
    assert not early_reads([product, "s_nop 7"] + sides[1:])


def test_no_attention_kernel_reads_a_product_early(tmp_path):
    from fp4_mqa_scoring_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    assert shutil.which(hipcc) or os.path.exists(hipcc)
    out = tmp_path / "attn.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([hipcc, *flags, "-I", os.path.join(ROOT, "include"), "-S", "--cuda-device-only",
                    os.path.join(build.PKG, "csrc", "mqa_kv_attn.hip"), "-o", str(out)], check=True, capture_output=True)
    found = kernels(out.read_text())
    assert len(found) > 40
    early = {name: reads for name, lines in found.items() if (reads := early_reads(lines))}
    assert not early, next(iter(early.items()))
