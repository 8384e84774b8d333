"""The compiled attention kernels never overwrite a matrix product's result before it is there (CPU).

A 16x16x32 product writes its registers up to eight wait states after its issue, so that an
instruction that writes one of them earlier would see its own value replaced by the late
result. The same walk as for early reads follows every path behind every product.
"""
import os
import subprocess

import pytest

from test_kv_wait_states import ROOT, STATES, kernels, operands, registers


def early_writes(lines):
    """(product, writer) pairs where fewer than STATES wait states lie between them on some path."""
    at = {x[:-1]: i for i, x in enumerate(lines) if x.endswith(":")}
    found = []
    for i, x in enumerate(lines):
        if not x.startswith("v_mfma"):
            continue
        result = registers(operands(x)[1][0])
        todo, seen = [(i + 1, 0, frozenset(result))], set()
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
                elif op.startswith("v_mfma"):     # the next product's result comes behind this one's
                    live = live - registers(args[0])
                elif op.startswith("v_") and args:
                    # both operands of a swap are written
                    written = set().union(*map(registers, args[:2] if "_swap_" in op or op.startswith("v_swap") else args[:1]))
                    if written & live:
                        found.append((x, y))
                        break
                elif op.startswith(("ds_read", "ds_bpermute", "ds_permute", "ds_swizzle", "global_load", "buffer_load", "scratch_load",
                                    "flat_load")) and args:
                    if "_lds_" not in op and registers(args[0]) & live:
                        found.append((x, y))
                        break
                passed += 1
    return found


def test_the_search_finds_an_early_write():
    product = "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]"
    for write in ("v_mov_b32_e32 v3, 0", "v_cndmask_b32_e32 v0, v12, v13, vcc", "v_permlane32_swap_b32_e32 v12, v2",
                  "ds_read_b128 v[0:3], v20", "global_load_dword v1, v[20:21], off"):
        assert early_writes([product, write]) and early_writes([product, "s_nop 6", write]), write
        assert not early_writes([product, "s_nop 7", write]), write
    for other in ("v_mov_b32_e32 v4, 0", "v_cmp_lt_f32_e32 vcc, v0, v1", "ds_write_b128 v20, v[0:3]",
                  "v_mfma_f32_16x16x32_bf16 v[0:3], v[4:7], v[8:11], v[0:3]"):
        assert not early_writes([product, other]), other
    # the write of one part under a mask, behind a branch
    sides = [product, "s_cbranch_vccnz .LBB0_1", "s_nop 3", "v_cndmask_b32_e32 v3, v12, v3, vcc", ".LBB0_1:", "s_nop 7"]
    assert early_writes(sides) == [(product, sides[3])]
    assert not early_writes([product, "s_nop 7"] + sides[1:])


def test_no_attention_kernel_overwrites_a_product_early(tmp_path):
    from fp4_mqa_scoring_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path / "attn.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([hipcc, *flags, "-I", os.path.join(ROOT, "include"), "-S", "--cuda-device-only",
                    os.path.join(build.PKG, "csrc", "mqa_kv_attn.hip"), "-o", str(out)], check=True, capture_output=True)
    found = kernels(out.read_text())
    assert len(found) > 40
    early = {name: writes for name, lines in found.items() if (writes := early_writes(lines))}
    assert not early, next(iter(early.items()))
