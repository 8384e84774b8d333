"""The compiled kernels of attention over caches in 4 bits neither read a matrix product's result before it is there nor
overwrite its registers, and keep nothing of their loops in scratch memory (CPU)."""
import os
import re
import subprocess

import pytest

from test_kv_wait_states import early_reads, kernels
from test_kv_wait_states_writes import early_writes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def listing(tmp_path_factory):
    from fp4_mqa_scoring_amd import build
    try:
        hipcc = build.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    out = tmp_path_factory.mktemp("fp4") / "fp4.s"
    flags = [f for f in build.HIPCC_FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run([hipcc, *flags, "-I", os.path.join(ROOT, "include"), "-S", "--cuda-device-only",
                    os.path.join(build.PKG, "csrc", "mqa_kv_fp4.hip"), "-o", str(out)], check=True, capture_output=True)
    found = kernels(out.read_text())
    assert len(found) == 40     # decode and selected, two types, ten shapes
    return found


def test_no_kernel_reads_a_product_early(listing):
    early = {name: reads for name, lines in listing.items() if (reads := early_reads(lines))}
    assert not early, next(iter(early.items()))


def test_no_kernel_overwrites_a_product_s_registers(listing):
    early = {name: writes for name, lines in listing.items() if (writes := early_writes(lines))}
    assert not early, next(iter(early.items()))


def innermost_loop(lines):
    """The shortest stretch that a branch back encloses with a matrix instruction in it."""
    at = {x[:-1]: i for i, x in enumerate(lines) if x.endswith(":")}
    loops = []
    for i, x in enumerate(lines):
        m = re.match(r"s_c?branch\w*\s+(\.LBB\w+)", x)
        if m and at.get(m[1], i) < i and any(y.startswith("v_mfma") for y in lines[at[m[1]]:i]):
            loops.append(lines[at[m[1]]:i])
    return min(loops, key=len)


def test_no_streaming_loop_spills(listing):
    """A scratch access would wait for every copy in flight."""
    spills = {name: [x for x in innermost_loop(lines) if x.startswith("scratch_")] for name, lines in listing.items()}
    assert not any(spills.values()), [n for n, x in spills.items() if x]
