"""Builds the HIP library libmqa_fp4.so in-tree for gfx950 (hipcc, no GPU needed)."""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmqa_fp4.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in ("mqa_kernels.hip", "mqa_api.hip", "mqa_quant.hip", "mqa_decode.hip",
                                               "mqa_kv_attn.hip", "mqa_kv_fp4.hip", "mqa_kv_evict.hip", "mqa_kv_write.hip",
                                               "mqa_kv_api.hip", "mqa_kv_write_api.hip")]
# measurement probes (bench only), a library of their own beside the operator's
PROBE_LIB = os.path.join(PKG, "libmqa_fp4_probe.so")
PROBE_SOURCES = [os.path.join(PKG, "csrc", "mqa_probe.hip")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    # packed fp32 VALU forms stay disabled on this target
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)


def _build_one(lib: str, sources, verbose: bool) -> None:
    """Compiles the sources side by side, then links them."""
    tmp = lib + ".tmp%d" % os.getpid()
    with tempfile.TemporaryDirectory() as where:
        objects = [os.path.join(where, os.path.basename(f) + ".o") for f in sources]
        with concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            flags = [f for f in HIPCC_FLAGS if f != "-shared"]
            list(pool.map(lambda fo: _run([hipcc(), *flags, "-I", os.path.join(ROOT, "include"), "-c", fo[0], "-o", fo[1]],
                                          verbose), zip(sources, objects)))
        _run([hipcc(), *HIPCC_FLAGS, *objects, "-o", tmp], verbose)
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    """Builds the operator library and the bench-only probe library."""
    _build_one(LIB, SOURCES, verbose)
    _build_one(PROBE_LIB, PROBE_SOURCES, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
