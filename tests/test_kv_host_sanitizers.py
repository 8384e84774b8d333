"""The key-value cache operators' host code (checks of arguments, strides and overlaps, plans of launches) under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU, no GPU call): the library with both on hipcc's host pass runs the host tests of these operators, and
through a stand-in for the HIP runtime the whole way of a call to its launches."""
import os
import subprocess

import pytest

host = pytest.importorskip("test_host_sanitizers", reason="its helpers run the sanitizers")     # may be left out of a copy of the tree

TESTS = ["tests/test_kv_abi_cpu.py", "tests/test_kv_append_abi_cpu.py", "tests/test_kv_overlap_cpu.py", "tests/test_kv_strides_cpu.py",
         "tests/test_kv_launches_cpu.py", "tests/test_kv_write_groups_cpu.py"]


def test_host_checks_and_launches_under_sanitizers(tmp_path):
    from fp4_mqa_scoring_amd import build as b
    try:
        hipcc = b.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not found")
    rt = host._runtime(hipcc, "libclang_rt.asan-x86_64.so")
    if rt is None:
        pytest.skip("clang sanitizer runtime not found")
    lib = str(tmp_path / "libmqa_fp4_san.so")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=undefined",
           "-Xarch_host", "-fno-omit-frame-pointer"]
    flags = [f for f in b.HIPCC_FLAGS if f != "-O3"] + ["-O1", "-g"] + san
    subprocess.run([hipcc, *flags, "-parallel-jobs=8", "-I", os.path.join(host.ROOT, "include"), *b.SOURCES, "-o", lib], check=True, capture_output=True)
    assert host._instrumented(lib)
    (tmp_path / "sanitized.py").write_text(
        f"import fp4_mqa_scoring_amd as m\nfrom fp4_mqa_scoring_amd import build\nm.LIB_PATH = build.LIB = {lib!r}\n"
        "def pytest_sessionfinish(session):\n    assert build.LIB in open('/proc/self/maps').read()\n")
    path = os.pathsep.join([str(tmp_path), host.ROOT] + ([os.environ["PYTHONPATH"]] if os.environ.get("PYTHONPATH") else []))
    host._run_tests(["-p", "sanitized", *TESTS], {"PYTHONPATH": path}, [rt])
