"""The C ABI's host code and that of the microscaled and optimizer launches (workspace layouts,
grids, a step's tables), rebuilt with AddressSanitizer and UndefinedBehaviorSanitizer on
the host pass alone, under the CPU tests of every entry point: refusals, and calls that get
as far as their launches."""
import os
import subprocess
import sys

import pytest

from tests.test_sanitizers import ROOT, _clang_asan_runtime

HOST = ("moe_api.hip", "adamw.hip", "mx.hip", "mx_gemm.hip")
TESTS = ("test_abi.py", "test_abi_mx.py", "test_abi_select.py", "test_abi_select_edges.py", "test_abi_adamw_scalars.py",
         "test_adamw_overlap.py", "test_mx_no_rows.py", "test_mx_wide_numbers.py", "test_host_launches.py")

CHILD = r"""
import sys
sys.path.insert(0, ROOT)
from sparse_expert_routing_amd import _lib
_lib.load(LIB)
import pytest
sys.exit(pytest.main(["-q", "-p", "no:cacheprovider", "-m", "not gpu", *[ROOT + "/tests/" + t for t in TESTS]]))
"""


def test_host_code_up_to_the_launches_under_asan_and_ubsan(tmp_path):
    from sparse_expert_routing_amd import build as B
    if not os.path.exists(B.HIPCC):
        pytest.skip("hipcc is not installed")
    rt = _clang_asan_runtime(B.HIPCC)
    if rt is None:
        pytest.skip("the compiler's AddressSanitizer runtime is not installed")
    # host pass only: every sanitizer flag sits behind -Xarch_host
    extra = ["-O1", "-g", "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
             "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    objs, jobs = [], []
    for src in B.sources():
        name = os.path.basename(src)
        objs.append(os.path.join(str(tmp_path) if name in HOST else B.BUILD, name + ".o"))
        if name in HOST:
            jobs.append(subprocess.Popen([B.HIPCC, *B.FLAGS, *extra, "-c", src, "-o", objs[-1]]))
        elif not os.path.exists(objs[-1]):
            pytest.skip("build the library first (its objects are reused)")
    assert [j.wait() for j in jobs] == [0] * len(HOST)
    lib = str(tmp_path / "libmoe_san.so")
    subprocess.check_call([B.HIPCC, f"--offload-arch={B.ARCH}", "-shared", "-fPIC", "-Xarch_host",
                           "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host",
                           "-shared-libsan", "-o", lib, *objs])
    env = dict(os.environ, LD_PRELOAD=rt, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="print_stacktrace=1")
    code = CHILD.replace("ROOT", repr(ROOT)).replace("LIB", repr(lib)).replace("TESTS", repr(TESTS))
    r = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=900,
                       cwd=str(tmp_path))
    assert r.returncode == 0, f"sanitizer run failed (exit {r.returncode}):\n{r.stdout[-4000:]}\n{r.stderr[-6000:]}"
    assert " passed" in r.stdout and "runtime error" not in r.stderr and "AddressSanitizer" not in r.stderr
