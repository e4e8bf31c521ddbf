"""The host code of the operators on drafted trees under AddressSanitizer and
UndefinedBehaviorSanitizer (CPU only).

tests/sanitized_tree_driver.cpp is linked against a build of their sources whose host side is
instrumented; the device code is never run here. Any sanitizer report aborts it.
"""
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from device_draft_verification_specverify_amd import build as b

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
ROCM_LIB = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(HIPCC))), "lib")
SAN = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
       "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]


def run(cmd):
    res = subprocess.run(cmd, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    if not os.path.exists(HIPCC) or shutil.which("g++") is None:
        pytest.skip("hipcc or g++ missing")
    d = tmp_path_factory.mktemp("san_tree")
    inc = ["-I", os.path.join(b.ROOT, "include")]
    host_san = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-fno-omit-frame-pointer"]
    units = [(src, str(d / (os.path.basename(src) + ".o"))) for src in b.TREE_SOURCES]
    drv_o, exe = str(d / "drv.o"), str(d / "drv")
    cmds = [[HIPCC, "-g", "-std=c++17", "-fPIC", "-w", f"--offload-arch={b.ARCH}", "-Xarch_device",
             "-O1", "-Xarch_host", "-O1", *SAN, *inc, "-c", src, "-o", obj] for src, obj in units]
    cmds.append(["g++", "-O1", "-g", "-std=c++17", *host_san, *inc, "-c",
                 os.path.join(b.ROOT, "tests", "sanitized_tree_driver.cpp"), "-o", drv_o])
    with ThreadPoolExecutor(max_workers=len(cmds)) as ex:
        list(ex.map(run, cmds))
    run(["g++", *host_san, *(obj for _, obj in units), drv_o, f"-L{ROCM_LIB}", "-lamdhip64",
         f"-Wl,-rpath,{ROCM_LIB}", "-o", exe])
    return exe


def test_tree_host_code_is_clean_under_sanitizers(driver):
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:abort_on_error=0",
               UBSAN_OPTIONS="print_stacktrace=1")
    res = subprocess.run([driver], capture_output=True, text=True, env=env, timeout=120)
    assert "ERROR: AddressSanitizer" not in res.stderr, res.stderr[-3000:]
    assert "runtime error" not in res.stderr, res.stderr[-3000:]
    assert res.returncode == 0, "\n".join(x for x in res.stdout.splitlines() if "FAIL" in x)[-3000:]
    assert res.stdout.count("\nok ") > 200
