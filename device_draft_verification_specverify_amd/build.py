"""Build libspecverify.so (HIP, gfx950) in place with hipcc.

Usage: python -m device_draft_verification_specverify_amd.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SOURCE = os.path.join(HERE, "csrc", "specverify.hip")
# The operators on drafted token trees, a translation unit each.
TREE_SOURCES = [os.path.join(HERE, "csrc", n)
                for n in ("tree_cache.hip", "tree_verify.hip", "tree_attention.hip")]
# The operators around a verification step, a translation unit each.
SERVING_SOURCES = [os.path.join(HERE, "csrc", n)
                   for n in ("serving_pages.hip", "serving_rotate.hip", "serving_attention.hip",
                             "serving_logits.hip")]
HOST_SOURCES = [os.path.join(HERE, "csrc", "bandit.cpp")]
INCLUDE = os.path.join(ROOT, "include")
LIBRARY = os.path.join(HERE, "libspecverify.so")
# The same sources with device-side index checks (-DSV_DEVICE_CHECKS): a debug
# build for running the GPU tests with every work unit's indices checked.
CHECKED_LIBRARY = os.path.join(HERE, "libspecverify_checked.so")
ARCH = "gfx950"

# Packed FP32 instructions stay off: the compiler must not form them.
# Machine-level loop-invariant code motion stays off too: it hoists per-thread
# addresses and constants out of the streaming loops into registers that stay
# live across them (about 20 extra VGPRs in the streaming kernel). Private
# arrays are not moved to LDS: that costs occupancy instead of registers.
HIP_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-shared", f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-disable-machine-licm",
    "-mllvm", "-disable-promote-alloca-to-lds",
    # (m0, named as clobbered by the LDS loads written out, is a reserved register)
    "-Wall", "-Wno-unused-function", "-Wno-inline-asm",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm)")


def _run(cmd: list[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and res.stderr.strip():
        print(res.stderr, file=sys.stderr)


def build(verbose: bool = False, extra_flags: list[str] | None = None,
          checked: bool = False) -> str:
    """Compile the sources into LIBRARY, or CHECKED_LIBRARY with the device-side
    index checks (always recompiles). Returns the path."""
    out = CHECKED_LIBRARY if checked else LIBRARY
    tmp = out + ".tmp"
    flags = [*HIP_FLAGS, *(extra_flags or []), *(["-DSV_DEVICE_CHECKS"] if checked else [])]
    with tempfile.TemporaryDirectory() as d:
        # one compiler per source, side by side, then one link
        units = [(src, os.path.join(d, os.path.basename(src) + ".o"))
                 for src in [SOURCE, *TREE_SOURCES, *SERVING_SOURCES, *HOST_SOURCES]]
        compile_flags = [f for f in flags if f != "-shared"]
        cmds = [[hipcc(), *compile_flags, "-I", INCLUDE, "-c", src, "-o", obj]
                for src, obj in units]
        with ThreadPoolExecutor(max_workers=min(len(cmds), 8)) as ex:
            list(ex.map(lambda c: _run(c, verbose), cmds))
        _run([hipcc(), "-shared", "-fPIC", f"--offload-arch={ARCH}", *(obj for _, obj in units),
              "-o", tmp], verbose)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(verbose=True, checked="--checked" in sys.argv[1:]))
