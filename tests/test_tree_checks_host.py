"""The build with device-side index checks covers the operators on drafted trees (no GPU needed):
in the compiled code of every kernel, each template instance for itself, a check can count."""
import os
import re
import shutil
import subprocess

import pytest

from device_draft_verification_specverify_amd import build as b

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.mark.parametrize("source,least", [("tree_cache.hip", 2), ("tree_verify.hip", 7),
                                          ("tree_attention.hip", 22)])
def test_every_kernel_counts_failed_index_checks(source, least, tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc missing")
    path = [s for s in b.TREE_SOURCES if s.endswith(source)][0]
    asm = tmp_path / "device.s"
    res = subprocess.run([HIPCC, "-S", "--cuda-device-only", "-O1", "-std=c++17", "-w",
                          f"--offload-arch={b.ARCH}", "-DSV_DEVICE_CHECKS", "-I", b.INCLUDE, path,
                          "-o", str(asm)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr[-3000:]
    text = asm.read_text()
    kernels = re.findall(r"^\s*\.amdhsa_kernel (\S+)", text, re.M)
    assert len(kernels) >= least
    for k in kernels:
        if "clear_kernel" in k:  # its one index is the bound of its loop
            continue
        body = text[text.index(f"\n{k}:"):]
        assert "sv_check_count" in body[:body.index(".Lfunc_end")], k
