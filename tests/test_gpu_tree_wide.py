"""GPU: verification where several workgroups share a request's rows (from 28673 ids on), in each
form that the library chooses by size, type and alignment, against the oracle for equality."""
from __future__ import annotations

import pytest

import test_gpu_tree_verify as ver

pytestmark = pytest.mark.gpu


# B, largest tree, ids (chunks of 4096 / workgroups a request): rows kept in registers (32000: 8 / 2;
# 128256: 32 / 8), shares of more chunks than are taken at once (37000: 10 / 2), more than 256
# workgroups (64 x 8), rows that begin anywhere because they are 50257 long, one workgroup each (300)
@pytest.mark.parametrize("mode", ver.MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,most,V", [(2, 14, 32000), (64, 3, 32000), (3, 10, 37000), (64, 3, 37000),
                                      (3, 10, 50257), (40, 3, 50257), (2, 9, 128256),
                                      (64, 2, 128256), (300, 2, 37000), (1, 20, 28673)])
def test_verify_shared_rows(mode, dtype, B, most, V):
    ver.check(ver.case(B + V + mode, B, most, "random", V, mode, dtype))


@pytest.mark.parametrize("mode", ver.MODES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_verify_shared_rows_of_few_tokens(mode, dtype):
    # many rejections one after the other
    ver.check(ver.case(3 + mode, 4, 24, "star", 60000, mode, dtype, zeros=True, sharp=4.0, near=0.1))


@pytest.mark.parametrize("dtype,stride", [("f32", 40005), ("bf16", 40003), ("bf16", 40008)])
def test_verify_shared_rows_of_odd_strides(dtype, stride):
    for mode in ver.MODES:
        ver.check(ver.case(70 + mode, 5, 9, "random", 40000, mode, dtype), stride=stride)
