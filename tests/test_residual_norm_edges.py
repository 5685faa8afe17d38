"""The norms around a block where the way that a row is taken changes: the longest rows that
are taken by their granules, and the first that are not."""
import pytest
import torch

from tests.test_residual_norm import check, inputs

F32, BF16 = torch.float32, torch.bfloat16

# 16-byte pieces that a row of d lies in at most: (d + 14) / 8 of bf16, (d + 6) / 4 of float32.
# Forward up to 1536 and 2048 of them, backward to 1536, with a gate for each element to 1024;
# from 256 rows on for each of those that are cut alike again (8 rows of 2 bytes, 4 of 4).
FORWARD = [(BF16, 2048, 12281), (BF16, 1024, 12282), (BF16, 2047, 12281), (F32, 1024, 8189), (F32, 512, 8190), (F32, 1023, 8189)]
BACKWARD = [(F32, 1024, 6141), (F32, 512, 6142)]
ELEMENTS = [(BF16, 2048, 8185), (BF16, 1024, 8186), (F32, 1024, 4093), (F32, 512, 4094)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [dict(post=True, rms=True), dict(post=True, gate=1), dict(post=False)], ids=str)
@pytest.mark.parametrize("dtype,rows,d", FORWARD + BACKWARD)
def test_longest_rows_by_granules(dtype, rows, d, kind):
    s = inputs(rows, d, dtype, dtype, **kind)
    check(s, scale=0.7, rms=kind.get("rms", False))


@pytest.mark.gpu
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,rows,d", ELEMENTS)
def test_longest_rows_by_granules_with_a_gate_for_each_element(dtype, rows, d, rms):
    check(inputs(rows, d, dtype, dtype, rms=rms, gate=rows), scale=0.7, rms=rms)
