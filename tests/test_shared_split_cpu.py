"""The arithmetic of split_weights (csrc/shared.cuh), restated for every weight of
a binade: what the two bf16 parts leave, and that both are above zero."""
import numpy as np
import pytest
import torch


@pytest.mark.parametrize("exponent", [16, 0, -1, -60, -119, -124])
def test_two_parts_of_a_weight(exponent):
    bits = np.arange(1 << 23, dtype=np.uint32) | np.uint32((exponent + 127) << 23)
    p = bits.view(np.float32)
    hi = ((p * np.float32(1 - 2.0 ** -9)).view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
    rest = p - hi
    assert np.array_equal(rest.astype(np.float64), p.astype(np.float64) - hi)  # exact
    lo = torch.from_numpy(rest).bfloat16().double().numpy()
    assert (hi > 0).all() and (lo > 0).all()
    off = np.abs(hi.astype(np.float64) + lo - p)
    assert (off <= np.maximum(2.0 ** -15 * p.astype(np.float64), 2.0 ** -134)).all()
