"""Limits of the map operators' binding (CPU)."""
import pytest
import torch

import memory_bound_cnn_wtconv_b200 as wt
from memory_bound_cnn_wtconv_b200 import maps


@pytest.mark.parametrize("shape", [((1 << 32) + 7, 1), (1 << 32, 4), (1 << 31, 1), (2, 1 << 31), (1 << 31, 1, 1, 1),
                                   (1, (1 << 32) + 1, 1, 1), (1, 1, 1 << 32, 1), (1, 1, 2, (1 << 32) + 2)], ids=str)
def test_extents_past_31_bits_are_refused(shape):
    # The descriptor's fields are C ints, which would take an extent modulo 2^32.
    with pytest.raises(ValueError, match="2147483647"):
        maps._Map(shape, torch.float32, wt.NHWC)


def test_largest_extents_are_taken():
    m = maps._Map(((1 << 31) - 1, 1), torch.bfloat16, wt.NHWC)
    assert (m.desc.B, m.desc.C, m.desc.H, m.desc.W) == ((1 << 31) - 1, 1, 1, 1) and m.rows == ((1 << 31) - 1,)


@pytest.mark.parametrize("device", ["meta", "cpu"])
def test_branch_dropout_draws_its_seed_on_the_cpu(device):
    # From torch's CPU generator, whatever device tensors are made on by default.
    torch.manual_seed(11)
    want = wt.BranchDropout(0.1).seed
    torch.manual_seed(11)
    with torch.device(device):
        assert wt.BranchDropout(0.1).seed == want
