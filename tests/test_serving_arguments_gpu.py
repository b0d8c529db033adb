"""Calls of the serving binding at the edges of what it takes: shapes of nothing, one token, half a
state."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_no_heads_are_an_error():
    """A shape without KV heads and tensors to match: refused, not divided by."""
    import compressed_attention_cvq_b200 as cvq
    q = torch.zeros((1, 0, 128), device="cuda")
    cb = torch.zeros((0, 16, 1, 256, 8), device="cuda")
    codes = torch.zeros((1, 0, 64, 1, 16), dtype=torch.uint8, device="cuda")
    shape = cvq.make_shape(1, 0, 0, 1, 64)
    with pytest.raises(ValueError):
        cvq.prefix_attend(shape, q, cb.unflatten(-1, (4, 2)), codes, codes, i32([1]), cb, 1)
