"""What the Python binding of the serving calls refuses before it looks at a tensor (no GPU)."""
import ctypes

import pytest
import torch

import compressed_attention_cvq_b200 as cvq
from compressed_attention_cvq_b200 import _binding as b


def test_a_shape_of_the_other_kind_is_refused():
    """The native side reads a structure by its address: a smaller one would be read past its end."""
    assert ctypes.sizeof(b.cvq_shape) < ctypes.sizeof(b.cvq_paged)
    shape, paged, x = cvq.make_shape(1, 8, 2, 1, 64), cvq.make_paged(1, 8, 2, 16, 4, 4), torch.zeros(1)
    for wrong in (paged, None, 5, ctypes.c_int(3)):
        with pytest.raises(TypeError):
            cvq.prefix_attend(wrong, x, x, x, x, x, x)
    for wrong in (shape, None, 5, ctypes.c_int(3)):
        with pytest.raises(TypeError):
            cvq.paged_append(wrong, x, x, x, x, x, x, x)
        with pytest.raises(TypeError):
            cvq.paged_attend(wrong, x, x, x, x, x)
