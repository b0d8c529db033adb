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


def test_one_token_of_a_fused_projection():
    """A single token's stride is of no meaning: its queries are rotated in place, and pieces of a
    projection of any width are taken."""
    import compressed_attention_cvq_b200 as cvq
    Hq, Hkv = 8, 2
    pg = cvq.make_paged(1, Hq, Hkv, 16, 4, 4)
    kp, vp = (torch.zeros((4, Hkv, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    args = (i32([0, 1]), i32([1]), i32([[2, 0, 1, 3]]), kp, vp)
    first = i32([5])
    for width in ((Hq + 2 * Hkv) * 128, (Hq + 2 * Hkv) * 128 + 3):
        row = torch.randn(1, width, device="cuda").bfloat16()
        q, k, v = row[:, :(Hq + 2 * Hkv) * 128].unflatten(1, (-1, 128)).split([Hq, Hkv, Hkv], 1)
        want = cvq.paged_append(pg, k.contiguous(), v.contiguous(), *args, q=q.clone(), pos_offsets=first)
        pages = kp.clone()
        kp.zero_()
        got = cvq.paged_append(pg, k, v, *args, q=q, q_out=q, pos_offsets=first)
        assert got is q and torch.equal(q, want) and torch.equal(kp, pages)


def test_half_a_state_is_refused():
    import compressed_attention_cvq_b200 as cvq
    pg = cvq.make_paged(1, 8, 2, 16, 4, 4)
    kp, vp = (torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros((1, 8, 128), dtype=torch.bfloat16, device="cuda")
    args = (pg, q, kp, vp, i32([[0, 1, 2, 3]]), i32([5]))
    o, z = torch.zeros((1, 8, 128), device="cuda"), torch.zeros((1, 8), device="cuda")
    for prev in ((None, z), (o, None)):
        with pytest.raises(TypeError, match="prev"):
            cvq.paged_attend(*args, prev=prev)
    cvq.paged_attend(*args, prev=(o, z))
