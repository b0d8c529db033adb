"""Serving calls over lengths whose offsets, or whose last chunk, pass 32 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
MOST = 2 ** 31 - 1


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_packed_codes_past_2_31_bits():
    """6-bit codes of 360 million tokens: bit 6 t of a row passes 2^31."""
    import compressed_attention_cvq_b200 as cvq
    T = 360_000_000 // 64 * 64
    assert 6 * T > 2 ** 31
    g = torch.Generator().manual_seed(1)
    kcb, vcb = torch.zeros(2, 1, 64, 32, 2), torch.zeros(2, 1, 64, 64)
    kcb[:, :, 1], vcb[:, :, 1] = torch.randn(2, 1, 32, 2, generator=g), torch.randn(2, 1, 64, generator=g)
    # every token has code 0, a key and value of zeros; a few at the end have code 1
    at = np.array([357_913_941, 357_913_942, 357_913_948, 359_999_000, T - 1])
    codes = torch.zeros((1, 1, 2, 1, T // 4 * 3), dtype=torch.uint8)
    for t in at:
        w = 1 << (6 * (int(t) % 4))
        for k in range(3):
            codes[..., int(t) // 4 * 3 + k] |= (w >> (8 * k)) & 255
    codes = codes.cuda()
    q = torch.randn(2, 4, 128, generator=g)
    # scores of code 1 of some tens, against which 2^29 tokens of score 0 still count
    q *= 200.0 / q.norm(dim=-1, keepdim=True)
    k = kcb[:, 0, 1].double().reshape(128).numpy()
    theta = 500000.0 ** (-np.arange(64) * 2.0 / 128)
    z = (k[0::2] + 1j * k[1::2]) * np.exp(1j * np.asarray(at)[:, None] * theta)
    keys = np.stack((z.real, z.imag), -1).reshape(len(at), 128)
    v = vcb[:, 0, 1].double().reshape(128).numpy()
    for dtype in (torch.float32, torch.bfloat16):
        x = q.to(dtype)
        s = x.double().numpy() @ keys.T / math.sqrt(128)                    # [2, 4, tokens]
        m = np.maximum(s.max(-1), 0)
        w = np.exp(s - m[..., None])
        total = w.sum(-1) + (T - len(at)) * np.exp(-m)
        lse, out = m + np.log(total), (w.sum(-1) / total)[..., None] * v
        shape = cvq.make_shape(2, 4, 1, 1, T, 500000.0, 128, 64, 6)
        got = cvq.prefix_attend(shape, x.cuda(), kcb[None].cuda(), codes, codes, i32([T]), vcb[None].cuda(),
                                out_dtype=torch.float32)
        # a score is off by 2^-19 of its terms at most, here below 200; a weight as a score is
        ds = 2.0 ** -19 * 200 * 1.5
        assert np.all(np.abs(got[1].double().cpu().numpy() - lse) <= ds + 1e-5)
        assert np.all(np.abs(got[0].double().cpu().numpy() - out) <= (2 * ds + 1e-4) * np.abs(v).max())
    assert cvq.fault_status(clear=True) == 0


def test_a_prefix_of_2_31_tokens():
    """The longest prefix there is, of one token's code: in both kernels its last tile ends beside 2^31."""
    import compressed_attention_cvq_b200 as cvq
    kcb, vcb = torch.zeros(1, 16, 1, 256, 4, 2, device="cuda"), torch.zeros(1, 16, 1, 256, 8, device="cuda")
    vcb[:, :, :, 0] = torch.randn(1, 16, 1, 8, device="cuda")
    codes = torch.zeros((1, 1, MOST, 1, 16), dtype=torch.uint8, device="cuda")
    v = vcb[0, :, 0, 0].reshape(128)
    for dtype in (torch.float32, torch.bfloat16):
        q = torch.randn(1, 1, 128, device="cuda").to(dtype)
        shape = cvq.make_shape(1, 1, 1, 1, MOST)
        out, lse = cvq.prefix_attend(shape, q, kcb, codes, codes, i32([MOST]), vcb, 4096, out_dtype=torch.float32)
        # Sums of weights, powers of two here, are exact.  A thread of the fp32 kernel adds one value 2^18
        # times, to a sum whose step is by then 2^-5 of it, so that each addition is off by half of that;
        # the other kernel takes sums of 16 tiles up, 128 of them: 12 16 2^-23 + 128 2^-24
        assert abs(float(lse) - math.log(MOST)) <= 1e-4
        assert torch.allclose(out[0, 0], v, rtol=2.0 ** -6 if dtype == torch.float32 else 4e-5, atol=0)
    assert cvq.fault_status(clear=True) == 0


def test_a_paged_sequence_of_2_31_tokens():
    """One page of one token, 2^31 - 1 times: the last chunk of 16 tokens passes 2^31."""
    import compressed_attention_cvq_b200 as cvq
    pg = cvq.make_paged(1, 4, 1, 1, 1, MOST)
    kp, vp = (torch.randn(1, 1, 1, 128, device="cuda").bfloat16() for _ in range(2))
    table = torch.zeros((1, MOST), dtype=torch.int32, device="cuda")
    q = torch.randn(1, 4, 128, device="cuda").bfloat16()
    out, lse = cvq.paged_attend(pg, q, kp, vp, table, i32([MOST]), 148, out_dtype=torch.float32)
    # sums of 64 chunks (128 additions, cut off at 2^-23) are taken up in fp32, 3600 of them a warp
    s = (q.double() @ kp[0, 0, 0].double()) / math.sqrt(128)
    assert torch.all((lse.double() - s - math.log(MOST)).abs() <= 1e-3)
    assert torch.allclose(out[0], vp[0, 0, 0].float().expand(4, 128), rtol=1e-3, atol=0)
    assert cvq.fault_status(clear=True) == 0
