"""Host-side refusals of the serving calls (no GPU): every call below carries one invalid
argument, or has nothing to do, so that none of them reaches a launch."""
import ctypes

import pytest
import torch

from compressed_attention_cvq_b200 import _binding as b

FAKE = 0x10000          # an aligned, non-null address that is never dereferenced
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 5


def shape(**kw):
    d = dict(batch=3, n_q_heads=32, n_kv_heads=8, R=2, t_cap=1024)
    d.update(kw)
    return b.make_shape(**d)


def paged(**kw):
    d = dict(batch=3, n_q_heads=32, n_kv_heads=8, head_dim=128, page_size=16, n_pages=10,
             max_pages=4, kv_dtype=b.CVQ_BF16, rope_base=500000.0, page_stride=0)
    d.update(kw)
    return b.cvq_paged(*d.values())


def prefix(s, **kw):
    a = dict(q=FAKE, qd=1, kcb=FAKE, ks=0, kc=FAKE, vc=FAKE, ln=FAKE, vcb=FAKE, vs=0, n=4,
             ws=FAKE, out=FAKE, od=0, lse=FAKE)
    a.update(kw)
    return b.lib.cvq_prefix_attend(ctypes.byref(s) if s is not None else None, *a.values(), None)


def append(p, **kw):
    a = dict(n=5, q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, d=1, off=FAKE, lens=FAKE,
             pos=FAKE, tab=FAKE, kp=FAKE, vp=FAKE, qo=FAKE)
    a.update(kw)
    return b.lib.cvq_paged_append(ctypes.byref(p) if p is not None else None, *a.values(), None)


def attend(p, **kw):
    a = dict(q=FAKE, qd=1, kp=FAKE, vp=FAKE, tab=FAKE, lens=FAKE, n=4, ws=FAKE, po=FAKE, pl=FAKE,
             out=FAKE + 16, od=0, lse=FAKE)
    a.update(kw)
    return b.lib.cvq_paged_attend(ctypes.byref(p) if p is not None else None, *a.values(), None)


@pytest.mark.parametrize("kw,st", [
    (dict(q=None), NULL), (dict(q=FAKE + 8), ALIGN), (dict(qd=3), UNSUPPORTED),
    (dict(qd=-1), UNSUPPORTED), (dict(kcb=None), NULL), (dict(vcb=FAKE + 4), ALIGN),
    (dict(kc=None), NULL), (dict(vc=FAKE + 1), ALIGN), (dict(ln=None), NULL),
    (dict(ln=FAKE + 2), ALIGN), (dict(ks=-4), SHAPE), (dict(vs=100), SHAPE),
    (dict(ks=16 * 2 * 256 * 8 + 2), ALIGN), (dict(n=0), WORKSPACE), (dict(n=4097), WORKSPACE),
    (dict(ws=None), NULL), (dict(ws=FAKE + 8), ALIGN), (dict(out=None), NULL),
    (dict(out=FAKE + 2), ALIGN), (dict(od=9), UNSUPPORTED), (dict(lse=None), NULL),
    (dict(lse=FAKE + 1), ALIGN)])
def test_prefix_refusals(kw, st):
    assert prefix(shape(), **kw) == st


def test_prefix_shapes():
    assert prefix(None) == NULL
    for kw, st in ((dict(head_dim=64), UNSUPPORTED), (dict(R=3), UNSUPPORTED), (dict(batch=0), SHAPE),
                   (dict(n_q_heads=12), SHAPE), (dict(n_q_heads=24), UNSUPPORTED),
                   (dict(t_cap=-1), SHAPE), (dict(rope_base=1.0), SHAPE),
                   (dict(group_dim=64, t_cap=100), SHAPE), (dict(group_dim=64, R=23), UNSUPPORTED)):
        assert prefix(shape(**kw)) == st, kw
        assert b.lib.cvq_prefix_workspace_bytes(ctypes.byref(shape(**kw)), 4) == 0
    assert b.lib.cvq_prefix_workspace_bytes(ctypes.byref(shape()), 0) == 0
    assert b.lib.cvq_prefix_workspace_bytes(ctypes.byref(shape()), 4) >= 3 * 32 * 4 * 130 * 4


@pytest.mark.parametrize("kw,st", [
    (dict(head_dim=64), UNSUPPORTED), (dict(kv_dtype=0), UNSUPPORTED), (dict(kv_dtype=3), UNSUPPORTED),
    (dict(batch=0), SHAPE), (dict(batch=70000), SHAPE), (dict(n_q_heads=0), SHAPE),
    (dict(n_q_heads=30), SHAPE), (dict(n_q_heads=24), UNSUPPORTED), (dict(n_q_heads=128), UNSUPPORTED),
    (dict(page_size=0), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=2048), SHAPE),
    (dict(n_pages=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(max_pages=1 << 28), SHAPE),
    (dict(rope_base=1.0), SHAPE), (dict(rope_base=float("nan")), SHAPE),
    (dict(page_stride=8 * 16 * 128 - 8), SHAPE), (dict(page_stride=-8), SHAPE),
    (dict(page_stride=8 * 16 * 128 + 4), ALIGN), (dict(page_stride=1 << 61), SHAPE)])
def test_paged_shapes(kw, st):
    p = paged(**kw)
    assert append(p) == st and attend(p) == st
    assert b.lib.cvq_paged_workspace_bytes(ctypes.byref(p), 4) == 0
    assert b.lib.cvq_paged_suggest_splits(ctypes.byref(p), 148) == 1


@pytest.mark.parametrize("kw,st", [
    (dict(n=-1), SHAPE), (dict(q=None), NULL), (dict(qo=None), NULL), (dict(q=FAKE + 8), ALIGN),
    (dict(qo=FAKE + 8), ALIGN), (dict(qs=4095), SHAPE), (dict(qs=4100), ALIGN),
    (dict(qs=4100, d=0), SHAPE), (dict(k=None), NULL), (dict(v=FAKE + 2), ALIGN),
    (dict(ks=1016), SHAPE), (dict(vs=1025), ALIGN), (dict(d=3), UNSUPPORTED), (dict(off=None), NULL),
    (dict(off=FAKE + 2), ALIGN), (dict(lens=None), NULL), (dict(pos=FAKE + 1), ALIGN),
    (dict(tab=None), NULL), (dict(kp=None), NULL), (dict(vp=FAKE + 8), ALIGN),
    (dict(qs=4104), SHAPE)])          # in place only when dense: q is q_out here
def test_append_refusals(kw, st):
    assert append(paged(), **kw) == st


def test_append_of_nothing():
    assert append(paged(), n=0) == 0
    assert append(paged(), n=0, q=None, qo=None, pos=None) == 0
    assert append(None) == NULL


@pytest.mark.parametrize("kw,st", [
    (dict(q=None), NULL), (dict(q=FAKE + 4), ALIGN), (dict(qd=5), UNSUPPORTED), (dict(kp=None), NULL),
    (dict(vp=FAKE + 8), ALIGN), (dict(tab=None), NULL), (dict(tab=FAKE + 2), ALIGN),
    (dict(lens=None), NULL), (dict(n=0), WORKSPACE), (dict(n=5000), WORKSPACE), (dict(ws=None), NULL),
    (dict(ws=FAKE + 8), ALIGN), (dict(po=None), NULL), (dict(pl=None), NULL), (dict(po=FAKE + 8), ALIGN),
    (dict(pl=FAKE + 2), ALIGN), (dict(out=None), NULL), (dict(out=FAKE + 8), ALIGN),
    (dict(od=4), UNSUPPORTED), (dict(lse=None), NULL), (dict(lse=FAKE + 3), ALIGN),
    (dict(out=FAKE, od=1), UNSUPPORTED)])     # prev_out is out, but of another type
def test_attend_refusals(kw, st):
    assert attend(paged(), **kw) == st


def test_attend_needs_a_shape():
    assert attend(None) == NULL


def test_split_suggestions_are_in_range():
    for B in (1, 7, 64, 60000):
        for t in (1, 64, 5000, 131072):
            for dt in (0, 1, 2):
                assert 1 <= b.lib.cvq_prefix_suggest_splits(ctypes.byref(shape(batch=B, t_cap=t)), dt, 148) <= 4096
            p = paged(batch=B, max_pages=-(-t // 16))
            assert 1 <= b.lib.cvq_paged_suggest_splits(ctypes.byref(p), 148) <= 4096


def test_binding_refuses_tensors_on_the_host():
    import compressed_attention_cvq_b200 as cvq
    x = torch.zeros(3, 32, 128)
    with pytest.raises(ValueError, match="CUDA"):
        cvq.prefix_attend(shape(), x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        cvq.paged_append(paged(), x, x, x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        cvq.paged_attend(paged(), x, x, x, x, x)
    with pytest.raises(ValueError, match="float16"):
        cvq.make_paged(1, 8, 2, 16, 4, 4, torch.int8)


def test_page_fault_bit():
    assert b.CVQ_PAGE_FAULT == 4 and b.fault_names(4 | 1) == ["copy_timeout", "page"]
