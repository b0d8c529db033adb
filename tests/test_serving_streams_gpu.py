"""The `stream` argument of the serving calls, with what the calls allocate for themselves: the
current stream is kept busy, or allocates, while the given one works."""
import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu
LONG = 100_000_000                 # clocks of a sleep on the device: some 50 ms


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def paged_call():
    """A call of several splits, so that arrivals are counted and partial states merged."""
    import compressed_attention_cvq_b200 as cvq
    B, Hq, Hkv, ps, m = 4, 8, 2, 16, 128
    g = torch.Generator(device="cuda").manual_seed(1)
    kp, vp = (torch.randn((B * m, Hkv, ps, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, Hq, 128), generator=g, device="cuda").bfloat16()
    table, lens = i32(np.arange(B * m).reshape(B, m)), i32([2048, 2047, 1000, 1])
    pg = cvq.make_paged(B, Hq, Hkv, ps, B * m, m)
    need = cvq.paged_workspace_alloc(pg, 4, "cuda").numel()
    return (lambda **kw: cvq.paged_attend(pg, q, kp, vp, table, lens, 4, **kw)), need


def prefix_call(t_cap):
    import compressed_attention_cvq_b200 as cvq
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=t_cap, R=2, seed=4)
    dev = {n: torch.from_numpy(d[n]).cuda() for n in ("key_cb", "val_cb", "key_codes", "val_codes")}
    x = torch.randn(4, 8, 128, device="cuda").bfloat16()
    shape, ln = cvq.shape_of(x, dev["key_codes"]), i32([t_cap - 7])
    need = cvq.prefix_workspace_alloc(shape, 3, "cuda").numel()
    return (lambda **kw: cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"], dev["val_codes"], ln,
                                           dev["val_cb"], 3, **kw)), need


CALLS = {"paged": paged_call, "prefix_fp32": lambda: prefix_call(640), "prefix": lambda: prefix_call(2304)}


@pytest.mark.parametrize("name", CALLS)
def test_a_busy_current_stream_holds_nothing_up(name):
    """The workspace is cleared in the order of the given stream, whatever the memory held before."""
    call, need = CALLS[name]()
    want = call()
    dirty = [torch.full((n,), 0x7f, dtype=torch.uint8, device="cuda")
             for n in (need, want[0].numel() * want[0].element_size(), want[1].numel() * 4)]
    del dirty
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    got = call(stream=st)
    st.synchronize()
    assert not torch.cuda.current_stream().query()           # it sleeps still
    got = [x.clone() for x in got]                           # behind the sleep: st is done
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("name", CALLS)
def test_memory_of_the_given_stream_stays_its_own(name):
    """What the call allocated and let go is not handed to the current stream while the given one
    has yet to use it."""
    call, need = CALLS[name]()
    want = call()
    sizes = [need, want[0].numel() * want[0].element_size(), want[1].numel() * 4]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(LONG)
    call(stream=st)                                          # outputs let go at once, too
    taken = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(4)]
    torch.cuda.current_stream().synchronize()
    assert not st.query()
    torch.cuda.synchronize()
    for t in taken:
        assert bool((t == 0x55).all())


def test_rotated_queries_of_the_given_stream():
    import compressed_attention_cvq_b200 as cvq
    n, Hq, Hkv = 64, 8, 2
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, v = (torch.randn((n, h, 128), generator=g, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv))
    kp, vp = (torch.zeros((8, Hkv, 16, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pg = cvq.make_paged(1, Hq, Hkv, 16, 8, 8)
    args = (pg, k, v, i32([0, n]), i32([n]), i32([[3, 1, 2, 0, 4, 5, 6, 7]]), kp, vp)
    want = cvq.paged_append(*args, q=q)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        torch.cuda._sleep(LONG)
    cvq.paged_append(*args, q=q, stream=st)
    taken = [torch.full((want.numel() * 2,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    for t in taken:
        assert bool((t == 0x55).all())
    got = cvq.paged_append(*args, q=q, stream=st)
    st.synchronize()
    assert torch.equal(got, want)


def test_the_current_stream_is_what_it_was():
    call, _ = paged_call()
    st = torch.cuda.Stream()
    before = torch.cuda.current_stream()
    call(stream=st)
    with pytest.raises(ValueError):
        call(stream=st, out=torch.zeros(1, device="cuda"))
    assert torch.cuda.current_stream() == before
    torch.cuda.synchronize()
    # the default stream, given by name
    want = call()
    with torch.cuda.stream(st):
        got = call(stream=torch.cuda.default_stream())
        assert torch.cuda.current_stream() == st
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0])
