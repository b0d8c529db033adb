"""One workspace for a server's calls: its batch and its split counts change from step to step, and
the shared prefix uses the same memory."""
import numpy as np
import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def paged(B, Hq, Hkv, longest, seed, ps=16):
    import compressed_attention_cvq_b200 as cvq
    g = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    m = -(-longest // ps)
    kp, vp = (torch.randn((B * m, Hkv, ps, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn((B, Hq, 128), generator=g, device="cuda").bfloat16()
    lens = rng.integers(1, longest + 1, B)
    lens[0] = longest
    return (cvq.make_paged(B, Hq, Hkv, ps, B * m, m), q, kp, vp,
            i32(rng.permutation(B * m).reshape(B, m)), i32(lens))


def test_batches_and_split_counts_in_turn():
    import compressed_attention_cvq_b200 as cvq
    calls = [(paged(*s, seed=i), n) for i, (s, n) in enumerate([
        ((6, 32, 8, 3000), 9), ((1, 8, 8, 5000), 4), ((6, 32, 8, 3000), 3), ((17, 16, 2, 1200), 5),
        ((2, 4, 1, 9000), 31), ((6, 32, 8, 3000), 9)])]
    want = [cvq.paged_attend(*a, n) for a, n in calls]
    need = max(cvq.paged_workspace_alloc(a[0], n, "cuda").numel() for a, n in calls)
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=2304, R=1, seed=4)
    dev = {n: torch.from_numpy(d[n]).cuda() for n in ("key_cb", "val_cb", "key_codes", "val_codes")}
    x = torch.randn(5, 8, 128, device="cuda").bfloat16()
    shape, ln = cvq.shape_of(x, dev["key_codes"]), i32([2200])

    def prefix(ws):
        return cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"], dev["val_codes"], ln,
                                 dev["val_cb"], 3, workspace=ws)
    need = max(need, cvq.prefix_workspace_alloc(shape, 3, "cuda").numel())
    want_p = prefix(None)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        for (a, n), w in zip(calls, want):
            for splits in (n, 1, n):
                out, lse = torch.full_like(w[0], 7.0), torch.full_like(w[1], 7.0)
                cvq.paged_attend(*a, splits, workspace=ws, out=out, lse=lse)
                if splits == n:
                    assert torch.equal(out, w[0]) and torch.equal(lse, w[1])
            got = prefix(ws)
            assert torch.equal(got[0], want_p[0]) and torch.equal(got[1], want_p[1])


def test_more_units_than_counters():
    """70000 sequences and KV heads: taken without splits, whatever the count asked for."""
    import compressed_attention_cvq_b200 as cvq
    a = paged(8750, 8, 8, 16, seed=3)
    want = cvq.paged_attend(*a, 1)
    for n in (2, 5):
        got = cvq.paged_attend(*a, n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_of_its_size_is_not_left():
    """Nothing is written before or behind the bytes that a call asks for."""
    import compressed_attention_cvq_b200 as cvq
    for a, n in ((paged(3, 8, 2, 1500, 1), 4), (paged(5, 6, 3, 777, 2), 3), (paged(1, 8, 1, 4097, 3), 17)):
        need = cvq.paged_workspace_alloc(a[0], n, "cuda").numel()
        big = torch.full((need + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
        big[4096:4096 + need] = 0
        cvq.paged_attend(*a, n, workspace=big[4096:4096 + need])
        assert bool((big[:4096] == 0x5a).all()) and bool((big[4096 + need:] == 0x5a).all())
    for group, R, t_cap, n, B in ((8, 1, 2304, 3, 7), (8, 2, 2304, 2, 33), (64, 5, 2304, 2, 3), (8, 2, 320, 4, 3),
                                  (8, 1, 9000, 1, 2)):
        d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=t_cap, R=R, seed=R, group_dim=group)
        dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
        x = torch.randn(B, 8, 128, device="cuda").half()
        shape = cvq.shape_of(x, dev["key_codes"], group_dim=group)
        need = cvq.prefix_workspace_alloc(shape, n, "cuda").numel()
        big = torch.full((need + 8192,), 0x5a, dtype=torch.uint8, device="cuda")
        outs = torch.full((B * 8 * 128 + 4096,), 7.0, dtype=torch.half, device="cuda")
        cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"], dev["val_codes"], i32([t_cap - 5]),
                          dev["val_cb"], n, workspace=big[4096:4096 + need],
                          out=outs[2048:2048 + B * 1024].view(B, 8, 128))
        assert bool((big[:4096] == 0x5a).all()) and bool((big[4096 + need:] == 0x5a).all())
        assert bool((outs[:2048] == 7).all()) and bool((outs[2048 + B * 1024:] == 7).all())


@pytest.mark.parametrize("group,R,t_cap", [(8, 1, 2304), (8, 2, 2304), (64, 12, 2304), (8, 2, 320), (8, 1, 40000)])
def test_what_a_prefix_workspace_holds_does_not_matter(group, R, t_cap):
    """Also through a call that makes its own, of memory that others have used."""
    import compressed_attention_cvq_b200 as cvq
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=t_cap, R=R, seed=R, group_dim=group)
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    x = torch.randn(5, 8, 128, device="cuda").half()
    shape = cvq.shape_of(x, dev["key_codes"], group_dim=group)
    ws = cvq.prefix_workspace_alloc(shape, 1, "cuda")

    def call(w):
        return cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"], dev["val_codes"], i32([t_cap - 5]),
                                 dev["val_cb"], 1, workspace=w)
    want = call(ws)
    for byte in (0xff, 0x7f, 0x55):                          # NaN, large and small numbers
        got = call(ws.fill_(byte))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        used = [torch.full_like(ws, byte) for _ in range(2)]
        del used
        got = call(None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
