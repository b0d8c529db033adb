"""cvq_paged_append and cvq_paged_attend against their float64 definitions, and a decode loop
that uses them together with the shared prefix."""
import numpy as np
import pytest
import torch

import serve_util as U
import workloads

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def np64(t):
    return t.double().cpu().numpy()


def pages_for(lens, ps, rng, spare=2, width=None):
    """A page table that hands out shuffled pages, and the number of pages in the pool."""
    need = [-(-int(n) // ps) for n in lens]
    total = sum(need) + spare
    order = rng.permutation(total)
    width = width or max(1, max(need))
    table = np.full((len(lens), width), -1, np.int32)      # entries past a length are not read
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, total


def setup(lens, Hq, Hkv, ps, dtype, cache, seed=0, stride=0, width=None):
    import compressed_attention_cvq_b200 as cvq
    rng = np.random.default_rng(seed)
    table, n = pages_for(lens, ps, rng, width=width)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dense = Hkv * ps * 128
    pools = []
    for _ in range(2):
        x = torch.randn((n, stride or dense), generator=gen, device="cuda").to(DT[cache])
        pools.append(x[:, :dense].unflatten(1, (Hkv, ps, 128)))
    q = torch.randn((len(lens), Hq, 128), generator=gen, device="cuda").to(DT[dtype])
    pg = cvq.make_paged(len(lens), Hq, Hkv, ps, n, table.shape[1], DT[cache], page_stride=stride)
    return pg, q, pools[0], pools[1], i32(table), i32(lens)


def verify(got, q, kp, vp, table, lens, dtype, cache, prev=None, out_dtype=None):
    out, lse = (np64(x) for x in got)
    q, kp, vp = np64(q), np64(kp), np64(vp)
    table, lens = table.cpu().numpy(), lens.cpu().numpy()
    prev = None if prev is None else tuple(np64(x) for x in prev)
    ref = U.paged_reference(q, kp, vp, table, lens, prev)
    # products are exact up to the split of a query of another type into two 16-bit parts and
    # of a weight into two: 2^-16 relative each, whatever the types
    e = 2.0 ** -16
    tol_o, tol_l = np.zeros_like(ref[0]), np.zeros_like(ref[1])
    n, Hkv, ps, _ = kp.shape
    g = q.shape[1] // Hkv
    for b in range(len(lens)):
        p = np.arange(min(max(int(lens[b]), 0), table.shape[1] * ps))
        page = table[b, p // ps]
        p, page = p[(page >= 0) & (page < n)], page[(page >= 0) & (page < n)]
        for h in range(Hkv):
            sl = slice(h * g, (h + 1) * g)
            k, v = kp[page, h, p % ps], vp[page, h, p % ps]
            o, z = U.attention(q[b, sl], k, v)
            tol_o[b, sl], tol_l[b, sl] = U.state_tolerance(q[b, sl], k, v, o, z, e, 0.0, e)
    if prev is not None:
        # the merged state moves by no more than its parts, its weights by the error of lse
        # and the rounding of an exponential of fp32 numbers of this size
        live = ~np.isneginf(prev[1])
        size = np.where(live, np.abs(np.where(live, prev[1], 0.0)), 0.0) + 1
        dw = tol_l + 2.0 ** -21 * size
        tol_o += dw[..., None] * np.where(live[..., None], np.abs(np.where(live[..., None], prev[0], 0.0)), 0.0)
        tol_o += dw[..., None] * np.abs(ref[0]) + 2.0 ** -22 * np.abs(ref[0])
        tol_l += 2.0 ** -20 * size
    U.check(out, lse, *ref, tol_o, tol_l, U.HALF[out_dtype or dtype])


@pytest.mark.parametrize("lens,Hq,Hkv,ps,dtype,cache", [
    ([1], 4, 1, 16, "bf16", "bf16"),
    ([0, 1, 2, 15, 16, 17, 33, 64], 32, 8, 16, "bf16", "bf16"),
    ([100, 0, 1000, 513], 8, 2, 8, "fp16", "fp16"),
    ([777, 3000, 1], 16, 2, 64, "fp32", "bf16"),          # 8 query heads per KV head
    ([777, 2999, 0, 12], 16, 2, 64, "fp32", "fp16"),
    ([130, 127], 6, 3, 128, "bf16", "fp16"),              # 2 per KV head, mixed types
    ([500, 499, 3], 5, 5, 32, "fp16", "bf16"),            # as many KV heads
    ([5000], 32, 8, 256, "bf16", "bf16"),
    ([70, 71, 200], 8, 8, 1, "bf16", "bf16"),             # one token to a page
    ([1500, 40], 8, 1, 1024, "fp32", "fp16"),
    ([33] * 70, 8, 2, 2, "bf16", "bf16"),
])
@pytest.mark.parametrize("with_prev", [False, True])
def test_attend_matches_the_definition(lens, Hq, Hkv, ps, dtype, cache, with_prev):
    import compressed_attention_cvq_b200 as cvq
    a = setup(lens, Hq, Hkv, ps, dtype, cache, seed=len(lens) + ps)
    prev = None
    if with_prev:
        gen = torch.Generator(device="cuda").manual_seed(3)
        prev = [torch.randn((len(lens), Hq, 128), generator=gen, device="cuda"),
                torch.randn((len(lens), Hq), generator=gen, device="cuda") * 4 + 5]
        prev[1][0, 0] = -torch.inf                          # no earlier part for this row
        prev[0][0, 0] = float("nan")
        prev = tuple(prev)
    got = cvq.paged_attend(*a, prev=prev)
    verify(got, *a[1:], dtype, cache, prev)
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("n_splits", [1, 2, 3, 8, 31, 33, 4096])
def test_any_split_count_and_output_type(n_splits):
    import compressed_attention_cvq_b200 as cvq
    a = setup([2000, 1, 0, 700, 1999], 8, 2, 16, "bf16", "bf16", seed=n_splits)
    ws = cvq.paged_workspace_alloc(a[0], n_splits, "cuda")
    for od in ("fp32", "bf16", "fp16", "fp32"):              # the workspace is reused as it is
        got = cvq.paged_attend(*a, n_splits, workspace=ws, out_dtype=DT[od])
        verify(got, *a[1:], "bf16", "bf16", None, od)


def test_in_place_merge_and_strided_pools():
    import compressed_attention_cvq_b200 as cvq
    a = setup([300, 0, 41], 8, 2, 16, "fp32", "bf16", stride=2 * 2 * 16 * 128 + 64)
    prev = (torch.randn(3, 8, 128, device="cuda"), torch.randn(3, 8, device="cuda"))
    keep = tuple(x.clone() for x in prev)
    got = cvq.paged_attend(*a, prev=prev, out=prev[0], lse=prev[1])
    assert got[0] is prev[0]
    verify(got, *a[1:], "fp32", "bf16", keep)


def test_what_lies_behind_a_sequence_is_not_read():
    import compressed_attention_cvq_b200 as cvq
    lens = [100, 17, 1, 0]
    a = setup(lens, 8, 2, 16, "bf16", "bf16", seed=2, width=9)
    want = cvq.paged_attend(*a)
    table, n = a[4].cpu().numpy(), a[0].n_pages
    for b, L in enumerate(lens):
        if L % 16:
            page = int(table[b, L // 16])
            a[2][page, :, L % 16:] = float("nan")
            a[3][page, :, L % 16:] = float("inf")
    a[4][a[4] < 0] = 2 ** 31 - 1                             # entries past a length
    got = cvq.paged_attend(*a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert cvq.fault_status(clear=True) == 0
    # lengths out of range are taken as the nearest possible ones
    full = setup([32, 32], 8, 2, 16, "bf16", "bf16", seed=3)
    want = cvq.paged_attend(*full)
    got = cvq.paged_attend(*full[:5], i32([10 ** 9, 33]))
    assert torch.equal(got[0], want[0])
    got = cvq.paged_attend(*full[:5], i32([-1, -2 ** 31]))
    assert torch.all(got[0] == 0) and torch.all(got[1] == -torch.inf)


def test_values_that_are_not_finite():
    """A NaN or infinity inside a sequence reaches its own KV head's rows only."""
    import compressed_attention_cvq_b200 as cvq
    a = setup([40, 40], 8, 2, 16, "bf16", "bf16", seed=5)
    want = cvq.paged_attend(*a)
    page = int(a[4][0, 1])
    a[3][page, 1, 3, 7] = float("inf")
    a[2][page, 0, 5, 0] = float("nan")
    out, lse = cvq.paged_attend(*a)
    assert torch.isnan(out[0, :4]).all() and torch.isnan(lse[0, :4]).all()
    assert not torch.isfinite(out[0, 4:, 7]).any()           # inf, or NaN out of its parts
    keep = [i for i in range(128) if i != 7]
    assert torch.equal(out[0, 4:][:, keep], want[0][0, 4:][:, keep])
    assert torch.equal(lse[0, 4:], want[1][0, 4:]) and torch.equal(out[1], want[0][1])


def test_large_and_tiny_magnitudes():
    import compressed_attention_cvq_b200 as cvq
    for dtype, cache, scale in (("fp32", "fp16", 2.0 ** 18), ("bf16", "fp16", 2.0 ** 20),
                                ("fp32", "fp16", 2.0 ** -20), ("bf16", "bf16", 2.0 ** 60)):
        a = list(setup([200, 3], 8, 2, 16, dtype, cache, seed=6))
        a[1] = (a[1].float() * scale).to(DT[dtype])
        a[2] = (a[2].float() / max(scale, 2.0 ** -8)).to(DT[cache])
        verify(cvq.paged_attend(*a), *a[1:], dtype, cache)


def test_page_indices_out_of_range():
    """Tested on the host side first (test_serve_host); here the kernel's own check skips the
    page, reports it, and the other tokens are attended to."""
    import compressed_attention_cvq_b200 as cvq
    a = setup([100, 64, 30], 8, 2, 16, "bf16", "bf16", seed=8)
    a[4][0, 2], a[4][1, 0], a[4][2, 0], a[4][2, 1] = -7, a[0].n_pages, 2 ** 31 - 1, -2 ** 31
    assert cvq.fault_status(clear=True) == 0
    got = cvq.paged_attend(*a)
    assert cvq.fault_status(clear=True) == 4
    verify(got, *a[1:], "bf16", "bf16")
    assert torch.all(got[0][2] == 0) and torch.all(got[1][2] == -torch.inf)


def test_same_bits_every_time():
    import compressed_attention_cvq_b200 as cvq
    a = setup([4000, 100, 2500], 32, 8, 16, "bf16", "bf16", seed=9)
    x = cvq.paged_attend(*a)
    for _ in range(4):
        y = cvq.paged_attend(*a)
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_pool_offsets_past_32_bits():
    import compressed_attention_cvq_b200 as cvq
    n, ps, Hkv = 140_000, 16, 8                              # 2.3e9 elements in each pool
    kp, vp = (torch.empty((n, Hkv, ps, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert kp.numel() > 2 ** 31
    table = torch.tensor([[n - 1, 131_072], [131_071, n - 2]], dtype=torch.int32, device="cuda")
    lens = i32([32, 19])
    pg = cvq.make_paged(2, 32, Hkv, ps, n, 2)
    k, v = (torch.randn(51, Hkv, 128, device="cuda").bfloat16() for _ in range(2))
    cvq.paged_append(pg, k, v, i32([0, 32, 51]), lens, table, kp, vp)
    q = torch.randn(2, 32, 128, device="cuda").bfloat16()
    got = cvq.paged_attend(pg, q, kp, vp, table, lens)
    used = table.flatten().long()
    small = i32([[0, 1], [2, 3]])
    verify(got, q, kp[used], vp[used], small, lens, "bf16", "bf16")
    kr = U.rotate(np64(k).swapaxes(0, 1), np.r_[0:32, 0:19]).swapaxes(0, 1)
    assert np.abs(np64(kp[n - 1].swapaxes(0, 1)) - kr[:16]).max() <= U.BF16 * np.abs(kr).max()


# --- append ----------------------------------------------------------------------------
def append_case(new, held, Hq, Hkv, ps, dtype, cache, seed=0, pad=0, fused=False, stride=0):
    lens = np.asarray(new) + np.asarray(held)
    pg, _, kp, vp, table, tl = setup(lens, Hq, Hkv, ps, dtype, cache, seed, stride)
    n = int(sum(new)) + pad
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    qkv = torch.randn((n, Hq + 2 * Hkv, 128), generator=gen, device="cuda").to(DT[dtype])
    q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
    if not fused:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    off = i32(np.concatenate([[0], np.cumsum(new)]))
    return pg, q, k, v, off, tl, table, kp, vp


def append_reference(q, k, v, new, lens, first, table, kp, vp):
    """What the pages and the queries hold afterwards, in float64."""
    q, k, v, kp, vp = (np64(x) for x in (q, k, v, kp, vp))
    qo = np.full(q.shape, np.nan)
    i = 0
    for b, m in enumerate(new):
        for j in range(m):
            p = int(lens[b]) - m + j
            qo[i] = U.rotate(q[i], np.full(q.shape[1], first[b] + p))
            page = table[b, p // kp.shape[2]] if 0 <= p < table.shape[1] * kp.shape[2] else -1
            if 0 <= page < kp.shape[0]:
                kp[page, :, p % kp.shape[2]] = U.rotate(k[i], np.full(k.shape[1], first[b] + p))
                vp[page, :, p % kp.shape[2]] = v[i]
            i += 1
    return qo, kp, vp


def append_check(got_q, kp, vp, ref, x_max, dtype, cache):
    """Rotated values: the rounding of their type, plus that of two fp32 products and of the
    sines (4 half steps of fp32 at the pair's magnitude, at most sqrt 2 of the largest)."""
    qo, rk, rv = ref
    slack = 2 ** 0.5 * x_max * 6 * U.FP32
    live = ~np.isnan(qo)
    d = np.abs(np64(got_q) - qo)[live] - U.HALF[dtype] * np.abs(qo[live])
    assert d.max(initial=-1) <= slack + 2.0 ** -25
    for x, r in ((kp, rk), (vp, rv)):
        d = np.abs(np64(x) - r) - U.HALF[cache] * np.abs(r)
        assert d.max() <= slack + 2.0 ** -25                 # half of fp16's smallest step


@pytest.mark.parametrize("new,held,Hq,Hkv,ps,dtype,cache,pad,fused", [
    ([1], [0], 4, 1, 16, "bf16", "bf16", 0, False),
    ([1] * 33, list(range(33)), 32, 8, 16, "bf16", "bf16", 0, False),
    ([5, 0, 300, 1], [3, 7, 0, 15], 8, 2, 8, "fp16", "fp16", 3, True),
    ([1000, 531], [0, 777], 28, 7, 16, "fp32", "fp16", 5, False),
    ([17, 200], [100, 1], 16, 2, 64, "fp32", "bf16", 0, True),
    ([64], [64], 6, 3, 64, "bf16", "fp16", 1, True),
    ([9, 8, 7], [1, 1, 1], 5, 5, 1, "fp16", "bf16", 0, False),
    ([1] * 300, [4] * 300, 8, 1, 4, "bf16", "bf16", 2, False),
    ([2500], [3], 8, 8, 128, "bf16", "bf16", 0, True),
])
def test_append_matches_the_definition(new, held, Hq, Hkv, ps, dtype, cache, pad, fused):
    import compressed_attention_cvq_b200 as cvq
    pg, q, k, v, off, lens, table, kp, vp = append_case(new, held, Hq, Hkv, ps, dtype, cache,
                                                        len(new), pad, fused)
    first = np.random.default_rng(1).integers(0, 131072, len(new))
    first[0] = 2 ** 31 - 1 - 10 ** 6                         # far positions keep their angles
    ref = append_reference(q, k, v, new, lens.tolist(), first, table.cpu().numpy(), kp, vp)
    q_out = torch.full((q.shape[0], Hq, 128), 3.0, dtype=q.dtype, device="cuda")
    got = cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q, q_out=q_out, pos_offsets=i32(first))
    assert got is q_out
    m = float(torch.stack([x.float().abs().max() for x in (q, k)]).max())
    append_check(got, kp, vp, ref, m, dtype, cache)
    if pad:
        assert torch.all(q_out[-pad:] == 3.0)                # rows behind the last sequence
    # without queries and offsets, into the same rows
    ref = append_reference(q, k, v, new, lens.tolist(), np.zeros(len(new), int), table.cpu().numpy(), kp, vp)
    assert cvq.paged_append(pg, k, v, off, lens, table, kp, vp) is None
    append_check(got[:0], kp, vp, (np.empty((0, Hq, 128)),) + ref[1:], m, dtype, cache)
    assert cvq.fault_status(clear=True) == 0


def test_append_in_place_no_tokens_and_strided_pool():
    import compressed_attention_cvq_b200 as cvq
    new, held = [3, 4], [0, 30]
    pg, q, k, v, off, lens, table, kp, vp = append_case(new, held, 8, 2, 16, "bf16", "bf16", 4,
                                                        stride=2 * 16 * 128 + 8)
    ref = append_reference(q, k, v, new, lens.tolist(), [0, 0], table.cpu().numpy(), kp, vp)
    cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q, q_out=q)
    append_check(q, kp, vp, ref, 6.0, "bf16", "bf16")
    before = kp.clone()
    none = k[:0].contiguous()
    assert cvq.paged_append(pg, none, none, off, lens, table, kp, vp) is None
    assert torch.equal(kp, before)


def test_append_skips_what_has_no_row():
    """Tokens before the start of a sequence, past its page table, or on a bad page are not
    stored, and the fault word says so; the others are."""
    import compressed_attention_cvq_b200 as cvq
    new, held = [4, 4, 4, 4], [0, 0, 14, 2]
    pg, q, k, v, off, lens, table, kp, vp = append_case(new, held, 8, 2, 16, "bf16", "bf16", 6)
    lens = i32([2, 4, 34, 6])          # two tokens before sequence 0, two past the table of 2
    table[3, 0] = pg.n_pages
    ref = append_reference(q, k, v, new, lens.tolist(), [0] * 4, table.cpu().numpy(), kp, vp)
    got = cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q)
    assert cvq.fault_status(clear=True) == 4
    append_check(got, kp, vp, ref, 6.0, "bf16", "bf16")


# --- together --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop_behind_a_shared_prefix(dtype, graph):
    """Six steps of five sequences behind one compressed prefix: append (rotating), attend to
    the prefix, attend to the pages and merge; equal to attention over the whole history."""
    import compressed_attention_cvq_b200 as cvq
    B, Hq, Hkv, R, L, ps = 5, 8, 2, 2, 700, 4
    d = workloads.small(batch=1, n_q_heads=Hq, n_kv_heads=Hkv, t_cap=704, R=R, seed=21, cb_std=0.7)
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    ln, first = i32([L]), i32([L] * B)
    held = np.array([0, 3, 4, 9, 1])
    table, n = pages_for(held + 6, ps, np.random.default_rng(2))
    kp, vp = (torch.zeros((n, Hkv, ps, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pg = cvq.make_paged(B, Hq, Hkv, ps, n, table.shape[1])
    table, off, lens = i32(table), i32(np.arange(B + 1)), i32(held)
    gen = torch.Generator(device="cuda").manual_seed(5)
    # what the sequences hold already
    k0, v0 = (torch.randn((int(held.sum()), Hkv, 128), generator=gen, device="cuda").to(DT[dtype]) for _ in range(2))
    cvq.paged_append(pg, k0, v0, i32(np.concatenate([[0], np.cumsum(held)])), lens, table, kp, vp,
                     pos_offsets=first)
    q, k, v = (torch.empty((B, h, 128), dtype=DT[dtype], device="cuda") for h in (Hq, Hkv, Hkv))
    shape = cvq.shape_of(q, dev["key_codes"])
    n1, n2 = cvq.prefix_suggest_splits(shape, q.dtype), cvq.paged_suggest_splits(pg)
    w1 = cvq.prefix_workspace_alloc(shape, n1, "cuda")
    w2 = cvq.paged_workspace_alloc(pg, n2, "cuda")

    def step():
        lens.add_(1)
        qr = cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q, pos_offsets=first)
        prev = cvq.prefix_attend(shape, qr, dev["key_cb"], dev["key_codes"], dev["val_codes"], ln,
                                 dev["val_cb"], n1, workspace=w1, out_dtype=torch.float32)
        return (qr, prev) + cvq.paged_attend(pg, qr, kp, vp, table, lens, n2, workspace=w2, prev=prev)

    g = None
    for i in range(6):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=gen, device="cuda"))
        if graph and i == 1:
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                res = step()
        if g is not None:
            g.replay()
        else:
            res = step()
        torch.cuda.synchronize()
        qr, prev, out, lse = res
        assert lens.tolist() == (held + i + 1).tolist()
        d["q"] = np64(qr)
        ref = U.prefix_reference(d, L)
        got = tuple(np64(x) for x in prev)
        # every score of the prefix within 2^-8 (fp16 operands; fp32 far below), on average
        tol = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -17
        assert np.abs(got[0] - ref[0]).max() <= tol and np.abs(got[1] - ref[1]).max() <= tol
        verify((out, lse), qr, kp, vp, table, lens, dtype, "bf16", prev)
        # and the whole history at once, with the prefix in 64 bits
        whole = U.paged_reference(np64(qr), np64(kp), np64(vp), table.cpu().numpy(), lens.tolist(), ref)
        assert np.abs(np64(out) - whole[0]).max() <= tol + U.HALF[dtype] * np.abs(whole[0]).max() + 1e-4
        assert np.abs(np64(lse) - whole[1]).max() <= tol + 1e-5
    assert cvq.fault_status(clear=True) == 0


def test_recent_window_behind_each_sequence_own_cache():
    """cvq_attend over each sequence's own codes, then its 16-bit recent tokens on top."""
    import compressed_attention_cvq_b200 as cvq
    from gpu_util import run_oracle, to_device
    d = workloads.small(batch=3, n_q_heads=8, n_kv_heads=2, t_cap=640, R=2, q_dtype="bf16",
                        cb_std=0.7, seq_lens=np.array([640, 0, 77], np.int32), seed=4)
    dd = to_device(d)
    shape = cvq.shape_of(dd["q"], dd["key_codes"])
    state = cvq.attend_fused(shape, dd["q"], dd["key_cb"], dd["key_codes"], dd["val_codes"],
                             dd["seq_lens"], dd["val_cb"], cvq.suggest_splits(shape))
    pg, _, kp, vp, table, lens = setup([50, 64, 0], 8, 2, 16, "bf16", "bf16", seed=1)
    got = cvq.paged_attend(pg, dd["q"], kp, vp, table, lens, prev=state, out_dtype=torch.float32)
    verify(got, dd["q"], kp, vp, table, lens, "bf16", "bf16", state, "fp32")
    ref = U.paged_reference(np64(dd["q"]), np64(kp), np64(vp), table.cpu().numpy(), lens.tolist(), run_oracle(d))
    assert np.abs(np64(got[0]) - ref[0]).max() <= 2e-3
    assert np.abs(np64(got[1]) - ref[1]).max() <= 1e-4 * np.abs(ref[1]).max()


@pytest.mark.parametrize("graphs", [False, True])
def test_streams_and_graphs(graphs):
    import compressed_attention_cvq_b200 as cvq
    a = setup([900, 0, 333, 64], 8, 2, 16, "bf16", "bf16", seed=12)
    n = cvq.paged_suggest_splits(a[0])
    ws = [cvq.paged_workspace_alloc(a[0], n, "cuda") for _ in range(2)]
    want = cvq.paged_attend(*a, n, workspace=ws[0])
    torch.cuda.synchronize()
    outs = []
    if graphs:                                               # two graphs, one workspace
        gs = []
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                outs.append(cvq.paged_attend(*a, n, workspace=ws[1]))
            gs.append(g)
        for g in gs + gs:
            g.replay()
    else:                                                    # two calls at once
        for w in ws:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                outs.append(cvq.paged_attend(*a, n, workspace=w))
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])


def test_short_sequences_in_a_wide_table():
    """A page table with room for 64K tokens and sequences of a few: every split count of the
    capacity's rule serves them, and the split follows the sequence."""
    import compressed_attention_cvq_b200 as cvq
    lens = [700, 0, 257, 64, 1025]
    a = setup(lens, 8, 2, 16, "bf16", "bf16", seed=21, width=4096)
    for n in (None, 1, 4, 300):
        verify(cvq.paged_attend(*a, n), *a[1:], "bf16", "bf16")


@pytest.mark.parametrize("call", ["append", "attend", "prefix", "prefix fp32"])
def test_captured_behind_a_copy_a_memset_and_a_join(call):
    """The kernels are launched under the end of whatever comes before them in the stream: in a
    graph also behind a copy, a memset and another stream, whose results they must see."""
    import compressed_attention_cvq_b200 as cvq
    if call == "append":
        pg, q, k, v, off, lens, table, kp, vp = append_case([3, 40], [5, 0], 8, 2, 16, "bf16", "bf16", 1)
        x, run = q, lambda: cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q)
    elif call == "attend":
        a = setup([300, 50], 8, 2, 16, "bf16", "bf16", seed=3)
        x = a[1]
        ws = cvq.paged_workspace_alloc(a[0], 4, "cuda")
        run = lambda: cvq.paged_attend(*a, 4, workspace=ws)[0]                     # noqa: E731
    else:
        d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=640, R=2, seed=4)
        dev = {n: torch.from_numpy(d[n]).cuda() for n in ("key_cb", "val_cb", "key_codes", "val_codes")}
        x = torch.randn(4, 8, 128, device="cuda").to(torch.float32 if "fp32" in call else torch.bfloat16)
        shape, ln = cvq.shape_of(x, dev["key_codes"]), i32([600])
        n = cvq.prefix_suggest_splits(shape, x.dtype)
        ws = cvq.prefix_workspace_alloc(shape, n, "cuda")
        run = lambda: cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"],  # noqa: E731
                                        dev["val_codes"], ln, dev["val_cb"], n, workspace=ws)[0]
    keep = x.clone()
    want = run().clone()
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.zero_()                                            # a memset or a kernel
        other.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(other):
            x[:1].copy_(keep[:1])
        x[1:].copy_(keep[1:])                                # copies on both branches
        torch.cuda.current_stream().wait_stream(other)
        got = run()
        after = got.clone()
    for _ in range(3):
        x.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        n = slice(None) if call != "append" else slice(0, 43)
        assert torch.equal(got[n], want[n]) and torch.equal(after[n], want[n])


@pytest.mark.parametrize("cache,scale", [("bf16", 2.0 ** 125), ("fp16", 2.0 ** 13), ("bf16", 2.0 ** -120)])
def test_values_near_the_ends_of_their_type(cache, scale):
    """Sums of weights and values stay inside fp32 wherever the output does."""
    import compressed_attention_cvq_b200 as cvq
    a = list(setup([700, 64], 8, 2, 16, "bf16", cache, seed=14))
    a[3] = (a[3].float().clamp(-1.9, 1.9) * scale).to(DT[cache])
    for n in (1, 2):
        out, lse = cvq.paged_attend(*a, n, out_dtype=torch.float32)
        # in units of the scale, where the absolute terms of the tolerance belong
        b = list(a)
        b[3] = a[3].double() / scale
        verify((out.double() / scale, lse), *b[1:], "bf16", cache, None, "fp32")


def test_the_stream_argument():
    import compressed_attention_cvq_b200 as cvq
    st = torch.cuda.Stream()
    a = setup([300, 50], 8, 2, 16, "bf16", "bf16", seed=3)
    want = cvq.paged_attend(*a)
    pg, q, k, v, off, lens, table, kp, vp = append_case([3, 40], [5, 0], 8, 2, 16, "bf16", "bf16", 1)
    want_q = cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q)
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=640, R=2, seed=4)
    dev = {n: torch.from_numpy(d[n]).cuda() for n in ("key_cb", "val_cb", "key_codes", "val_codes")}
    x = torch.randn(4, 8, 128, device="cuda").bfloat16()
    shape, ln = cvq.shape_of(x, dev["key_codes"]), i32([600])

    def prefix(**kw):
        return cvq.prefix_attend(shape, x, dev["key_cb"], dev["key_codes"], dev["val_codes"], ln,
                                 dev["val_cb"], **kw)
    want_p = prefix()
    outs = [[torch.zeros_like(y) for y in w] for w in (want, want_p)]
    q_out = torch.zeros_like(want_q)
    ws = cvq.paged_workspace_alloc(a[0], cvq.paged_suggest_splits(a[0]), "cuda")
    wp = cvq.prefix_workspace_alloc(shape, cvq.prefix_suggest_splits(shape, x.dtype), "cuda")
    torch.cuda.synchronize()
    cvq.paged_attend(*a, workspace=ws, out=outs[0][0], lse=outs[0][1], stream=st)
    prefix(workspace=wp, out=outs[1][0], lse=outs[1][1], stream=st)
    cvq.paged_append(pg, k, v, off, lens, table, kp, vp, q=q, q_out=q_out, stream=st)
    st.synchronize()
    for got, w in zip(outs, (want, want_p)):
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
    assert torch.equal(q_out[:43], want_q[:43])


def test_tensors_that_do_not_fit_are_refused():
    """Every wrong tensor of the three calls is a ValueError that names it, before any launch."""
    import compressed_attention_cvq_b200 as cvq
    pg, q, kp, vp, table, lens = setup([40, 3], 8, 2, 16, "bf16", "bf16", seed=1)
    ws = cvq.paged_workspace_alloc(pg, 2, "cuda")
    state = (torch.zeros(2, 8, 128, device="cuda"), torch.zeros(2, 8, device="cuda"))
    base = dict(q=q, k_pages=kp, v_pages=vp, page_table=table, seq_lens=lens, n_splits=2,
                workspace=ws, prev=state)
    bad = [dict(q=q.cpu()), dict(q=q[:1]), dict(q=q.double()), dict(q=q.transpose(0, 1)),
           dict(q=q.expand(2, 8, 128)[:, :, :64]), dict(k_pages=kp.half()), dict(v_pages=vp[:-1]),
           dict(k_pages=kp.transpose(1, 2)), dict(v_pages=vp.cpu()), dict(page_table=table.long()),
           dict(page_table=table[:, :1].contiguous()), dict(page_table=table.t().contiguous().t()),
           dict(seq_lens=lens[:1]), dict(seq_lens=lens.float()), dict(workspace=ws[:100]),
           dict(workspace=ws.cpu()), dict(n_splits=0), dict(n_splits=5000),
           dict(prev=(state[0].half(), state[1])), dict(prev=(state[0], state[1][:, :4])),
           dict(prev=(state[0].cpu(), state[1])), dict(out=q.float()[:1]), dict(lse=state[1].double()),
           dict(out=state[0], out_dtype=torch.bfloat16), dict(out_dtype=torch.float64)]
    for kw in bad:
        with pytest.raises(ValueError):
            cvq.paged_attend(pg, **{**base, **kw})
    for kw in (dict(q=None), dict(k_pages=3), dict(out_dtype="bf16")):
        with pytest.raises(TypeError):
            cvq.paged_attend(pg, **{**base, **kw})
    apg, aq, k, v, off, al, at, akp, avp = append_case([3, 4], [0, 2], 8, 2, 16, "bf16", "bf16")
    base = dict(k=k, v=v, tok_offsets=off, seq_lens=al, page_table=at, k_pages=akp, v_pages=avp, q=aq)
    before = akp.clone()
    for kw in [dict(k=k.cpu()), dict(k=k.double()), dict(v=v.float()), dict(v=v[:3]), dict(q=aq[:, :4]),
               dict(q=aq.half()), dict(k=k[:, :, ::2]), dict(q=aq.transpose(1, 2)),
               dict(tok_offsets=off[:2]), dict(tok_offsets=off.long()), dict(seq_lens=al.cpu()),
               dict(pos_offsets=al[:1]), dict(pos_offsets=al.float()), dict(q_out=aq.float()),
               dict(q_out=aq[:3]), dict(q=None, q_out=aq), dict(k_pages=akp.half()), dict(k=k[0])]:
        with pytest.raises(ValueError):
            cvq.paged_append(apg, **{**base, **kw})
    odd = torch.zeros(7 * (256 + 4), dtype=torch.bfloat16, device="cuda").as_strided((7, 2, 128), (260, 128, 1))
    with pytest.raises(cvq.CvqError):                        # a token stride of 520 bytes
        cvq.paged_append(apg, **{**base, "k": odd})
    assert torch.equal(akp, before)
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=640, R=2, seed=4)
    dev = {n: torch.from_numpy(d[n]).cuda() for n in ("key_cb", "val_cb", "key_codes", "val_codes")}
    x = torch.randn(4, 8, 128, device="cuda").bfloat16()
    shape = cvq.shape_of(x, dev["key_codes"])
    base = dict(q=x, prefix_len=i32([600]), **dev)
    for kw in [dict(q=x.cpu()), dict(q=x[:3]), dict(q=x.double()), dict(prefix_len=i32([6, 6])),
               dict(prefix_len=i32([6]).long()), dict(key_cb=dev["key_cb"].half()),
               dict(key_cb=dev["val_cb"]), dict(val_cb=dev["key_cb"]), dict(key_cb=dev["key_cb"][:1]),
               dict(key_codes=dev["key_codes"][:, :, :639]), dict(val_codes=dev["val_codes"].int()),
               dict(val_codes=dev["val_codes"].cpu()), dict(key_codes=dev["key_codes"].transpose(2, 3)),
               dict(n_splits=0), dict(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda")),
               dict(out=x.float()[:2]), dict(out_dtype=torch.int8)]:
        with pytest.raises(ValueError):
            cvq.prefix_attend(shape, **{**base, **kw})
    cvq.prefix_attend(shape, **base)
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("cache,Hq,bound", [("bf16", 8, 3e-6), ("fp16", 8, 3e-6), ("bf16", 2, 3e-6)])
def test_fp32_outputs_over_long_sequences(cache, Hq, bound):
    """Relative to the result's norm: operands in three parts are off by 2^-24 each (fp16 pages, two:
    2^-22), sums of 64 chunks in the accumulators by at most 64 x 2^-23 x 1/2 of their own size
    on average, and those sums, taken every 64 chunks, by one rounding: below 64 x 2^-24 = 3.8e-6
    at the worst, and less as the accumulators start from nothing (half of it) and the errors of
    128 dims and 4 warps are not all of one sign (3e-6 leaves room for the scores' 2^-22 x |s|)."""
    import compressed_attention_cvq_b200 as cvq
    a = setup([30000, 9000, 70], Hq, 2, 32, "fp32", cache, seed=8)
    out, lse = cvq.paged_attend(*a)
    ref = U.paged_reference(np64(a[1]), np64(a[2]), np64(a[3]), a[4].cpu().numpy(), a[5].tolist())
    for b in range(3):
        assert np.linalg.norm(np64(out)[b] - ref[0][b]) <= bound * np.linalg.norm(ref[0][b])
        assert np.abs(np64(lse)[b] - ref[1][b]).max() <= 1e-6 * np.abs(ref[1][b]).max()
