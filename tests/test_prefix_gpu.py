"""cvq_prefix_attend against the float64 definition: both code layouts, every head grouping
and query type, prefixes from nothing to several tiles with odd ends, and the ways a program
calls it (split counts, streams, graphs, shared codebooks, long caches)."""
import numpy as np
import pytest
import torch

import serve_util as U
import workloads

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def make(B, Hq, Hkv, t_cap, R, dtype, group=8, seed=0, shared=False, std=None):
    """Seeded inputs on the device and the same values in float64."""
    d = workloads.small(batch=1, n_q_heads=Hq, n_kv_heads=Hkv, t_cap=t_cap, R=R, seed=seed,
                        cb_std=std or (1.0 / R) ** 0.5, group_dim=group)
    q = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((B, Hq, 128))).to(DT[dtype])
    d["q"] = q.double().numpy()
    if shared:
        d["key_cb"], d["val_cb"] = d["key_cb"][:1], d["val_cb"][:1]
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    if shared:
        dev["key_cb"], dev["val_cb"] = dev["key_cb"][0], dev["val_cb"][0]
    dev["q"] = q.cuda()
    return d, dev


def call(cvq, dev, length, group=8, bits=0, n_splits=None, codes=None, **kw):
    kc, vc = codes or (dev["key_codes"], dev["val_codes"])
    shape = cvq.shape_of(dev["q"], kc, group_dim=group, code_bits=bits)
    ln = torch.tensor([length], dtype=torch.int32, device="cuda")
    return cvq.prefix_attend(shape, dev["q"], dev["key_cb"], kc, vc, ln, dev["val_cb"], n_splits,
                             **kw)


def verify(d, got, length, dtype, out_dtype=None, seen_codes=64):
    out, lse = (x.double().cpu().numpy() for x in got)
    length = min(max(length, 0), d["key_codes"].shape[-1] if d["group_dim"] == 64
                 else d["key_codes"].shape[2])
    ref_o, ref_l = U.prefix_reference(d, length)
    # 16-bit queries may be multiplied as fp16 operands: a decoded key carries the rounding of
    # its R codewords and of the rotated sum, a value that of its codewords and sum, a weight
    # one; the queries themselves fit
    R = d["R"]
    e = 0.0 if dtype == "fp32" else U.FP16
    se = e * np.sqrt(2 + R)
    B, Hq, _ = ref_o.shape
    Hkv = d["key_codes"].shape[1]
    g = Hq // Hkv
    tol_o, tol_l = np.zeros_like(ref_o), np.zeros_like(ref_l)
    for h in range(Hkv):
        hc = h if d["key_cb"].shape[0] > 1 else 0
        kcb = d["key_cb"][hc].astype(np.float64)
        k = U.rotate(U.decode(d["key_codes"][0, h], kcb.reshape(*kcb.shape[:3], -1), d["group_dim"])[:length],
                     np.arange(length))
        vcb = d["val_cb"][hc].astype(np.float64)
        v = U.decode(d["val_codes"][0, h], vcb, d["group_dim"])[:length]
        # a value sum_r c_r comes out as (sum_r c_r (1 + a_r)) (1 + b) with independent a_r, b of
        # at most e: off by sum_r c_r a_r + b v, whose variance is e^2 / 3 (sum_r c_r^2 + v^2).
        # The codewords may cancel, so this is not bounded by a multiple of v^2
        v_sq = v ** 2 + U.decode(d["val_codes"][0, h], vcb ** 2, d["group_dim"])[:length]
        sl = slice(h * g, (h + 1) * g)
        for b in range(B):
            tol_o[b, sl], tol_l[b, sl] = U.state_tolerance(
                d["q"][b, sl], k, v, ref_o[b, sl], ref_l[b, sl], se, e, e, seen_codes, v_sq)
    U.check(out, lse, ref_o, ref_l, tol_o, tol_l, U.HALF[out_dtype or dtype])


@pytest.mark.parametrize("B,Hq,Hkv,t_cap,length,R,dtype", [
    (4, 32, 8, 1000, 1000, 1, "fp32"),
    (1, 4, 1, 64, 64, 1, "bf16"),
    (1, 1, 1, 1, 1, 1, "bf16"),
    (3, 8, 2, 700, 699, 2, "bf16"),
    (16, 32, 8, 1024, 1024, 2, "bf16"),
    (5, 16, 2, 1500, 1237, 2, "fp16"),        # 8 query heads per KV head
    (33, 4, 1, 640, 513, 1, "bf16"),          # 132 rows of one KV head
    (70, 8, 2, 900, 897, 2, "fp16"),          # 280 rows
    (9, 6, 3, 2000, 1999, 1, "bf16"),         # 2 query heads per KV head
    (17, 3, 3, 1300, 1281, 2, "fp16"),        # as many KV heads as query heads
    (130, 8, 1, 300, 255, 2, "bf16"),         # 1040 rows
    (2, 8, 2, 4096, 4095, 2, "fp32"),
    (40, 8, 2, 500, 500, 1, "fp32"),
    (7, 32, 8, 5000, 4900, 1, "fp16"),
])
def test_matches_the_definition(B, Hq, Hkv, t_cap, length, R, dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(B, Hq, Hkv, t_cap, R, dtype, seed=B + t_cap)
    verify(d, call(cvq, dev, length), length, dtype)
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("B,Hq,Hkv,t_cap,length,R,dtype,bits", [
    (2, 8, 2, 512, 512, 11, "bf16", 6), (3, 8, 2, 512, 301, 11, "fp32", 8),
    (5, 4, 1, 1024, 1000, 21, "fp16", 6), (20, 16, 2, 320, 319, 1, "bf16", 8),
    (1, 2, 1, 64, 1, 22, "bf16", 6), (9, 8, 8, 1280, 1277, 5, "bf16", 8),
])
def test_paper_layout(B, Hq, Hkv, t_cap, length, R, dtype, bits):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(B, Hq, Hkv, t_cap, R, dtype, 64, seed=R)
    codes = None
    if bits == 6:
        shape = cvq.shape_of(dev["q"][:1], dev["key_codes"], group_dim=64)
        shape.code_bits = 6
        codes = [cvq.pack_codes6(shape, dev[k]) for k in ("key_codes", "val_codes")]
    verify(d, call(cvq, dev, length, 64, bits, codes=codes), length, dtype)
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("length", [-5, 0, 1, 2, 63, 64, 65, 127, 128, 129, 400, 10 ** 6])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_lengths_from_nothing(length, dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(6, 8, 2, 400, 2, dtype, seed=5)
    for n in (1, 3):
        verify(d, call(cvq, dev, length, n_splits=n), length, dtype)


def test_empty_capacity():
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(2, 8, 2, 64, 1, "bf16")
    dev["key_codes"], dev["val_codes"] = dev["key_codes"][:, :, :0], dev["val_codes"][:, :, :0]
    some = torch.zeros(64, dtype=torch.uint8, device="cuda")
    shape = cvq.shape_of(dev["q"], dev["key_codes"])
    # an empty tensor has no address: the library asks for one, as its other calls do
    with pytest.raises(cvq.CvqError):
        call(cvq, dev, 0, n_splits=1)
    from compressed_attention_cvq_b200 import _binding as b
    import ctypes
    ws = cvq.prefix_workspace_alloc(shape, 1, "cuda")
    out = torch.full((2, 8, 128), 7.0, device="cuda")
    lse = torch.full((2, 8), 7.0, device="cuda")
    ln = torch.tensor([3], dtype=torch.int32, device="cuda")
    b.check(b.lib.cvq_prefix_attend(
        ctypes.byref(shape), dev["q"].data_ptr(), b.CVQ_BF16, dev["key_cb"].data_ptr(), 0,
        some.data_ptr(), some.data_ptr(), ln.data_ptr(), dev["val_cb"].data_ptr(), 0, 1,
        ws.data_ptr(), out.data_ptr(), b.CVQ_F32, lse.data_ptr(),
        torch.cuda.current_stream().cuda_stream), "prefix")
    assert torch.all(out == 0) and torch.all(lse == -torch.inf)


@pytest.mark.parametrize("n_splits", [1, 2, 5, 17, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_any_split_count_and_output_type(n_splits, dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(12, 8, 2, 2100, 2, dtype, seed=9)
    for od in ("fp32", "bf16", "fp16"):
        got = call(cvq, dev, 2077, n_splits=n_splits, out_dtype=DT[od])
        assert got[0].dtype == DT[od]
        verify(d, got, 2077, dtype, od)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_shared_codebook_and_repeated_codes(dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(10, 8, 2, 600, 2, dtype, shared=True, seed=3)
    verify(d, call(cvq, dev, 600), 600, dtype)
    # every token the same code: all keys the same but for their rotation, every value equal
    for k in ("key_codes", "val_codes"):
        d[k][:] = 255
        dev[k].fill_(255)
    # every token then carries the same roundings a_r, b: out = sum_t p_t (v + dv) = v + dv, so
    # that nothing averages out (one independent error instead of 64)
    verify(d, call(cvq, dev, 600), 600, dtype, seen_codes=1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_what_lies_behind_the_prefix_does_not_matter(dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(8, 8, 2, 1000, 1, dtype, seed=4)
    # entry 0 of every codebook is not finite, and only tokens behind the prefix use it
    for k in ("key_codes", "val_codes"):
        d[k][d[k] == 0] = 1
        dev[k].copy_(torch.from_numpy(d[k]))
    want = call(cvq, dev, 777)
    dev["key_cb"][:, :, :, 0] = float("nan")
    dev["val_cb"][:, :, :, 0] = float("inf")
    for k in ("key_codes", "val_codes"):
        dev[k][:, :, 777:] = 0
    got = call(cvq, dev, 777)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sharp_and_large_scores(dtype):
    """Keys ten times as large: the softmax is nearly one-hot and its maximum moves."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(4, 8, 2, 1500, 2, dtype, seed=6, std=7.0)
    verify(d, call(cvq, dev, 1500), 1500, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_same_bits_every_time(dtype):
    import compressed_attention_cvq_b200 as cvq
    _, dev = make(20, 16, 4, 3000, 2, dtype, seed=7)
    a = call(cvq, dev, 2999)
    for _ in range(3):
        b = call(cvq, dev, 2999)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_streams_and_graphs(dtype):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(16, 8, 2, 1200, 2, dtype, seed=8)
    shape = cvq.shape_of(dev["q"], dev["key_codes"])
    n = cvq.prefix_suggest_splits(shape, DT[dtype])
    ln = torch.tensor([1111], dtype=torch.int32, device="cuda")

    def go(ws, o=None, z=None):
        return cvq.prefix_attend(shape, dev["q"], dev["key_cb"], dev["key_codes"],
                                 dev["val_codes"], ln, dev["val_cb"], n, workspace=ws, out=o, lse=z)

    ws = [cvq.prefix_workspace_alloc(shape, n, "cuda") for _ in range(3)]
    want = go(ws[0])
    torch.cuda.synchronize()
    # two calls at once on two streams
    got = []
    for w in ws[:2]:
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got.append(go(w))
    torch.cuda.synchronize()
    # two captured graphs that share one workspace, replayed one after the other with another
    # length and other queries
    outs = [(torch.empty_like(want[0]), torch.empty_like(want[1])) for _ in range(2)]
    graphs = []
    for o, z in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go(ws[2], o, z)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o, z in got + outs:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])
    ln.fill_(70)
    graphs[0].replay()
    torch.cuda.synchronize()
    verify(d, outs[0], 70, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_head_offsets_past_32_bits(dtype):
    """A cache capacity whose later heads start beyond 2^31 code bytes."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(3, 16, 4, 512, 2, dtype, seed=11)
    cap = 18_000_000
    kc, vc = (torch.empty((1, 4, cap, 2, 16), dtype=torch.uint8, device="cuda") for _ in range(2))
    assert 3 * cap * 32 > 2 ** 31 // 2 and 4 * cap * 32 > 2 ** 31
    kc[:, :, :512], vc[:, :, :512] = dev["key_codes"], dev["val_codes"]
    # whole splits are empty: only the first holds the 500 tokens
    verify(d, call(cvq, dev, 500, codes=(kc, vc), n_splits=2), 500, dtype)


@pytest.mark.parametrize("group,R,bits", [(8, 1, 0), (8, 2, 0), (64, 1, 8), (64, 4, 6), (64, 11, 8)])
@pytest.mark.parametrize("length", [0, 1, 63, 64, 65, 127, 129, 192, 513, 640])
@pytest.mark.parametrize("cap", [640, 2048])         # in fp32, and on the tensor cores
def test_short_prefixes_in_a_larger_cache(group, R, bits, length, cap):
    """Lengths around the tiles of 64 and the pairs' steps of 128 tokens, in a cache with more
    room, as one split and as several."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(5, 8, 2, cap, R, "fp16", group, seed=R + length)
    codes = None
    if bits == 6:
        shape = cvq.shape_of(dev["q"][:1], dev["key_codes"], group_dim=64)
        shape.code_bits = 6
        codes = [cvq.pack_codes6(shape, dev[k]) for k in ("key_codes", "val_codes")]
    for n in (1, 3):
        verify(d, call(cvq, dev, length, group, bits, n, codes), length, "fp16")
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("B,g", [(31, 4), (32, 4), (33, 4), (128, 1), (129, 1), (32, 8), (1, 8)])
@pytest.mark.parametrize("R", [1, 2])
def test_row_counts_around_a_block(B, g, R):
    """124 to 258 rows of a KV head, and 8: a block holds 128."""
    import compressed_attention_cvq_b200 as cvq
    for cap in (700, 2050):
        d, dev = make(B, 2 * g, 2, cap, R, "bf16", seed=B + R)
        verify(d, call(cvq, dev, 690), 690, "bf16")


@pytest.mark.parametrize("group,R", [(8, 1), (8, 2), (64, 3), (64, 11)])
@pytest.mark.parametrize("k_scale,v_scale", [(2.0 ** 20, 1.0), (2.0 ** -30, 2.0 ** -40), (1.0, 2.0 ** 60),
                                             (2.0 ** 12, 2.0 ** 110)])
@pytest.mark.parametrize("cap", [640, 2048])
def test_codebooks_far_from_one(group, R, k_scale, v_scale, cap):
    """Codebooks that leave fp16's range as they are; the queries take the keys' scale back."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(4, 8, 2, cap, R, "bf16", group, seed=R)
    for name, f in (("key_cb", k_scale), ("val_cb", v_scale)):
        d[name] = (d[name] * np.float32(f)).astype(np.float32)
        dev[name] = torch.from_numpy(d[name]).cuda()
    dev["q"] = (dev["q"].double() / k_scale).bfloat16()
    d["q"] = dev["q"].double().cpu().numpy()
    got = call(cvq, dev, 600, group, out_dtype=torch.float32)
    # measured in units of the values' scale, where the absolute terms of the tolerance belong
    d["val_cb"] = d["val_cb"] / v_scale
    verify(d, (got[0].double() / v_scale, got[1]), 600, "bf16", "fp32")


@pytest.mark.parametrize("cap", [640, 2048])
def test_queries_far_from_one(cap):
    import compressed_attention_cvq_b200 as cvq
    for f in (2.0 ** -100, 2.0 ** 90):
        d, dev = make(3, 8, 2, cap, 2, "bf16", seed=2)
        d["key_cb"] = (d["key_cb"] / np.float32(f)).astype(np.float32)
        dev["key_cb"] = torch.from_numpy(d["key_cb"]).cuda()
        dev["q"] = (dev["q"].double() * f).bfloat16()
        d["q"] = dev["q"].double().cpu().numpy()
        verify(d, call(cvq, dev, 640), 640, "bf16")
    # a row of zeros attends evenly; a row that is not finite leaves the others alone
    d, dev = make(3, 8, 2, cap, 2, "bf16", seed=3)
    want = call(cvq, dev, 640)
    dev["q"][0, 1] = 0
    dev["q"][1, 5, 7] = float("nan")
    dev["q"][2, 2, 9] = float("inf")
    out, lse = call(cvq, dev, 640)
    assert torch.allclose(lse[0, 1], torch.tensor(640.0).log().cuda(), atol=1e-6)
    assert torch.isnan(out[1, 5]).all() and torch.isnan(lse[1, 5]) and torch.isnan(out[2, 2]).all()
    same = torch.ones(3, 8, dtype=torch.bool)
    same[0, 1] = same[1, 5] = same[2, 2] = False
    assert torch.equal(out[same], want[0][same]) and torch.equal(lse[same], want[1][same])


@pytest.mark.parametrize("R,dtype,bits", [(12, "bf16", 6), (22, "fp16", 8), (21, "fp32", 6)])
@pytest.mark.parametrize("cap", [640, 2048])
def test_many_rounds(R, dtype, bits, cap):
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(6, 8, 2, cap, R, dtype, 64, seed=R)
    codes = None
    if bits == 6:
        shape = cvq.shape_of(dev["q"][:1], dev["key_codes"], group_dim=64)
        shape.code_bits = 6
        codes = [cvq.pack_codes6(shape, dev[k]) for k in ("key_codes", "val_codes")]
    verify(d, call(cvq, dev, 601, 64, bits, codes=codes), 601, dtype)


def test_long_streams_keep_their_phases():
    """A split of hundreds of tiles: the keys' turning phases are taken anew every 64 tiles."""
    import compressed_attention_cvq_b200 as cvq
    for R, group in ((1, 8), (2, 8), (2, 64)):
        d, dev = make(2, 4, 1, 30016, R, "fp16", group, seed=R)
        verify(d, call(cvq, dev, 30001, group, n_splits=1), 30001, "fp16")


@pytest.mark.parametrize("R", [12, 13, 16, 17, 21])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** 25])
def test_rounds_beyond_the_held_ones(R, scale):
    """More rounds than a pair of SMs holds: the others come from the workspace's copy, or, where
    their scale is not the usual one, from the codebooks."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(7, 8, 2, 2048, R, "fp16", 64, seed=R)
    for name in ("key_cb", "val_cb"):
        d[name] = (d[name] * np.float32(scale)).astype(np.float32)
        dev[name] = torch.from_numpy(d[name]).cuda()
    if scale > 1:
        # keys of 2^10 and queries of 2^-10, all exact, so that scores stay as they were
        d["key_cb"] /= np.float32(scale / 2.0 ** 10)
        dev["key_cb"] = torch.from_numpy(d["key_cb"]).cuda()
        dev["q"] = (dev["q"].double() / 2.0 ** 10).half()
    d["q"] = dev["q"].double().cpu().numpy()
    got = call(cvq, dev, 1000, 64, 0, 2, out_dtype=torch.float32)
    d["val_cb"] = d["val_cb"] / scale
    verify(d, (got[0].double() / scale, got[1]), 1000, "fp16", "fp32")
    assert cvq.fault_status(clear=True) == 0


@pytest.mark.parametrize("R", [1, 2])
def test_the_tensor_cores_calls(R):
    """What the tests above ask of small caches in fp32, of a cache large enough for the tensor
    cores: one codebook for all heads, one code for all tokens, what lies behind the prefix, sharp
    scores, streams and graphs with one workspace, any output type and split count."""
    import compressed_attention_cvq_b200 as cvq
    d, dev = make(10, 8, 2, 2100, R, "bf16", shared=True, seed=3)
    verify(d, call(cvq, dev, 2100), 2100, "bf16")
    for k in ("key_codes", "val_codes"):
        d[k][:] = 255
        dev[k].fill_(255)
    verify(d, call(cvq, dev, 2100), 2100, "bf16", seen_codes=1)
    d, dev = make(4, 8, 2, 2500, R, "bf16", seed=6, std=7.0)
    verify(d, call(cvq, dev, 2500), 2500, "bf16")
    d, dev = make(8, 8, 2, 2400, R, "bf16", seed=4)
    for k in ("key_codes", "val_codes"):
        d[k][d[k] == 0] = 1
        dev[k].copy_(torch.from_numpy(d[k]))
    shape = cvq.shape_of(dev["q"], dev["key_codes"])
    n = cvq.prefix_suggest_splits(shape, torch.bfloat16)
    ln = torch.tensor([1777], dtype=torch.int32, device="cuda")
    ws = [cvq.prefix_workspace_alloc(shape, n, "cuda") for _ in range(2)]

    def go(w, **kw):
        return cvq.prefix_attend(shape, dev["q"], dev["key_cb"], dev["key_codes"], dev["val_codes"],
                                 ln, dev["val_cb"], n, workspace=w, **kw)
    want = go(ws[0])
    dev["key_cb"][:, :, :, 0] = float("nan")
    dev["val_cb"][:, :, :, 0] = float("inf")
    for k in ("key_codes", "val_codes"):
        dev[k][:, :, 1777:] = 0
    torch.cuda.synchronize()
    got = []
    for w in ws:                                             # two calls at once
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            got.append(go(w))
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(go(ws[0]))
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    for o, z in got:
        assert torch.equal(o, want[0]) and torch.equal(z, want[1])
    for od in ("fp32", "fp16"):
        for k in (1, 3, 4096):
            verify(d, call(cvq, dev, 1777, n_splits=k, out_dtype=DT[od]), 1777, "bf16", od)
    assert cvq.fault_status(clear=True) == 0
