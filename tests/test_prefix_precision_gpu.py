"""cvq_prefix_attend of 16-bit queries holds what fp32 holds, whatever kernel a call takes: outputs
and lse against the float64 definition, far inside the tolerances of fp16 operands."""
import numpy as np
import pytest
import torch

import serve_util as U
import workloads

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}

# Relative errors of one product's factors, by the arithmetic of the kernels.
#   key: its rounds' fp32 sum (R 2^-24), the rotation (2^-23), a phase that was turned on 15 times
#     at most (15 times its own rounding and its step's: 30 2^-24 < 2^-19), two 11-bit parts (2^-22)
#   value: the sum, and two parts; weight: exp2 (2^-22) of a score, and two parts
SCORE = 2.0 ** -19 + 2.0 ** -21
VALUE = 2.0 ** -20
WEIGHT = 2.0 ** -21
# Outputs are summed by instructions that cut off: 2^-23 of what is held, 12 times a tile of 64 tokens,
# 16 tiles at most before the sum is taken up in fp32 (some tens of such sums, rounded to 2^-24 each).
CUTS = (12 * 16 + 32) * 2.0 ** -23


def run(B, Hq, Hkv, t_cap, length, R, dtype, group=8, n_splits=None, seed=0, std=None, out="fp32", **kw):
    import compressed_attention_cvq_b200 as cvq

    d = workloads.small(batch=1, n_q_heads=Hq, n_kv_heads=Hkv, t_cap=t_cap, R=R, seed=seed,
                        cb_std=std or (1.0 / R) ** 0.5, group_dim=group)
    q = torch.from_numpy(np.random.default_rng(seed + 1).standard_normal((B, Hq, 128))).to(DT[dtype])
    d["q"] = q.double().numpy()
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    shape = cvq.shape_of(q, dev["key_codes"], group_dim=group)
    ln = torch.tensor([length], dtype=torch.int32, device="cuda")
    got = cvq.prefix_attend(shape, q.cuda(), dev["key_cb"], dev["key_codes"], dev["val_codes"], ln,
                            dev["val_cb"], n_splits, out_dtype=DT[out], **kw)
    assert cvq.fault_status(clear=True) == 0
    return d, got


def check(d, got, length, out="fp32"):
    out_, lse_ = (x.double().cpu().numpy() for x in got)
    ref_o, ref_l = U.prefix_reference(d, length)
    B, Hq, _ = ref_o.shape
    Hkv = d["key_codes"].shape[1]
    g = Hq // Hkv
    tol_o, tol_l = np.zeros_like(ref_o), np.zeros_like(ref_l)
    for h in range(Hkv):
        kcb = d["key_cb"][h].astype(np.float64)
        k = U.rotate(U.decode(d["key_codes"][0, h], kcb.reshape(*kcb.shape[:3], -1), d["group_dim"])[:length],
                     np.arange(length))
        vcb = d["val_cb"][h].astype(np.float64)
        v = U.decode(d["val_codes"][0, h], vcb, d["group_dim"])[:length]
        v_sq = v ** 2 + U.decode(d["val_codes"][0, h], vcb ** 2, d["group_dim"])[:length]
        sl = slice(h * g, (h + 1) * g)
        for b in range(B):
            rows = d["q"][b, sl]
            tol_o[b, sl], tol_l[b, sl] = U.state_tolerance(rows, k, v, ref_o[b, sl], ref_l[b, sl],
                                                           SCORE, VALUE, WEIGHT, 64, v_sq)
            # what a running sum holds at most, in units of the final sum of weights
            p = np.exp(rows @ k.T / np.sqrt(128) - ref_l[b, sl][:, None])
            for i in range(g):
                most = np.abs(np.cumsum(p[i][:, None] * v, 0)).max(0)
                # a split or a stream may hold the difference of two such sums
                tol_o[b, sl.start + i] += CUTS * 2 * most
    U.check(out_, lse_, ref_o, ref_l, tol_o, tol_l, U.HALF[out])


@pytest.mark.parametrize("group,R", [(8, 1), (8, 2), (64, 1), (64, 9), (64, 10), (64, 11), (64, 12), (64, 22)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("t_cap,length", [(320, 319), (2304, 2300)])      # a kernel each
def test_as_exact_as_fp32(group, R, dtype, t_cap, length):
    d, got = run(5, 8, 2, t_cap, length, R, dtype, group, seed=R)
    check(d, got, length)


@pytest.mark.parametrize("length", [1, 3, 64, 100, 500])
@pytest.mark.parametrize("group,R", [(8, 1), (8, 2), (64, 3)])
def test_few_tokens_in_a_large_cache(length, group, R):
    """Nothing averages out over a few tokens: a score that is off is an lse that is off."""
    d, got = run(3, 8, 2, 4096, length, R, "bf16", group, seed=length)
    check(d, got, length)


@pytest.mark.parametrize("group,R", [(8, 1), (8, 2), (64, 2)])
@pytest.mark.parametrize("n_splits", [1, 2])
def test_long_streams_do_not_drift(group, R, n_splits):
    """A cluster of CTAs that takes tens of thousands of tokens alone: sums in the matrix
    instructions are taken up in fp32 on the way."""
    d, got = run(2, 4, 1, 40000, 39999, R, "bf16", group, n_splits, seed=R)
    check(d, got, 39999)


def test_sharp_scores_stay_exact():
    """Nearly one-hot rows: the maximum moves, and one value's parts are the output."""
    for R in (1, 2):
        d, got = run(4, 8, 2, 2500, 2500, R, "bf16", seed=6, std=3.0)
        check(d, got, 2500)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_of_the_queries_type_are_rounded_once(dtype):
    for group, R in ((8, 1), (8, 2), (64, 11)):
        d, got = run(6, 8, 2, 4096, 4001, R, dtype, group, seed=3, out=dtype)
        check(d, got, 4001, dtype)


@pytest.mark.parametrize("group,R", [(8, 1), (8, 2), (64, 2)])
def test_tiny_queries_and_codebooks(group, R):
    """Scores that are nothing beside 1: every token weighs the same, also in a tile that the prefix
    fills in part (masked scores times a scale that underflows would be NaN)."""
    import compressed_attention_cvq_b200 as cvq
    d = workloads.small(batch=1, n_q_heads=8, n_kv_heads=2, t_cap=2304, R=R, seed=1, group_dim=group)
    d["key_cb"] = (d["key_cb"] * np.float32(2.0 ** -100)).astype(np.float32)
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    q = (torch.randn(3, 8, 128, dtype=torch.float64) * 2.0 ** -60).bfloat16()
    d["q"] = q.double().numpy()
    ln = torch.tensor([2111], dtype=torch.int32, device="cuda")
    got = cvq.prefix_attend(cvq.shape_of(q, dev["key_codes"], group_dim=group), q.cuda(), dev["key_cb"],
                            dev["key_codes"], dev["val_codes"], ln, dev["val_cb"], out_dtype=torch.float32)
    check(d, got, 2111)


@pytest.mark.parametrize("t_cap", [16, 48, 272, 2064, 2096])
@pytest.mark.parametrize("R", [1, 5, 11, 14])
def test_capacities_of_16_tokens(t_cap, R):
    """One-byte codes of 64-scalar groups: rows are whole pieces of 16 bytes, not of 64."""
    for length in (t_cap, t_cap - 9):
        d, got = run(3, 8, 2, t_cap, length, R, "fp16", 64, seed=t_cap + R)
        check(d, got, length)


@pytest.mark.parametrize("group,R", [(64, 14), (64, 22), (8, 2), (8, 1)])
def test_layers_that_share_a_workspace(group, R):
    """Calls with codebooks of their own, one after another through one workspace: rounds that are not
    held in shared memory come from this call's codebooks."""
    import compressed_attention_cvq_b200 as cvq
    layers = [run(4, 8, 2, 2304, 2200, R, "bf16", group, 2, seed=s) for s in (1, 2, 3)]
    shape = cvq.shape_of(torch.zeros(4, 8, 128), torch.from_numpy(layers[0][0]["key_codes"]), group_dim=group)
    ws = cvq.prefix_workspace_alloc(shape, 2, "cuda")
    ins = []
    for d, _ in layers:
        dev = [torch.from_numpy(d[k]).cuda() for k in ("key_cb", "key_codes", "val_codes", "val_cb")]
        ins.append((torch.from_numpy(d["q"]).bfloat16().cuda(), dev))
    ln = torch.tensor([2200], dtype=torch.int32, device="cuda")
    for _ in range(3):
        got = [cvq.prefix_attend(shape, q, kcb, kc, vc, ln, vcb, 2, workspace=ws, out_dtype=torch.float32)
               for q, (kcb, kc, vc, vcb) in ins]
        for (o, z), (_, (wo, wz)) in zip(got, layers):
            assert torch.equal(o, wo) and torch.equal(z, wz)
