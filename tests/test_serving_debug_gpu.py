"""The debug build (libcvq_debug.so: -DCVQ_DEBUG_BOUNDS) on small serving calls of every kernel, at odd
batches, lengths and split counts: its range checks of pages, codes, tiles, partial states, counters and
output rows all pass, and the results are those of the other build.  In a child process, because the
binding picks its library when it is first loaded."""
import os
import subprocess
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import numpy as np, torch
sys.path.insert(0, %(root)r)
import workloads
import compressed_attention_cvq_b200 as cvq
from compressed_attention_cvq_b200 import _binding as b
assert b.LIB_PATH.endswith(%(lib)r), b.LIB_PATH
out = []
i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
def done(*ts):
    word = cvq.fault_status(clear=True)
    assert word == 0, (len(out), b.fault_names(word))
    out.extend(t.float().cpu().numpy() for t in ts)
for group, R, cap, n, B, Hq, Hkv, length, dt in (
        (8, 1, 2305, 3, 33, 8, 2, 2300, torch.bfloat16), (8, 2, 2100, 2, 5, 16, 2, 2099, torch.float16),
        (8, 1, 5000, 1, 2, 3, 3, 5000, torch.bfloat16), (64, 3, 2064, 3, 4, 8, 2, 2060, torch.bfloat16),
        (64, 12, 2304, 1, 2, 4, 1, 2300, torch.float16), (8, 1, 200, 2, 3, 8, 2, 199, torch.float32),
        (8, 2, 700, 5, 17, 8, 2, 650, torch.float32), (64, 5, 320, 2, 20, 8, 2, 300, torch.float32)):
    d = workloads.small(batch=1, n_q_heads=Hq, n_kv_heads=Hkv, t_cap=cap, R=R, seed=R + cap, group_dim=group)
    dev = {k: torch.from_numpy(d[k]).cuda() for k in ("key_cb", "val_cb", "key_codes", "val_codes")}
    q = torch.from_numpy(np.random.default_rng(cap).standard_normal((B, Hq, 128))).to(dt).cuda()
    for bits in ((0,) if group == 8 or cap %% 64 else (0, 6)):
        codes = dev["key_codes"], dev["val_codes"]
        shape = cvq.shape_of(q, codes[0], group_dim=group)
        if bits:
            one = cvq.shape_of(q[:1], codes[0], group_dim=group)
            one.code_bits = shape.code_bits = bits
            codes = [cvq.pack_codes6(one, c) for c in codes]
        done(*cvq.prefix_attend(shape, q, dev["key_cb"], *codes, i32([length]), dev["val_cb"], n))
for lens, Hq, Hkv, ps, dt, kv, n in (
        ([1500, 0, 37, 1], 8, 2, 16, torch.bfloat16, torch.bfloat16, 4), ([777], 3, 3, 8, torch.float32, torch.float16, 2),
        ([2049, 2048, 900], 16, 2, 64, torch.float16, torch.float16, 9), ([5, 300], 4, 2, 1, torch.float32, torch.bfloat16, 1)):
    rng, g = np.random.default_rng(ps), torch.Generator(device="cuda").manual_seed(ps)
    m = max(-(-x // ps) for x in lens)
    pool = len(lens) * m
    kp, vp = (torch.randn((pool, Hkv, ps, 128), generator=g, device="cuda").to(kv) for _ in range(2))
    table = i32(rng.permutation(pool).reshape(len(lens), m))
    pg = cvq.make_paged(len(lens), Hq, Hkv, ps, pool, m, kv)
    new = [min(x, 1 + k) for k, x in enumerate(lens)]
    t = sum(new) + 2
    q, k, v = (torch.randn((t, h, 128), generator=g, device="cuda").to(dt) for h in (Hq, Hkv, Hkv))
    qr = torch.zeros_like(q)
    cvq.paged_append(pg, k, v, i32(np.concatenate([[0], np.cumsum(new)])), i32(lens), table, kp, vp, q=q, q_out=qr)
    done(qr, kp, vp)
    done(*cvq.paged_attend(pg, qr[:len(lens)].contiguous(), kp, vp, table, i32(lens), n))
np.savez(sys.argv[1], *out)
"""


def run(tmp_path, debug):
    lib = "libcvq_debug.so" if debug else "libcvq.so"
    env = {k: v for k, v in os.environ.items() if k != "CVQ_LIBRARY"}
    if debug:
        env["CVQ_LIBRARY"] = "debug"
    to = str(tmp_path / (lib + ".npz"))
    r = subprocess.run([sys.executable, "-c", CHILD % {"root": ROOT, "lib": lib}, to], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr
    with np.load(to) as f:
        return [f[k] for k in f.files]


def test_debug_build_of_the_serving_calls(tmp_path):
    if not os.path.exists(os.path.join(ROOT, "compressed_attention_cvq_b200", "libcvq_debug.so")):
        from compressed_attention_cvq_b200 import build
        build.build(debug_bounds=True)
    a, b = run(tmp_path, False), run(tmp_path, True)
    assert len(a) == len(b) > 20
    for x, y in zip(a, b):
        # the same arithmetic, but for products and sums that the compiler may join differently
        assert np.array_equal(np.isfinite(x), np.isfinite(y))
        assert np.allclose(x, y, rtol=2.0 ** -7, atol=1e-5)
