"""Float64 definitions of the serving operators, by loops over sequences and heads, for the
tests (numpy only)."""
import numpy as np

D = 128
BF16, FP16, FP32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24      # half a step, relative
HALF = {"bf16": BF16, "fp16": FP16, "fp32": FP32}


def rotate(x, pos, base=500000.0):
    """RoPE of x [..., 128] (interleaved pairs) at integer position(s) pos [...]."""
    theta = np.float64(base) ** (-np.arange(64) * 2.0 / D)
    ang = np.asarray(pos, np.float64)[..., None] * theta
    z = (x[..., 0::2] + 1j * x[..., 1::2]) * np.exp(1j * ang)
    return np.stack((z.real, z.imag), -1).reshape(x.shape)


def attention(q, k, v):
    """q [rows, 128] against k, v [T, 128]: (out, lse); T = 0 gives 0 and -inf."""
    if len(k) == 0:
        return np.zeros_like(q), np.full(len(q), -np.inf)
    s = q @ k.T / np.sqrt(D)
    m = s.max(-1, keepdims=True)
    p = np.exp(s - m)
    z = p.sum(-1, keepdims=True)
    return p @ v / z, (m + np.log(z))[:, 0]


def merge(a, b):
    """Two states (out, lse) of the same rows -> the state over both parts; an out whose lse is
    -inf does not count, whatever it holds."""
    (oa, la), (ob, lb) = ((np.where(np.isneginf(z)[..., None], 0.0, o), z) for o, z in (a, b))
    m = np.maximum(la, lb)
    ref = np.where(np.isneginf(m), 0.0, m)
    wa, wb = np.exp(la - ref), np.exp(lb - ref)
    with np.errstate(divide="ignore"):
        lse = ref + np.log(wa + wb)
    den = np.where(wa + wb > 0, wa + wb, 1.0)
    return (wa[..., None] * oa + wb[..., None] * ob) / den[..., None], lse


def decode(codes, cb, group_dim):
    """Codes of one KV head (token-major [T, R, 16], or planar [2, R, T]) and its codebook
    [groups, R, entries, dims] -> [T, 128]."""
    if group_dim == 64:
        codes = np.moveaxis(codes, -1, 0).swapaxes(1, 2)          # [T, R, 2]
    G = np.arange(cb.shape[0])
    return sum(cb[G, r, codes[:, r]] for r in range(cb.shape[1])).reshape(len(codes), D)


def prefix_reference(d, length, base=500000.0):
    """d: workloads.small(..., batch=1) codes with d["q"] [B, Hq, 128]."""
    q = np.asarray(d["q"], np.float64)
    B, Hq, _ = q.shape
    Hkv = d["key_codes"].shape[1]
    g = Hq // Hkv
    out, lse = np.zeros(q.shape), np.zeros((B, Hq))
    for h in range(Hkv):
        hc = h if d["key_cb"].shape[0] > 1 else 0
        kcb = d["key_cb"][hc].astype(np.float64)
        kcb = kcb.reshape(*kcb.shape[:3], -1)
        k = decode(d["key_codes"][0, h], kcb, d["group_dim"])[:length]
        v = decode(d["val_codes"][0, h], d["val_cb"][hc].astype(np.float64), d["group_dim"])[:length]
        k = rotate(k, np.arange(length), base)
        o, z = attention(q[:, h * g:(h + 1) * g].reshape(-1, D), k, v)
        out[:, h * g:(h + 1) * g] = o.reshape(B, g, D)
        lse[:, h * g:(h + 1) * g] = z.reshape(B, g)
    return out, lse


def paged_reference(q, k_pages, v_pages, table, lens, prev=None):
    """q [B, Hq, 128], pools [n, Hkv, ps, 128], table [B, max]: entries outside the pool hold
    no tokens."""
    B, Hq, _ = q.shape
    n, Hkv, ps, _ = k_pages.shape
    g = Hq // Hkv
    out, lse = np.zeros(q.shape), np.zeros((B, Hq))
    for b in range(B):
        p = np.arange(min(max(int(lens[b]), 0), table.shape[1] * ps))
        page = table[b, p // ps]
        p, page = p[(page >= 0) & (page < n)], page[(page >= 0) & (page < n)]
        for h in range(Hkv):
            sl = slice(h * g, (h + 1) * g)
            out[b, sl], lse[b, sl] = attention(q[b, sl], k_pages[page, h, p % ps], v_pages[page, h, p % ps])
    return merge((out, lse), prev) if prev is not None else (out, lse)


def state_tolerance(q, k, v, out, lse, score_err=0.0, v_err=0.0, p_err=0.0, seen_codes=0,
                    v_sq=None):
    """Six standard deviations of (out, lse) errors of rows q [rows, 128] over k, v [T, 128]
    when products of a score carry independent relative errors of at most score_err (each uniform:
    rms = bound / sqrt 3), values v_err and weights p_err, plus fp32 sums.  seen_codes: errors
    of one codebook entry are shared by every token that uses it, so averaging over tokens
    stops at about that many independent ones."""
    if len(k) == 0:
        return np.full(out.shape, 1e-30), np.full(lse.shape, 1e-30)
    v_sq = v ** 2 if v_sq is None else v_sq            # what v_err is relative to
    s = q @ k.T / np.sqrt(D)
    p = np.exp(s - lse[:, None])
    rms = np.sqrt((q ** 2) @ (k ** 2).T / D)                       # of a score's products
    ds2 = (score_err ** 2 / 3) * rms ** 2 + (2.0 ** -22) ** 2 * (1 + s ** 2)
    share = (1.0 / seen_codes if seen_codes else 0.0)
    w = p ** 2 + share * p                                         # weight of independent errors
    dev2 = np.einsum("rt,td->rd", w * (ds2 + p_err ** 2 / 3), v ** 2) \
        + (w * (ds2 + p_err ** 2 / 3)).sum(-1)[:, None] * out ** 2 \
        + np.einsum("rt,td->rd", w, v_sq) * (v_err ** 2 / 3)
    rms_v = np.sqrt(p @ v ** 2)
    tol_o = 6 * np.sqrt(dev2) + 2.0 ** -19 * rms_v
    # the sum of weights is kept in fp32; p_err does not enter it
    tol_l = 6 * np.sqrt((w * ds2).sum(-1)) + 2.0 ** -21 * (1 + np.abs(lse))
    return tol_o, tol_l


def check(out, lse, ref_out, ref_lse, tol_o, tol_l, half):
    """out / lse (numpy float64) within the tolerances plus the rounding of the output type."""
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse))
    fin = ~np.isneginf(ref_lse)
    assert np.all(out[~fin] == 0)
    eo = np.abs(out - ref_out)[fin] - half * np.abs(ref_out[fin]) - tol_o[fin]
    el = np.abs(lse[fin] - ref_lse[fin]) - tol_l[fin]
    assert np.all(eo <= 0), f"out off by {np.abs(out - ref_out)[fin].max():.3e}, {eo.max():.3e} over"
    assert np.all(el <= 0), f"lse off by {np.abs(lse[fin] - ref_lse[fin]).max():.3e}, {el.max():.3e} over"
