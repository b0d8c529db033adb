"""Measured cases of three serving operators: decode attention of a batch over one shared
compressed prefix, the rotating append to a 16-bit paged cache, and the decode attention over
those pages.

run() computes each of them in a plain form out of elementary torch operations, or, with
`own` true, through the package's public calls; exact() computes the definition in float64.
"""
import math

import numpy as np
import torch

own = False

D = 128
BASE = 500000.0
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def prefix(batch, hq, hkv, t_cap, length, rounds, dtype, group=8, bits=8, **more):
    return dict(kind="prefix", batch=batch, hq=hq, hkv=hkv, t_cap=t_cap, length=length,
                rounds=rounds, dtype=dtype, group=group, bits=bits, **more)


def append(batch, hq, hkv, page, tokens, pad, held, dtype, cache, fused, **more):
    return dict(kind="append", batch=batch, hq=hq, hkv=hkv, page=page, tokens=tokens, pad=pad,
                held=held, dtype=dtype, cache=cache, fused=fused, **more)


def paged(batch, hq, hkv, page, shortest, longest, dtype, cache, prev, **more):
    return dict(kind="paged", batch=batch, hq=hq, hkv=hkv, page=page, shortest=shortest,
                longest=longest, dtype=dtype, cache=cache, prev=prev, **more)


def listed():
    return [
        # a few requests behind a short system prompt, fp32 queries: latency counts
        prefix(4, 32, 8, 1024, 1000, 1, "fp32", name="prefix_B4_T1000_R1_fp32"),
        # the 32K layer's cache at 2 bits, read by 16 sequences at once
        prefix(16, 32, 8, 32768, 32768, 2, "bf16", name="prefix_B16_T32768_R2_bf16"),
        # the 128K layer's cache at 1 bit, read by 32 sequences: the largest
        prefix(32, 32, 8, 131072, 131072, 1, "bf16", name="prefix_B32_T131072_R1_bf16"),
        # odd sizes: 8 query heads per KV head, a prefix that ends inside its last tile
        prefix(7, 16, 2, 12352, 12345, 2, "fp16", name="prefix_B7_g8_T12345_R2_fp16"),
        # the paper's 1-bit layout: 64-scalar groups, 11 rounds, packed 6-bit codes
        prefix(16, 32, 8, 32768, 32768, 11, "bf16", 64, 6, name="prefix_B16_T32768_R11_g64"),
        # one decode step of 32 sequences: one new token each, behind a shared prefix
        append(32, 32, 8, 16, 32, 0, 500, "bf16", "bf16", False, name="append_decode_B32"),
        # a chunk of 4 prompts, taken as views of a fused q-k-v projection
        append(4, 32, 8, 64, 8192, 0, 0, "bf16", "bf16", True, name="append_prompt_8192"),
        # ragged continuation with rows behind the last sequence, fp32 into fp16 pages
        append(13, 28, 7, 16, 1531, 5, 777, "fp32", "fp16", False, name="append_ragged_1531"),
        # recent tokens only, folded into the state of a compressed prefix
        paged(32, 32, 8, 16, 1, 128, "bf16", "bf16", True, name="paged_window_B32_L128"),
        # the ragged batch: 16 sequences of 1024 to 8192 tokens
        paged(16, 32, 8, 16, 1024, 8192, "bf16", "bf16", False, name="paged_B16_L1024_8192"),
        # one long sequence
        paged(1, 32, 8, 64, 131071, 131071, "fp16", "fp16", False, name="paged_B1_L131071"),
        # a full server: 64 sequences of up to 16K, fp32 queries
        paged(64, 32, 8, 32, 8192, 16384, "fp32", "bf16", True, name="paged_B64_L16384_fp32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["prefix", "prefix", "append", "paged"])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 4, 4, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    cache = rng.choice(["bf16", "fp16"])
    page = rng.choice([8, 16, 32, 64, 128])
    if kind == "prefix":
        group = rng.choice([8, 8, 8, 64])
        length = _log(rng, 1, 131072)
        batch = _log(rng, 1, 64)
        # fp32 queries are served for small batches; nothing costs more than the largest case
        most = (16 * 32 * 32768 if dtype == "fp32" or group == 64 else 32 * 32 * 131072)
        if group == 64:
            g, rounds, bits = 4, rng.choice([1, 5, 11, 21]), rng.choice([6, 8])
            most = most * 11 // max(11, rounds)
        else:
            rounds, bits = rng.choice([1, 2]), 8
        length = max(1, min(length, most // (batch * g * hkv)))
        t_cap = -(-length // 64) * 64
        return prefix(batch, g * hkv, hkv, t_cap, length, rounds, dtype, group, bits)
    if kind == "append":
        batch = _log(rng, 1, 64)
        tokens = batch + _log(rng, 1, 16384) - 1
        return append(batch, g * hkv, hkv, page, tokens, rng.choice([0, 0, 3]), _log(rng, 1, 4096),
                      dtype, cache, rng.random() < 0.5)
    batch = _log(rng, 1, 64)
    longest = _log(rng, 1, min(131072, 64 * 16384 // batch))
    shortest = max(0, int(longest * rng.choice([0.0, 0.1, 0.5, 1.0])))
    return paged(batch, g * hkv, hkv, page, shortest, longest, dtype, cache, rng.random() < 0.5)


def _lengths(case):
    """Lengths of the sequences of an append or paged case: a function of the case alone."""
    r = np.random.RandomState(case["batch"] * 7919 + case.get("longest", case.get("tokens")))
    if case["kind"] == "paged":
        n = r.randint(case["shortest"], case["longest"] + 1, case["batch"])
        n[0] = case["longest"]
        return n
    # ragged shares of the tokens, at least one each
    cuts = np.sort(r.choice(case["tokens"] - 1, case["batch"] - 1, replace=False)) + 1
    return np.diff(np.concatenate([[0], cuts, [case["tokens"]]]))


def _held(case):
    """Tokens that each sequence of an append case holds before the call."""
    r = np.random.RandomState(case["tokens"] + 5)
    return r.randint(0, case["held"] + 1, case["batch"])


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32 if dtype != torch.float64 else dtype, device="cuda")
    return x.normal_(0.0, std, generator=g).to(dtype)


def _ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _table(case, lens, seed):
    """Page table of sequences that hold `lens` tokens: pages in shuffled order."""
    need = -(-np.asarray(lens) // case["page"])
    total = int(need.sum())
    order = np.random.RandomState(seed % (1 << 31)).permutation(total + 3)
    width = max(1, int(need.max()))
    table = np.zeros((len(need), width), np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return _ints(table), total + 3, width


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    if case["kind"] == "prefix":
        B, hq, hkv, T, R = (case[k] for k in ("batch", "hq", "hkv", "t_cap", "rounds"))
        std = 1.0 / math.sqrt(R)
        if case["group"] == 8:
            s["key_cb"] = _normal(g, (hkv, 16, R, 256, 4, 2), torch.float32, std)
            s["val_cb"] = _normal(g, (hkv, 16, R, 256, 8), torch.float32, std)
            codes, top = (1, hkv, T, R, 16), 256
        else:
            s["key_cb"] = _normal(g, (hkv, 2, R, 64, 32, 2), torch.float32, std)
            s["val_cb"] = _normal(g, (hkv, 2, R, 64, 64), torch.float32, std)
            # 6-bit codes are packed 4 to 3 bytes: any byte is a valid piece of a row
            codes = (1, hkv, 2, R, T * 3 // 4 if case["bits"] == 6 else T)
            top = 256 if case["bits"] == 6 else 64
        s["key_codes"] = torch.randint(top, codes, generator=g, device="cuda", dtype=torch.uint8)
        s["val_codes"] = torch.randint(top, codes, generator=g, device="cuda", dtype=torch.uint8)
        s["q"] = _normal(g, (B, hq, D), DT[case["dtype"]])
        s["length"] = _ints([case["length"]])
    elif case["kind"] == "append":
        B, hq, hkv, n = case["batch"], case["hq"], case["hkv"], case["tokens"] + case["pad"]
        new = _lengths(case)
        lens = new + _held(case)
        s["table"], pages, s["width"] = _table(case, lens, seed)
        s["k_pages"] = _normal(g, (pages, hkv, case["page"], D), DT[case["cache"]])
        s["v_pages"] = _normal(g, (pages, hkv, case["page"], D), DT[case["cache"]])
        s["lens"] = _ints(lens)
        s["offsets"] = _ints(np.concatenate([[0], np.cumsum(new)]))
        s["first"] = _ints(np.random.RandomState(case["tokens"]).randint(0, 131072, B))
        if case["fused"]:
            qkv = _normal(g, (n, hq + 2 * hkv, D), DT[case["dtype"]])
            s["q"], s["k"], s["v"] = qkv.split([hq, hkv, hkv], 1)
        else:
            s["q"], s["k"], s["v"] = (_normal(g, (n, h, D), DT[case["dtype"]])
                                      for h in (hq, hkv, hkv))
    else:
        B, hq, hkv = case["batch"], case["hq"], case["hkv"]
        lens = _lengths(case)
        s["table"], pages, s["width"] = _table(case, lens, seed)
        s["k_pages"] = _normal(g, (pages, hkv, case["page"], D), DT[case["cache"]])
        s["v_pages"] = _normal(g, (pages, hkv, case["page"], D), DT[case["cache"]])
        s["lens"] = _ints(lens)
        s["q"] = _normal(g, (B, hq, D), DT[case["dtype"]])
        s["prev"] = None
        if case["prev"]:
            s["prev"] = (_normal(g, (B, hq, D), torch.float32, 0.2),
                         _normal(g, (B, hq), torch.float32) + 6.0)
    return s


# ---------------------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------------------
def _rotate(x, pos):
    """RoPE of x [..., n, 128] (interleaved pairs) at positions pos [n]; angles in 64 bits."""
    theta = BASE ** (-torch.arange(0, D, 2, device=x.device, dtype=torch.float64) / D)
    ang = pos.double()[:, None] * theta
    c, sn = ang.cos().float(), ang.sin().float()
    re, im = x[..., 0::2], x[..., 1::2]
    return torch.stack((re * c - im * sn, re * sn + im * c), -1).flatten(-2)


def _codes(codes, case):
    """Codes as [Hkv, T, R, groups] whole numbers."""
    if case["group"] == 8:
        return codes[0].long()
    c = codes[0].int()
    if case["bits"] == 6:
        w = c.unflatten(-1, (-1, 3))
        w = w[..., 0] | (w[..., 1] << 8) | (w[..., 2] << 16)
        c = torch.stack([(w >> sh) & 63 for sh in (0, 6, 12, 18)], -1).flatten(-2)
    return (c & 63).permute(0, 3, 2, 1).long()


def _decode(codes, cb):
    """Sum over rounds of cb [Hkv, groups, R, entries, dims] at codes [Hkv, T, R, groups]."""
    h = torch.arange(cb.shape[0], device=cb.device)[:, None, None]
    G = torch.arange(cb.shape[1], device=cb.device)
    return sum(cb[h, G, r, codes[:, :, r]] for r in range(cb.shape[2])).flatten(-2)


def _softmax(s, seen, v):
    """(softmax(s) @ v, ln sum exp s) over the last axis where `seen`; nothing seen: 0, -inf."""
    s = s.masked_fill(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = (s - m.masked_fill(m == -math.inf, 0.0)).exp()
    z = p.sum(-1, keepdim=True)
    return (p @ v) / z.masked_fill(z == 0, 1.0), (z.log() + m)[..., 0]


def _prefix_plain(s):
    case, q = s["case"], s["q"]
    B, hkv, T = case["batch"], case["hkv"], case["t_cap"]
    t = torch.arange(T, device=q.device)
    k = _rotate(_decode(_codes(s["key_codes"], case), s["key_cb"].flatten(-2)), t)
    v = _decode(_codes(s["val_codes"], case), s["val_cb"])
    qh = q.float().view(B, hkv, -1, D).transpose(0, 1).flatten(1, 2)
    o, lse = _softmax(qh @ k.transpose(-1, -2) * D ** -0.5, t < s["length"], v)
    o = o.view(hkv, B, -1, D).transpose(0, 1).reshape(B, -1, D)
    return o.to(q.dtype), lse.view(hkv, B, -1).transpose(0, 1).reshape(B, -1)


def _append_plain(s):
    n, page = s["k"].shape[0], s["case"]["page"]
    i = torch.arange(n, device=s["k"].device)
    b = torch.searchsorted(s["offsets"].long(), i, right=True) - 1
    live = b < s["case"]["batch"]
    b = b.clamp(max=s["case"]["batch"] - 1)
    local = s["lens"].long()[b] - s["offsets"].long()[b + 1] + i
    pos = local + s["first"].long()[b]
    at, row = s["table"].long()[b, (local // page).clamp(max=s["width"] - 1)][live], (local % page)[live]
    k = _rotate(s["k"].float().transpose(0, 1), pos).transpose(0, 1)
    s["k_pages"][at, :, row] = k[live].to(s["k_pages"].dtype)
    s["v_pages"][at, :, row] = s["v"][live].float().to(s["v_pages"].dtype)
    q = _rotate(s["q"].float().transpose(0, 1), pos).transpose(0, 1).to(s["q"].dtype)
    return q[:s["case"]["tokens"]], s["k_pages"], s["v_pages"]


def _paged_plain(s):
    case, q = s["case"], s["q"]
    B, hkv = case["batch"], case["hkv"]
    k, v = (x[s["table"].long()].transpose(1, 2).flatten(2, 3).float()
            for x in (s["k_pages"], s["v_pages"]))
    seen = torch.arange(k.shape[2], device=q.device) < s["lens"][:, None, None, None]
    o, lse = _softmax(q.float().view(B, hkv, -1, D) @ k.transpose(-1, -2) * D ** -0.5, seen, v)
    o, lse = o.reshape(B, -1, D), lse.reshape(B, -1)
    if s["prev"] is not None:
        m = torch.maximum(lse, s["prev"][1])
        a, p = (lse - m).exp(), (s["prev"][1] - m).exp()
        o = (a[..., None] * o + p[..., None] * s["prev"][0]) / (a + p)[..., None]
        lse = m + (a + p).log()
    return o.to(q.dtype), lse


# ---------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------
def _own(s):
    import compressed_attention_cvq_b200 as cvq

    case = s["case"]
    if case["kind"] == "prefix":
        if "plan" not in s:
            shape = cvq.shape_of(s["q"], s["key_codes"], BASE, case["group"], case["bits"])
            n = cvq.prefix_suggest_splits(shape, s["q"].dtype)
            s["plan"] = shape, n, cvq.prefix_workspace_alloc(shape, n, s["q"].device)
        shape, n, ws = s["plan"]
        return cvq.prefix_attend(shape, s["q"], s["key_cb"], s["key_codes"], s["val_codes"],
                                 s["length"], s["val_cb"], n, workspace=ws,
                                 out_dtype=s["q"].dtype)
    if "plan" not in s:
        s["plan"] = cvq.make_paged(case["batch"], case["hq"], case["hkv"], case["page"],
                                   s["k_pages"].shape[0], s["width"], s["k_pages"].dtype, BASE)
    paged_shape = s["plan"]
    if case["kind"] == "append":
        q = cvq.paged_append(paged_shape, s["k"], s["v"], s["offsets"], s["lens"], s["table"],
                             s["k_pages"], s["v_pages"], q=s["q"], pos_offsets=s["first"])
        return q[:case["tokens"]], s["k_pages"], s["v_pages"]
    if "splits" not in s:
        s["splits"] = cvq.paged_suggest_splits(paged_shape)
        s["ws"] = cvq.paged_workspace_alloc(paged_shape, s["splits"], s["q"].device)
    return cvq.paged_attend(paged_shape, s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"],
                            s["splits"], workspace=s["ws"], prev=s["prev"], out_dtype=s["q"].dtype)


def run(state):
    if own:
        return _own(state)
    return {"prefix": _prefix_plain, "append": _append_plain,
            "paged": _paged_plain}[state["case"]["kind"]](state)


# ---------------------------------------------------------------------------------------
# the work a pass cannot do without
# ---------------------------------------------------------------------------------------
def work(case):
    B, hq, hkv = case["batch"], case["hq"], case["hkv"]
    io = SIZE[case["dtype"]]
    if case["kind"] == "prefix":
        T, R = case["length"], case["rounds"]
        if case["group"] == 8:
            codes, books = 2 * 16 * R * T * hkv, 2 * 16 * R * 256 * 8 * 4 * hkv
        else:
            codes = 2 * 2 * R * T * hkv * case["bits"] // 8
            books = 2 * 2 * R * 64 * 64 * 4 * hkv
        return {"bytes": codes + books + B * hq * (2 * D * io + 4), "flops": 4 * D * B * hq * T}
    kv = SIZE[case["cache"]]
    if case["kind"] == "append":
        n = case["tokens"]
        return {"bytes": n * D * (2 * hq * io + 2 * hkv * (io + kv)),
                "flops": 6 * n * (hq + hkv) * D // 2}
    total = int(_lengths(case).sum())
    prev = B * hq * (4 * D + 4) if case["prev"] else 0
    return {"bytes": 2 * total * hkv * D * kv + B * hq * (2 * D * io + 4) + prev,
            "flops": 4 * D * hq * total}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _exact_turn(z, pos):
    """z (complex128 [..., 64]) times e^{i theta_j pos}."""
    j = torch.arange(64, device=z.device, dtype=torch.float64)
    ang = pos.to(torch.float64).unsqueeze(-1) * torch.exp(-2.0 * j / D * math.log(BASE))
    return z * torch.polar(torch.ones_like(ang), ang)


def _exact_attention(q, k, v):
    """One KV head: q [rows, 128], k and v [T, 128] in float64 -> (out, lse)."""
    if k.shape[0] == 0:
        return torch.zeros_like(q), torch.full_like(q[:, 0], -math.inf)
    s = torch.einsum("rd,td->rt", q, k) / math.sqrt(D)
    lse = torch.logsumexp(s, -1)
    return torch.einsum("rt,td->rd", torch.exp(s - lse[:, None]), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    q = s["q"].double()
    if case["kind"] == "append":
        n, page = case["tokens"], case["page"]
        new, held = _lengths(case), _held(case)
        table, first = s["table"].cpu().numpy(), s["first"].cpu().numpy()
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        local = np.concatenate([h + np.arange(m) for h, m in zip(held, new)])
        seq = np.repeat(np.arange(case["batch"]), new)
        pos = torch.from_numpy(local + first[seq]).cuda()[:, None]
        at = torch.from_numpy(table[seq, local // page]).long().cuda()
        row = torch.from_numpy(local % page).cuda()
        turned = [torch.view_as_real(_exact_turn(torch.view_as_complex(
            x[:n].double().reshape(n, -1, 64, 2)), pos)).reshape(n, -1, D) for x in (s["q"], s["k"])]
        kp[at, :, row] = turned[1]
        vp[at, :, row] = s["v"][:n].double()
        return turned[0], kp, vp
    out, lse = torch.empty_like(q), torch.empty_like(q[..., 0])
    g = case["hq"] // case["hkv"]
    if case["kind"] == "prefix":
        L, R = case["length"], case["rounds"]
        for h in range(case["hkv"]):
            cols = [[], []]
            for i, (codes, cb) in enumerate((("key_codes", "key_cb"), ("val_codes", "val_cb"))):
                c, book = s[codes][0, h], s[cb][h].double().flatten(3)
                if case["group"] == 64:
                    if case["bits"] == 6:
                        bit = torch.arange(6 * case["t_cap"], device=c.device)
                        one = (c[..., bit // 8].int() >> (bit % 8)) & 1
                        c = (one.unflatten(-1, (-1, 6)) << torch.arange(6, device=c.device)).sum(-1)
                    c = c.permute(2, 1, 0)
                for G in range(book.shape[0]):
                    part = torch.zeros(L, book.shape[-1], dtype=torch.float64, device=q.device)
                    for r in range(R):
                        part += book[G, r].index_select(0, c[:L, r, G].int())
                    cols[i].append(part)
            k = torch.view_as_complex(torch.cat(cols[0], -1).reshape(L, 64, 2))
            k = torch.view_as_real(_exact_turn(k, torch.arange(L, device=q.device))).reshape(L, D)
            o, z = _exact_attention(q[:, h * g:(h + 1) * g].reshape(-1, D), k, torch.cat(cols[1], -1))
            out[:, h * g:(h + 1) * g] = o.view(-1, g, D)
            lse[:, h * g:(h + 1) * g] = z.view(-1, g)
        return out, lse
    for b, L in enumerate(_lengths(case).tolist()):
        used = s["table"][b, :-(-L // case["page"])].long()
        k, v = (x[used].double().transpose(0, 1).flatten(1, 2)[:, :L] for x in (s["k_pages"], s["v_pages"]))
        for h in range(case["hkv"]):
            sl = slice(h * g, (h + 1) * g)
            out[b, sl], lse[b, sl] = _exact_attention(q[b, sl], k[h], v[h])
    if s["prev"] is not None:
        both = torch.stack((lse, s["prev"][1].double()))
        total = torch.logsumexp(both, 0)
        w = torch.exp(both - total)
        out = w[0, ..., None] * out + w[1, ..., None] * s["prev"][0].double()
        lse = total
    return out, lse
