"""Binding of the serving calls: attention of a batch over one shared compressed prefix, the
16-bit paged cache and the attention over it (cvq_prefix_attend, cvq_paged_append,
cvq_paged_attend).

One decode step of a batch behind a shared prefix:

    qr = paged_append(paged, k, v, tok_offsets, seq_lens, page_table, k_pages, v_pages,
                      q=q, pos_offsets=prefix_lens)
    prev = prefix_attend(shape, qr, key_cb, key_codes, val_codes, prefix_len, val_cb, n,
                         workspace=ws, out_dtype=torch.float32)
    out, lse = paged_attend(paged, qr, k_pages, v_pages, page_table, seq_lens, n_paged,
                            workspace=ws_paged, prev=prev)

Tensors are checked against the shapes that the library is told (it gets plain pointers);
work is enqueued on the current CUDA stream of the tensors' device.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _binding as _b

_DTYPE = {torch.float32: _b.CVQ_F32, torch.bfloat16: _b.CVQ_BF16, torch.float16: _b.CVQ_F16}


def _dtype(dt, name):
    try:
        return _DTYPE[dt]
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {dt}") from None


def _check(t, name, dev, dtype, shape):
    """A dense tensor of this device, type and shape."""
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _cuda(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.device


def _on(dev):
    """The library launches on the current device: make it the tensors' own."""
    return (contextlib.nullcontext() if torch.cuda.current_device() == dev.index
            else torch.cuda.device(dev))


def _stream(stream, dev):
    return (stream if stream is not None else torch.cuda.current_stream(dev)).cuda_stream


def _sm_count(sm_count):
    if sm_count is not None:
        return sm_count
    return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count


def _workspace(ws, need, dev, what):
    if need == 0:
        raise ValueError(f"invalid shape or n_splits for {what}")
    if ws is None:
        return torch.zeros(need, dtype=torch.uint8, device=dev)
    if ws.device != dev or ws.numel() * ws.element_size() < need or not ws.is_contiguous():
        raise ValueError(f"workspace must be {need} dense bytes on {dev}")
    return ws


def _outputs(out, lse, out_dtype, default, B, Hq, dev):
    if out is None:
        out = torch.empty((B, Hq, 128), dtype=out_dtype or default, device=dev)
    elif out_dtype is not None and out.dtype != out_dtype:
        raise ValueError(f"out has dtype {out.dtype}, expected {out_dtype}")
    if lse is None:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=dev)
    _check(out, "out", dev, out.dtype, (B, Hq, 128))
    _check(lse, "lse", dev, torch.float32, (B, Hq))
    return out, lse


# --- the shared prefix -----------------------------------------------------------------
def prefix_suggest_splits(shape, q_dtype=torch.bfloat16, sm_count=None):
    return _b.lib.cvq_prefix_suggest_splits(ctypes.byref(shape), _dtype(q_dtype, "q"),
                                            _sm_count(sm_count))


def prefix_workspace_alloc(shape, n_splits, device):
    return _workspace(None, _b.lib.cvq_prefix_workspace_bytes(ctypes.byref(shape), n_splits),
                      torch.device(device), "cvq_prefix_workspace_bytes")


def _codebook(cb, name, dev, shape, key):
    """Check a codebook [(Hkv,) groups, R, entries, ...] and give its head stride."""
    one = ((2, shape.R, 64) if shape.group_dim == 64 else (16, shape.R, 256))
    d = 64 if shape.group_dim == 64 else 8
    one += (d // 2, 2) if key else (d,)
    per_head = cb.dim() == len(one) + 1
    _check(cb, name, dev, torch.float32, ((shape.n_kv_heads,) if per_head else ()) + one)
    return cb.numel() // shape.n_kv_heads if per_head else 0


def prefix_attend(shape, q, key_cb, key_codes, val_codes, prefix_len, val_cb, n_splits=None,
                  workspace=None, out=None, lse=None, out_dtype=None, stream=None):
    """Attention of shape.batch query tokens q [B, Hq, 128] (fp32, bf16 or fp16, rotated)
    over ONE code cache key_codes / val_codes [(1,) Hkv, t_cap, R, 16] (64-scalar groups:
    planar [(1,) Hkv, 2, R, t_cap], packed 3 t_cap / 4) of prefix_len [1] int32 tokens.
    Returns (out [B, Hq, 128] of out_dtype, default q's type, and lse [B, Hq] fp32)."""
    dev = _cuda(q, "q")
    B, Hq, Hkv = shape.batch, shape.n_q_heads, shape.n_kv_heads
    _check(q, "q", dev, q.dtype, (B, Hq, 128))
    if shape.group_dim == 64:
        codes = (Hkv, 2, shape.R, shape.t_cap * 3 // 4 if shape.code_bits == 6 else shape.t_cap)
    else:
        codes = (Hkv, shape.t_cap, shape.R, 16)
    for t, name in ((key_codes, "key_codes"), (val_codes, "val_codes")):
        _check(t, name, dev, torch.uint8, ((1,) if t.dim() == len(codes) + 1 else ()) + codes)
    _check(prefix_len, "prefix_len", dev, torch.int32, (1,))
    kstride = _codebook(key_cb, "key_cb", dev, shape, True)
    vstride = _codebook(val_cb, "val_cb", dev, shape, False)
    with _on(dev):
        if n_splits is None:
            n_splits = prefix_suggest_splits(shape, q.dtype)
        workspace = _workspace(workspace, _b.lib.cvq_prefix_workspace_bytes(
            ctypes.byref(shape), n_splits), dev, "cvq_prefix_workspace_bytes")
        out, lse = _outputs(out, lse, out_dtype, q.dtype, B, Hq, dev)
        st = _b.lib.cvq_prefix_attend(
            ctypes.byref(shape), q.data_ptr(), _dtype(q.dtype, "q"), key_cb.data_ptr(), kstride,
            key_codes.data_ptr(), val_codes.data_ptr(), prefix_len.data_ptr(), val_cb.data_ptr(),
            vstride, n_splits, workspace.data_ptr(), out.data_ptr(), _dtype(out.dtype, "out"),
            lse.data_ptr(), _stream(stream, dev))
    _b.check(st, "cvq_prefix_attend")
    return out, lse


# --- the paged cache -------------------------------------------------------------------
def make_paged(batch, n_q_heads, n_kv_heads, page_size, n_pages, max_pages,
               dtype=torch.bfloat16, rope_base=500000.0, page_stride=0, head_dim=128):
    """cvq_paged: a pool of n_pages pages [Hkv, page_size, 128] of `dtype` for keys and one
    for values, and page tables of max_pages entries per sequence."""
    return _b.cvq_paged(batch, n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages,
                        _dtype(dtype, "pages"), rope_base, page_stride)


def paged_suggest_splits(paged, sm_count=None):
    return _b.lib.cvq_paged_suggest_splits(ctypes.byref(paged), _sm_count(sm_count))


def paged_workspace_alloc(paged, n_splits, device):
    """Zeroed workspace for paged_attend (every call leaves it ready for the next)."""
    return _workspace(None, _b.lib.cvq_paged_workspace_bytes(ctypes.byref(paged), n_splits),
                      torch.device(device), "cvq_paged_workspace_bytes")


def _pages(paged, k_pages, v_pages, page_table, seq_lens, dev):
    shape = (paged.n_pages, paged.n_kv_heads, paged.page_size, 128)
    dense = paged.n_kv_heads * paged.page_size * 128
    strides = (paged.page_stride or dense, paged.page_size * 128, 128, 1)
    for t, name in ((k_pages, "k_pages"), (v_pages, "v_pages")):
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
        if _DTYPE.get(t.dtype) != paged.kv_dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, not the cache's")
        if tuple(t.shape) != shape or any(n > 1 and x != y for n, x, y in
                                          zip(shape, t.stride(), strides)):
            raise ValueError(f"{name} must be {shape} with strides {strides}, got "
                             f"{tuple(t.shape)} with {t.stride()}")
    _check(page_table, "page_table", dev, torch.int32, (paged.batch, paged.max_pages))
    _check(seq_lens, "seq_lens", dev, torch.int32, (paged.batch,))


def _tokens(t, name, dev, dtype, n, heads):
    """Token stride of [n, heads, 128] whose heads are dense (tokens may be strided)."""
    if t.device != dev or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} on {dev}")
    if tuple(t.shape) != (n, heads, 128) or t.stride(2) != 1 or (heads > 1 and t.stride(1) != 128):
        raise ValueError(f"{name} must be [{n}, {heads}, 128] with dense heads")
    return t.stride(0) if n > 1 else max(t.stride(0), heads * 128)


def paged_append(paged, k, v, tok_offsets, seq_lens, page_table, k_pages, v_pages, q=None,
                 q_out=None, pos_offsets=None, stream=None):
    """Write k, v [n, Hkv, 128] (keys rotated) into the pages at the end of their sequences,
    whose lengths seq_lens [B] already count them; token i belongs to sequence b for
    tok_offsets[b] <= i < tok_offsets[b+1].  Its RoPE position is pos_offsets[b] (or 0) plus
    its index in the sequence.  q [n, Hq, 128], if given, is rotated into q_out (returned)."""
    dev = _cuda(k, "k")
    n = k.shape[0]
    _pages(paged, k_pages, v_pages, page_table, seq_lens, dev)
    ks = _tokens(k, "k", dev, k.dtype, n, paged.n_kv_heads)
    vs = _tokens(v, "v", dev, k.dtype, n, paged.n_kv_heads)
    _check(tok_offsets, "tok_offsets", dev, torch.int32, (paged.batch + 1,))
    if pos_offsets is not None:
        _check(pos_offsets, "pos_offsets", dev, torch.int32, (paged.batch,))
    qs = 0
    if q is not None:
        qs = _tokens(q, "q", dev, k.dtype, n, paged.n_q_heads)
        if q_out is None:
            q_out = torch.empty((n, paged.n_q_heads, 128), dtype=q.dtype, device=dev)
        _check(q_out, "q_out", dev, q.dtype, (n, paged.n_q_heads, 128))
    elif q_out is not None:
        raise ValueError("q_out without q")
    if n == 0:
        return q_out
    with _on(dev):
        st = _b.lib.cvq_paged_append(
            ctypes.byref(paged), n, None if q is None else q.data_ptr(), qs, k.data_ptr(), ks,
            v.data_ptr(), vs, _dtype(k.dtype, "k"), tok_offsets.data_ptr(), seq_lens.data_ptr(),
            None if pos_offsets is None else pos_offsets.data_ptr(), page_table.data_ptr(),
            k_pages.data_ptr(), v_pages.data_ptr(), None if q is None else q_out.data_ptr(),
            _stream(stream, dev))
    _b.check(st, "cvq_paged_append")
    return q_out


def paged_attend(paged, q, k_pages, v_pages, page_table, seq_lens, n_splits=None, workspace=None,
                 prev=None, out=None, lse=None, out_dtype=None, stream=None):
    """Attention of one query token per sequence, q [B, Hq, 128] (rotated), over the pages of
    its seq_lens[b] tokens; prev = (out, lse) in fp32 of an earlier part of the sequences
    (prefix_attend, attend_fused) is merged in.  Returns (out, lse) as prefix_attend."""
    dev = _cuda(q, "q")
    B, Hq = paged.batch, paged.n_q_heads
    _check(q, "q", dev, q.dtype, (B, Hq, 128))
    _pages(paged, k_pages, v_pages, page_table, seq_lens, dev)
    po = pl = None
    if prev is not None:
        _check(prev[0], "prev out", dev, torch.float32, (B, Hq, 128))
        _check(prev[1], "prev lse", dev, torch.float32, (B, Hq))
        po, pl = prev[0].data_ptr(), prev[1].data_ptr()
    with _on(dev):
        if n_splits is None:
            n_splits = paged_suggest_splits(paged)
        workspace = _workspace(workspace, _b.lib.cvq_paged_workspace_bytes(
            ctypes.byref(paged), n_splits), dev, "cvq_paged_workspace_bytes")
        out, lse = _outputs(out, lse, out_dtype, q.dtype, B, Hq, dev)
        st = _b.lib.cvq_paged_attend(
            ctypes.byref(paged), q.data_ptr(), _dtype(q.dtype, "q"), k_pages.data_ptr(),
            v_pages.data_ptr(), page_table.data_ptr(), seq_lens.data_ptr(), n_splits,
            workspace.data_ptr(), po, pl, out.data_ptr(), _dtype(out.dtype, "out"),
            lse.data_ptr(), _stream(stream, dev))
    _b.check(st, "cvq_paged_attend")
    return out, lse
