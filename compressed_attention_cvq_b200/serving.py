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

Tensors are checked against the shapes that the library is told (it gets plain pointers), in
native code (csrc/serving_module.cpp): wrong devices, types, shapes and strides are ValueErrors.
Work is enqueued on the current CUDA stream of the tensors' device, or on `stream`: then as if it
were the current one, so that outputs and workspaces which the call allocates are that stream's too.
"""
from __future__ import annotations

import ctypes
from ctypes import addressof

import torch

from . import _binding as _b

_DTYPE = {torch.float32: _b.CVQ_F32, torch.bfloat16: _b.CVQ_BF16, torch.float16: _b.CVQ_F16}


class _Native:
    """The module _serving, bound to the loaded library on first use."""

    def __getattr__(self, name):
        try:
            from . import _serving
        except ImportError as e:
            raise ImportError(f"_serving.so is not built or does not load ({e}); run "
                              "`python -m compressed_attention_cvq_b200.build`") from e
        fns = ("cvq_prefix_workspace_bytes", "cvq_prefix_suggest_splits", "cvq_prefix_attend",
               "cvq_paged_append", "cvq_paged_workspace_bytes", "cvq_paged_suggest_splits",
               "cvq_paged_attend")
        _serving.bind(_b.check, *(ctypes.cast(getattr(_b.lib, f), ctypes.c_void_p).value
                                  for f in fns))
        for f in ("prefix_attend", "paged_append", "paged_attend"):
            setattr(self, f, getattr(_serving, f))      # later lookups skip __getattr__
        return getattr(_serving, name)


_native = _Native()


def _dtype(dt, name):
    try:
        return _DTYPE[dt]
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {dt}") from None


def _sm_count(sm_count):
    if sm_count is not None:
        return sm_count
    return torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count


def _workspace(need, dev, what):
    if need == 0:
        raise ValueError(f"invalid shape or n_splits for {what}")
    return torch.zeros(need, dtype=torch.uint8, device=dev)


def _at(struct, kind):
    """Address of a shape, whose type the native side cannot see."""
    if not isinstance(struct, kind):
        raise TypeError(f"expected a {kind.__name__}, got {type(struct).__name__}")
    return addressof(struct)


def _raw(stream):
    return None if stream is None else stream.cuda_stream


# --- the shared prefix -----------------------------------------------------------------
def prefix_suggest_splits(shape, q_dtype=torch.bfloat16, sm_count=None):
    return _b.lib.cvq_prefix_suggest_splits(ctypes.byref(shape), _dtype(q_dtype, "q"),
                                            _sm_count(sm_count))


def prefix_workspace_alloc(shape, n_splits, device):
    return _workspace(_b.lib.cvq_prefix_workspace_bytes(ctypes.byref(shape), n_splits), device,
                      "cvq_prefix_workspace_bytes")


def prefix_attend(shape, q, key_cb, key_codes, val_codes, prefix_len, val_cb, n_splits=None,
                  workspace=None, out=None, lse=None, out_dtype=None, stream=None):
    """Attention of shape.batch query tokens q [B, Hq, 128] (fp32, bf16 or fp16, rotated)
    over ONE code cache key_codes / val_codes [(1,) Hkv, t_cap, R, 16] (64-scalar groups:
    planar [(1,) Hkv, 2, R, t_cap], packed 3 t_cap / 4) of prefix_len [1] int32 tokens.
    Returns (out [B, Hq, 128] of out_dtype, default q's type, and lse [B, Hq] fp32)."""
    return _native.prefix_attend(_at(shape, _b.cvq_shape), q, key_cb, key_codes, val_codes, prefix_len,
                                 val_cb, n_splits, workspace, out, lse, out_dtype, _raw(stream))


# --- the paged cache -------------------------------------------------------------------
def make_paged(batch, n_q_heads, n_kv_heads, page_size, n_pages, max_pages,
               dtype=torch.bfloat16, rope_base=500000.0, page_stride=0, head_dim=128):
    """cvq_paged: a pool of n_pages pages [Hkv, page_size, 128] of `dtype` for keys and one
    for values, and page tables of max_pages entries per sequence."""
    return _b.cvq_paged(batch, n_q_heads, n_kv_heads, head_dim, page_size, n_pages, max_pages,
                        _dtype(dtype, "pages"), rope_base, page_stride)


def paged_suggest_splits(paged, sm_count=None):
    """A split count for sequences of like lengths; a batch with one sequence far longer than the
    others wants that of the one alone (batch 1)."""
    return _b.lib.cvq_paged_suggest_splits(ctypes.byref(paged), _sm_count(sm_count))


def paged_workspace_alloc(paged, n_splits, device):
    """Zeroed workspace for paged_attend.  Every call leaves it ready for the next, of any shape
    and split count that it has room for; prefix_attend may use it in between."""
    return _workspace(_b.lib.cvq_paged_workspace_bytes(ctypes.byref(paged), n_splits), device,
                      "cvq_paged_workspace_bytes")


def paged_append(paged, k, v, tok_offsets, seq_lens, page_table, k_pages, v_pages, q=None,
                 q_out=None, pos_offsets=None, stream=None):
    """Write k, v [n, Hkv, 128] (keys rotated) into the pages at the end of their sequences,
    whose lengths seq_lens [B] already count them; token i belongs to sequence b for
    tok_offsets[b] <= i < tok_offsets[b+1].  Its RoPE position is pos_offsets[b] (or 0) plus
    its index in the sequence.  q [n, Hq, 128], if given, is rotated into q_out (returned)."""
    return _native.paged_append(_at(paged, _b.cvq_paged), k, v, tok_offsets, seq_lens, page_table,
                                k_pages, v_pages, q, q_out, pos_offsets, _raw(stream))


def paged_attend(paged, q, k_pages, v_pages, page_table, seq_lens, n_splits=None, workspace=None,
                 prev=None, out=None, lse=None, out_dtype=None, stream=None):
    """Attention of one query token per sequence, q [B, Hq, 128] (rotated), over the pages of
    its seq_lens[b] tokens; prev = (out, lse) in fp32 of an earlier part of the sequences
    (prefix_attend, attend_fused) is merged in.  Returns (out, lse) as prefix_attend."""
    prev_out, prev_lse = (None, None) if prev is None else prev
    return _native.paged_attend(_at(paged, _b.cvq_paged), q, k_pages, v_pages, page_table, seq_lens,
                                n_splits, workspace, prev_out, prev_lse, out, lse, out_dtype,
                                _raw(stream))
