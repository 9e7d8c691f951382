"""Eviction from the paged KV cache: the attention weight that every cached key has received, the
choice of the rows to keep by it, and moving those together (C ABI: include/hstu_evict.h).

    hstu_kv_append(k, v, seq_offsets, kv_cache, weights=weights, **table)
    out, lse = hstu_softmax_fwd(q, kv_cache, seq_offsets, ..., return_lse=True, **table)
    hstu_kv_weights(q, lse, kv_cache, seq_offsets, weights, ..., **table)
    kept, shorter = hstu_kv_select(weights, budget=4096, recent=256, max_seqlen_k=Sk, **table)
    hstu_kv_compact(kv_cache, kept, weights=weights, **table)
    table = shorter

("RecOps Running Case Documentation", Inputs and Outputs table: kv_cache, page_offsets, page_ids,
last_page_len.) The work runs in libhstu_fwd.so; this module checks torch tensors and passes their
pointers to its C ABI on the current stream. Nothing is kept between calls.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _abi
from .kv_cache import _INDEX, _PACK_CACHE, _call, _cache, _row_dtype, _rows, _tensor

__all__ = ["hstu_kv_weights", "hstu_kv_select", "hstu_kv_compact"]

_PACK_WEIGHTS = struct.Struct("@PqPqiiiiifPPii").pack
_PACK_SELECT = struct.Struct("@iiiiqPPPqPiiiiPPPPP").pack
_PACK_COMPACT = struct.Struct("@PiiPPqi4x").pack
_MOST = 1 << 30  # of budget and max_seqlen_k


def _count(x, name, least, most=_MOST):
    x = int(x)
    if not least <= x <= most:
        raise ValueError(f"{name} must be in [{least}, {most}], got {x}")
    return x


def hstu_kv_weights(q, lse, kv_cache, seq_offsets, weights, *, max_seqlen, max_seqlen_k,
                    page_offsets, page_ids, last_page_len, causal=True, alpha=1.0, accumulate=True,
                    kv_scale=None, kv_group_scale=None, k_descale=None, v_descale=None,
                    status=None):
    """Add the attention weights that the cached keys receive from q; returns weights.

    weights [num_pages, Nk, page_size] fp32 gets, for every cached row of the sequences and kv head,
    sum exp(alpha q k - lse) over the queries that see it and their heads of the kv head: added to
    what it holds, or with accumulate=False in its place (0 where no query sees the row). lse
    [T, Nq] fp32 is hstu_softmax_fwd's of the same call; its other arguments are the same here. To
    weigh keys by the last tokens of a prompt alone, pass those tokens' q, lse and seq_offsets.
    Elements of weights that belong to no cached row are left as they are, with what earlier rows of
    their place have received: hstu_kv_append, given weights, sets those of new rows to 0. No page may
    belong to two sequences. Repeated calls give the same bits."""
    c = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale,
               kv_group_scale, k_descale, v_descale, status)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dtype = _row_dtype(c, q.dtype)
    q_stride = _rows(q, "q", c.device, q.dtype, None, c.D)
    T, Nq, _ = q.shape
    if Nq % c.Nk:
        raise ValueError(f"q's heads ({Nq}) must be a multiple of the cache's ({c.Nk})")
    dev = kv_cache.device
    lse_ptr = _tensor(lse, "lse", dev, torch.float32, (T, Nq))
    to = _tensor(weights, "weights", dev, torch.float32, (kv_cache.shape[0], c.Nk, c.sizes[4]))
    try:
        args = _PACK_WEIGHTS(q.data_ptr(), q_stride, seq_offsets.data_ptr(), T, dtype, Nq,
                             int(max_seqlen), int(max_seqlen_k), bool(causal), float(alpha),
                             lse_ptr, to, bool(accumulate), 0)
    except (struct.error, OverflowError):  # max_seqlen, max_seqlen_k or alpha that no C type holds
        raise _abi.HstuError(_abi.HSTU_ERR_INVALID_ARG, "hstu_kv_weights") from None
    _call("hstu_kv_weights", c, args)
    return weights


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(cache_sizes, budget, bound):
    """hstu_compact_workspace for these sizes (it reads no pointer)."""
    need = ctypes.c_longlong(0)
    _abi.check(_abi.lib().hstu_compact_workspace(
        _PACK_CACHE(*cache_sizes, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0, 0),
        _PACK_COMPACT(0, budget, bound, 0, 0, 0, 0), ctypes.byref(need)), "hstu_compact_workspace")
    return need.value


class _Table:
    """What _call needs of a call that has no cache."""
    __slots__ = ("packed", "device")


def _explain_select(weights, page_offsets, page_ids, last_page_len):
    """Raises for what is wrong with these tensors."""
    for t, name in ((weights, "weights"), (page_offsets, "page_offsets"), (page_ids, "page_ids"),
                    (last_page_len, "last_page_len")):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    dev, index = weights.device, page_offsets.dtype
    if dev.type != "cuda":
        raise ValueError("the KV cache operators run on CUDA tensors only")
    if weights.dim() != 3:
        raise ValueError(f"weights must be [num_pages, Nk, page_size], got {list(weights.shape)}")
    if index not in _INDEX:
        raise TypeError("index tensors must be int32 or int64")
    if page_offsets.dim() != 1 or page_offsets.shape[0] < 1 or page_ids.dim() != 1:
        raise ValueError("page_offsets must be [B + 1], page_ids one-dimensional")
    B = page_offsets.shape[0] - 1
    _tensor(weights, "weights", dev, torch.float32, weights.shape)
    _tensor(page_offsets, "page_offsets", dev, index, (B + 1,))
    _tensor(page_ids, "page_ids", dev, index, page_ids.shape)
    _tensor(last_page_len, "last_page_len", dev, index, (B,))


def hstu_kv_select(weights, *, budget, max_seqlen_k, page_offsets, page_ids, last_page_len,
                   recent=0, status=None):
    """Choose the rows of a cache to keep, by their attention weights.

    weights [num_pages, Nk, page_size] fp32 (hstu_kv_weights). Of every sequence and kv head,
    min(length, budget) rows are kept: the last `recent` and those of the largest weights among the
    others (of equal weights the earlier; a NaN counts as less than any). max_seqlen_k bounds the
    lengths. Returns kept [B, Nk, budget] int32, their positions in increasing order and -1 behind
    them, and the table of the shorter sequences, a dict of page_offsets, page_ids and last_page_len
    as they are once hstu_kv_compact has moved the rows: each sequence keeps its first pages, and
    entries of page_ids behind the last are -1. Pages that it no longer names are free."""
    try:  # one pass over what is usually right; _explain_select says what is not
        dev = weights.get_device()
        pages, Nk, page_size = weights.shape
        index = page_offsets.dtype
        B1, = page_offsets.shape
        ids, = page_ids.shape
        ok = (dev >= 0 and index in _INDEX and B1 > 0 and weights.dtype is torch.float32 and
              weights.is_contiguous() and last_page_len.shape == (B1 - 1,))
        for t in (page_offsets, page_ids, last_page_len):
            ok = ok and t.dtype is index and t.get_device() == dev and t.is_contiguous()
    except (AttributeError, ValueError, TypeError):
        ok = False
    if not ok:
        _explain_select(weights, page_offsets, page_ids, last_page_len)
        raise ValueError("weights and the page table do not fit together")
    B = B1 - 1
    budget, recent = _count(budget, "budget", 1), min(_count(recent, "recent", 0, 1 << 62), _MOST)
    bound = _count(max_seqlen_k, "max_seqlen_k", 1)
    status_ptr = 0 if status is None else _tensor(status, "status", weights.device, torch.int32,
                                                  (1,))
    kept = torch.empty((B, Nk, budget), dtype=torch.int32, device=weights.device)
    new = {"page_offsets": torch.empty_like(page_offsets), "page_ids": torch.empty_like(page_ids),
           "last_page_len": torch.empty_like(last_page_len)}
    if not B:  # nothing for the library to do
        new["page_offsets"].zero_()
        new["page_ids"].fill_(-1)
        return kept, new
    t = _Table()
    t.device = dev
    t.packed = _PACK_SELECT(B, Nk, page_size, index is torch.int64, pages, page_offsets.data_ptr(),
                            page_ids.data_ptr(), last_page_len.data_ptr(), ids, weights.data_ptr(),
                            budget, recent, bound, 0, kept.data_ptr(),
                            new["page_offsets"].data_ptr(), new["page_ids"].data_ptr(),
                            new["last_page_len"].data_ptr(), status_ptr)
    _call("hstu_kv_select", t)
    return kept, new


def hstu_kv_compact(kv_cache, kept, *, page_offsets, page_ids, last_page_len, max_seqlen_k=None,
                    weights=None, kv_scale=None, kv_group_scale=None, status=None):
    """Move the kept rows of a cache together, in place; returns kv_cache.

    kept [B, Nk, budget] int32 is hstu_kv_select's (or positions of the caller's own choice:
    increasing, -1 behind the last). Row r of every sequence and kv head becomes the K and V row at
    position kept[b, hk, r], with its scales and factors, and its entry of weights if that is given
    [num_pages, Nk, page_size]. The table is the one from before, of which max_seqlen_k may bound the
    lengths; the one that hstu_kv_select returned describes the result. Rows that are not written
    keep what they hold, entries of weights too (pass weights to the hstu_kv_append that fills them
    next); a cache with static factors (k_descale) keeps those. No page may belong to
    two sequences."""
    if not isinstance(page_offsets, torch.Tensor):
        raise TypeError("page_offsets must be a torch.Tensor")
    c = _cache(kv_cache, page_offsets, page_offsets, page_ids, last_page_len, kv_scale,
               kv_group_scale, None, None, status)
    dev = kv_cache.device
    if not isinstance(kept, torch.Tensor) or kept.dim() != 3:
        raise ValueError("kept must be a [B, Nk, budget] torch.Tensor")
    kept_ptr = _tensor(kept, "kept", dev, torch.int32, (c.B, c.Nk, kept.shape[2]))
    w = 0 if weights is None else _tensor(weights, "weights", dev, torch.float32,
                                          (kv_cache.shape[0], c.Nk, c.sizes[4]))
    bound = _MOST if max_seqlen_k is None else _count(max_seqlen_k, "max_seqlen_k", 1)
    if not c.B or not kept.shape[2]:
        return kv_cache
    need = _workspace_bytes(c.sizes, kept.shape[2], bound)
    workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    _call("hstu_kv_compact", c, _PACK_COMPACT(kept_ptr, kept.shape[2], bound, w,
                                              workspace.data_ptr(), need, 0))
    return kv_cache
