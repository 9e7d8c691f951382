"""Paged KV cache operators: writing new rows into the cache that hstu_fwd reads, reading
rows back, and softmax attention over it (C ABI: include/hstu_kv.h).

    hstu_kv_append(k, v, seq_offsets, kv_cache, page_offsets=po, page_ids=ids,
                   last_page_len=last, kv_scale=scale)
    out = hstu_softmax_fwd(q, kv_cache, seq_offsets, max_seqlen=Sq, max_seqlen_k=Sk,
                           page_offsets=po, page_ids=ids, last_page_len=last, kv_scale=scale)

("RecOps Running Case Documentation", Inputs and Outputs table: kv_cache, page_offsets,
page_ids, last_page_len; feature table, "Page" and "FP8 quantization types".) The work runs in
libhstu_fwd.so; this module checks torch tensors and passes their pointers to its C ABI on
the current stream. Nothing is kept between calls: workspaces come from torch's allocator.
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _abi

__all__ = ["hstu_kv_append", "hstu_kv_read", "hstu_softmax_fwd"]

_ROWS = {torch.float32: _abi.HSTU_F32, torch.float16: _abi.HSTU_F16, torch.bfloat16: _abi.HSTU_BF16}
_CACHE = {**_ROWS, torch.float8_e4m3fn: _abi.HSTU_FP8_E4M3}
_INDEX = (torch.int32, torch.int64)
_FP8 = torch.float8_e4m3fn

# The C structs as bytes (their layouts are those of the ctypes mirrors in _abi): one pack is
# a fraction of the cost of setting their fields.
_PACK_CACHE = struct.Struct("@8iPPqPPPqPPP").pack
_PACK_ROWS = struct.Struct("@PPqqPqii").pack
_PACK_ATTN = struct.Struct("@PqPqiiiiifPPPqi4x").pack


def _tensor(t, name, dev, dtype, shape):
    """A contiguous tensor of this device, type and shape."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, name, dev, dtype, heads, head_dim):
    """Elements between the rows of t [T, heads, head_dim], whose rows are contiguous (heads
    None: any number)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 3 or shape[2] != head_dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [T, {'N' if heads is None else heads}, {head_dim}], "
                         f"got {list(shape)}")
    width = shape[1] * head_dim
    if t.is_contiguous():
        return width
    row, head, last = t.stride()
    if last != 1 or (head != head_dim and shape[1] > 1) or (row < width and shape[0] > 1):
        raise ValueError(f"the rows of {name} must be contiguous and may not overlap, "
                         f"got strides {list(t.stride())}")
    return row if shape[0] > 1 else width


def _factors(k_descale, v_descale, dev, B, Nk):
    """Granularity and fp32 device tensors of the static E4M3 factors."""
    if k_descale is None and v_descale is None:
        return _abi.HSTU_DESCALE_CAST, None, None
    if k_descale is None or v_descale is None:
        raise ValueError("k_descale and v_descale go together")
    ts = [x if isinstance(x, torch.Tensor) else
          torch.full((1,), float(x), dtype=torch.float32, device=dev)
          for x in (k_descale, v_descale)]
    if ts[0].shape != ts[1].shape:
        raise ValueError("k_descale and v_descale must have one shape")
    shape = tuple(ts[0].shape)
    for name, t in zip(("k_descale", "v_descale"), ts):
        _tensor(t, name, dev, torch.float32, t.shape)
    if shape in ((), (1,)):
        return _abi.HSTU_DESCALE_TENSOR, *ts
    if shape == (B,):
        return _abi.HSTU_DESCALE_BATCH, *ts
    if shape == (B, Nk):
        return _abi.HSTU_DESCALE_HEAD, *ts
    raise ValueError(f"k_descale and v_descale must be one factor, [{B}] or [{B}, {Nk}], "
                     f"got {list(shape)}")


def _explain_cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale):
    """Raises for what is wrong with these tensors."""
    if not isinstance(kv_cache, torch.Tensor):
        raise TypeError("kv_cache must be a torch.Tensor")
    dev = kv_cache.device
    if dev.type != "cuda":
        raise ValueError("the KV cache operators run on CUDA tensors only")
    if kv_cache.dtype not in _CACHE:
        raise TypeError(f"unsupported kv_cache dtype {kv_cache.dtype}")
    if kv_cache.dim() != 5 or kv_cache.shape[1] != 2:
        raise ValueError("kv_cache must be [num_pages, 2, page_size, Nk, D], got "
                         f"{list(kv_cache.shape)}")
    if not kv_cache.is_contiguous():
        raise ValueError("kv_cache must be contiguous")
    pages, _, page_size, Nk, _ = kv_cache.shape
    if not isinstance(seq_offsets, torch.Tensor):
        raise TypeError("seq_offsets must be a torch.Tensor")
    index = seq_offsets.dtype
    if index not in _INDEX:
        raise TypeError("index tensors must be int32 or int64")
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
        raise ValueError("seq_offsets must be [B + 1]")
    B = seq_offsets.shape[0] - 1
    _tensor(seq_offsets, "seq_offsets", dev, index, seq_offsets.shape)
    _tensor(page_offsets, "page_offsets", dev, index, (B + 1,))
    _tensor(last_page_len, "last_page_len", dev, index, (B,))
    if not isinstance(page_ids, torch.Tensor) or page_ids.dim() != 1:
        raise ValueError("page_ids must be a one-dimensional torch.Tensor")
    _tensor(page_ids, "page_ids", dev, index, page_ids.shape)
    if kv_scale is not None:
        _tensor(kv_scale, "kv_scale", dev, torch.uint8, (pages, 2, Nk, page_size))


class _Cache:
    """The checked hstu_kv_cache (packed) and what the entry points need of it."""
    __slots__ = ("packed", "device", "index", "dtype", "B", "Nk", "D", "sizes", "keep")


def _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale, k_descale,
           v_descale, status):
    c = _Cache()
    try:  # one pass over what is usually right; _explain_cache says what is not
        dev = c.device = kv_cache.get_device()
        pages, two, page_size, Nk, D = kv_cache.shape
        index = seq_offsets.dtype
        B1, = seq_offsets.shape
        num_ids, = page_ids.shape
        ok = (dev >= 0 and two == 2 and kv_cache.dtype in _CACHE and index in _INDEX and B1 > 0 and
              kv_cache.is_contiguous() and page_offsets.shape == (B1,) and
              last_page_len.shape == (B1 - 1,) and
              (kv_scale is None or
               (kv_scale.dtype is torch.uint8 and kv_scale.get_device() == dev and
                kv_scale.shape == (pages, 2, Nk, page_size) and kv_scale.is_contiguous())))
        for t in (seq_offsets, page_offsets, page_ids, last_page_len):
            ok = ok and t.dtype is index and t.get_device() == dev and t.is_contiguous()
    except (AttributeError, ValueError, TypeError):
        ok = False
    if not ok:
        _explain_cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale)
        raise ValueError("kv_cache and its page table do not fit together")
    c.dtype, c.index, c.B, c.Nk, c.D, c.keep = kv_cache.dtype, index, B1 - 1, Nk, D, None
    fp8 = c.dtype is _FP8
    descale, kd, vd = _abi.HSTU_DESCALE_CAST, 0, 0
    if kv_scale is not None or k_descale is not None or v_descale is not None:
        if not fp8:
            raise ValueError("kv_scale, k_descale and v_descale go with FP8 E4M3 caches")
        if kv_scale is None:
            descale, *c.keep = _factors(k_descale, v_descale, kv_cache.device, c.B, Nk)
            kd, vd = c.keep[0].data_ptr(), c.keep[1].data_ptr()
        elif k_descale is not None or v_descale is not None:
            raise ValueError("a cache has row scales (kv_scale) or static factors, not both")
    status_ptr = 0 if status is None else _tensor(status, "status", kv_cache.device, torch.int32,
                                                  (1,))
    c.sizes = (_CACHE[c.dtype], c.B, Nk, D, page_size, index is torch.int64, descale)
    c.packed = _PACK_CACHE(*c.sizes, 0, kv_cache.data_ptr(),
                           0 if kv_scale is None else kv_scale.data_ptr(), pages,
                           page_offsets.data_ptr(), page_ids.data_ptr(), last_page_len.data_ptr(),
                           num_ids, kd, vd, status_ptr)
    return c


def _row_dtype(c, dtype):
    code = _ROWS.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    if c.dtype is not dtype and c.dtype is not _FP8:
        raise TypeError(f"{dtype} rows need a kv_cache of their type or of FP8 E4M3, got "
                        f"{c.dtype}")
    return code


def _call(name, c, *args):
    """One entry point on the cache's device and that device's current stream."""
    fn = getattr(_abi.lib(), name)
    if torch._C._cuda_getDevice() == c.device:
        status = fn(c.packed, *args, torch._C._cuda_getCurrentRawStream(c.device))
    else:
        with torch.cuda.device(c.device):
            status = fn(c.packed, *args, torch._C._cuda_getCurrentRawStream(c.device))
    if status:
        _abi.check(status, name)


def _copy(name, c, k, v, seq_offsets, new=False):
    """hstu_kv_append / hstu_kv_read of the rows k and v (new: just allocated, nothing to check)."""
    dtype = _row_dtype(c, k.dtype)
    T = k.shape[0]
    if new:
        k_stride = v_stride = c.Nk * c.D
    else:
        k_stride = _rows(k, "k", c.device, k.dtype, c.Nk, c.D)
        v_stride = _rows(v, "v", c.device, k.dtype, c.Nk, c.D)
        if v.shape[0] != T:
            raise ValueError("k and v must have one shape")
    _call(name, c, _PACK_ROWS(k.data_ptr(), v.data_ptr(), k_stride, v_stride,
                              seq_offsets.data_ptr(), T, dtype, 0))


@functools.lru_cache(maxsize=4096)
def _workspace_bytes(device, cache_sizes, attn_sizes):
    """hstu_softmax_workspace for these sizes (it reads no pointer) on this device."""
    need = ctypes.c_longlong(0)
    with torch.cuda.device(device):
        _abi.check(_abi.lib().hstu_softmax_workspace(
            _PACK_CACHE(*cache_sizes, 0, 0, 0, 1, 0, 0, 0, 0, 0, 0, 0),
            _PACK_ATTN(0, 0, 0, *attn_sizes, 0, 0, 0, 0, 0), ctypes.byref(need)),
            "hstu_softmax_workspace")
    return need.value


def hstu_kv_append(k, v, seq_offsets, kv_cache, *, page_offsets, page_ids, last_page_len,
                   kv_scale=None, k_descale=None, v_descale=None, status=None):
    """Write new rows into the paged cache; returns kv_cache.

    k, v [T, Nk, D] fp32, fp16 or bf16; rows of D * Nk contiguous elements, which may be
    slices of a wider tensor (a fused projection's output). seq_offsets [B+1] gives each
    sequence its new rows. kv_cache [num_pages, 2, page_size, Nk, D] (page_size 32, 128 or
    256, D a multiple of 16 up to 256) of k's type or float8_e4m3fn. page_offsets [B+1],
    page_ids and last_page_len [B] describe the sequences with the new rows, which are their
    last ones. Index tensors: int32 or int64, all of one type.

    E4M3 caches are quantised: kv_scale [num_pages, 2, Nk, page_size] uint8 takes one power of
    two per row and head, 2^(kv_scale - 127), the smallest that brings the row's largest
    magnitude to 448 or less; k_descale / v_descale (floats or one-element fp32 tensors, [B] or
    [B, Nk]: hstu_fwd's factors) divide the rows; neither is a plain cast. Rounding is to
    nearest even, saturating at +-448. (hstu_fwd reads the last two forms; a cache with row
    scales goes to hstu_softmax_fwd, or to hstu_fwd by way of hstu_kv_read.)

    status: an int32 tensor of one element that is set to 1 where offsets, lengths or page ids
    are found invalid on the device (nothing of such a sequence is written)."""
    c = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale, k_descale,
               v_descale, status)
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    _copy("hstu_kv_append", c, k, v, seq_offsets)
    return kv_cache


def hstu_kv_read(kv_cache, seq_offsets, *, page_offsets, page_ids, last_page_len,
                 total_tokens=None, dtype=None, kv_scale=None, k_descale=None, v_descale=None,
                 k=None, v=None, status=None):
    """Read rows of the paged cache back as contiguous k, v [T, Nk, D] (what hstu_fwd takes
    with seq_offsets_k = seq_offsets): the last seq_offsets[b+1] - seq_offsets[b] rows of each
    sequence, which is all of it when that is its length. total_tokens = T, at least
    seq_offsets[B]. dtype: fp32, fp16 or bf16 (default: the cache's; for an E4M3 cache, which is
    dequantised by kv_scale or k_descale / v_descale, bf16). k and v may be given instead (rows
    as for hstu_kv_append); rows of no sequence are left as they were. Other arguments as for
    hstu_kv_append."""
    c = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale, k_descale,
               v_descale, status)
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    new = k is None
    if new:
        if total_tokens is None:
            raise ValueError("hstu_kv_read needs total_tokens, or k and v")
        if dtype is None:
            dtype = torch.bfloat16 if c.dtype is _FP8 else c.dtype
        _row_dtype(c, dtype)
        shape = (int(total_tokens), c.Nk, c.D)
        k = torch.empty(shape, dtype=dtype, device=kv_cache.device)
        v = torch.empty(shape, dtype=dtype, device=kv_cache.device)
    elif not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    elif dtype not in (None, k.dtype) or total_tokens not in (None, k.shape[0]):
        raise ValueError("dtype and total_tokens must be those of k")
    _copy("hstu_kv_read", c, k, v, seq_offsets, new)
    return k, v


def hstu_softmax_fwd(q, kv_cache, seq_offsets, *, max_seqlen, max_seqlen_k, page_offsets,
                     page_ids, last_page_len, causal=True, alpha=1.0, kv_scale=None,
                     k_descale=None, v_descale=None, out=None, return_lse=False, status=None):
    """Softmax attention of the newest tokens of each sequence over its paged cache, which
    holds their keys too (hstu_kv_append first).

    q [T, Nq, D] fp32, fp16 or bf16 (rows may be slices of a wider tensor), Nq a multiple of
    the cache's Nk; the cache of q's type or float8_e4m3fn (kv_scale or k_descale / v_descale as
    hstu_kv_append wrote it). The n = seq_offsets[b+1] - seq_offsets[b] queries of a sequence
    are its last n positions; with causal=True each sees the keys up to its own position, with
    causal=False all of them (n may then exceed the keys: cross attention). max_seqlen bounds n,
    max_seqlen_k the cached keys of a sequence.

    out = softmax(alpha q k^T) v with q's shape and type; with return_lse also ln sum exp(alpha
    q k) [T, Nq] fp32. A row that sees no key gets 0 (lse -inf); rows of no sequence are left
    as allocated. Other arguments as for hstu_kv_append."""
    c = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale, k_descale,
               v_descale, status)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    dtype = _row_dtype(c, q.dtype)
    q_stride = _rows(q, "q", c.device, q.dtype, None, c.D)
    T, Nq, D = shape = q.shape
    if Nq % c.Nk:
        raise ValueError(f"q's heads ({Nq}) must be a multiple of the cache's ({c.Nk})")
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=q.device)
        out_ptr = out.data_ptr()
    else:
        out_ptr = _tensor(out, "out", kv_cache.device, q.dtype, shape)
    lse = torch.empty((T, Nq), dtype=torch.float32, device=q.device) if return_lse else None
    sizes = (T, dtype, Nq, int(max_seqlen), int(max_seqlen_k), bool(causal), float(alpha))
    try:
        need = _workspace_bytes(c.device, c.sizes, sizes)
    except (struct.error, OverflowError):  # max_seqlen, max_seqlen_k or alpha that no C type holds
        raise _abi.HstuError(_abi.HSTU_ERR_INVALID_ARG, "hstu_softmax_fwd") from None
    workspace = torch.empty((need,), dtype=torch.uint8, device=q.device) if need else None
    _call("hstu_softmax_fwd", c,
          _PACK_ATTN(q.data_ptr(), q_stride, seq_offsets.data_ptr(), *sizes, out_ptr,
                     0 if lse is None else lse.data_ptr(),
                     0 if workspace is None else workspace.data_ptr(), need, 0))
    return (out, lse) if return_lse else out
