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

import torch

from . import _abi

__all__ = ["hstu_kv_append", "hstu_kv_read", "hstu_softmax_fwd"]

_ROWS = {torch.float32: _abi.HSTU_F32, torch.float16: _abi.HSTU_F16, torch.bfloat16: _abi.HSTU_BF16}
_CACHE = {**_ROWS, torch.float8_e4m3fn: _abi.HSTU_FP8_E4M3}
_INDEX = (torch.int32, torch.int64)


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
    """Elements between the rows of t [T, heads, head_dim], whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or t.shape[2] != head_dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [T, {'N' if heads is None else heads}, {head_dim}], "
                         f"got {list(t.shape)}")
    row, head, last = t.stride()
    width = t.shape[1] * head_dim
    if last != 1 or (head != head_dim and t.shape[1] > 1) or (row < width and t.shape[0] > 1):
        raise ValueError(f"the rows of {name} must be contiguous and may not overlap, "
                         f"got strides {list(t.stride())}")
    return row if t.shape[0] > 1 else width


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


def _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale, k_descale,
           v_descale, status):
    """The checked hstu_kv_cache, and the tensors made for it (kept until the launch)."""
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
    pages, _, page_size, Nk, D = kv_cache.shape
    if not isinstance(seq_offsets, torch.Tensor):
        raise TypeError("seq_offsets must be a torch.Tensor")
    index = seq_offsets.dtype
    if index not in _INDEX:
        raise TypeError("index tensors must be int32 or int64")
    if seq_offsets.dim() != 1 or seq_offsets.shape[0] < 1:
        raise ValueError("seq_offsets must be [B + 1]")
    B = seq_offsets.shape[0] - 1
    _tensor(seq_offsets, "seq_offsets", dev, index, seq_offsets.shape)
    c = _abi.KVCache()
    c.page_offsets = _tensor(page_offsets, "page_offsets", dev, index, (B + 1,))
    c.last_page_len = _tensor(last_page_len, "last_page_len", dev, index, (B,))
    if not isinstance(page_ids, torch.Tensor) or page_ids.dim() != 1:
        raise ValueError("page_ids must be a one-dimensional torch.Tensor")
    c.page_ids = _tensor(page_ids, "page_ids", dev, index, page_ids.shape) or None
    c.num_page_ids = page_ids.shape[0]
    fp8 = kv_cache.dtype == torch.float8_e4m3fn
    keep = None
    if not fp8 and not (kv_scale is None and k_descale is None and v_descale is None):
        raise ValueError("kv_scale, k_descale and v_descale go with FP8 E4M3 caches")
    if kv_scale is not None:
        if k_descale is not None or v_descale is not None:
            raise ValueError("a cache has row scales (kv_scale) or static factors, not both")
        c.kv_scale = _tensor(kv_scale, "kv_scale", dev, torch.uint8, (pages, 2, Nk, page_size))
    elif fp8:
        c.descale, kd, vd = _factors(k_descale, v_descale, dev, B, Nk)
        if kd is not None:
            keep = (kd, vd)
            c.k_descale, c.v_descale = kd.data_ptr(), vd.data_ptr()
    if status is not None:
        c.status = _tensor(status, "status", dev, torch.int32, (1,))
    c.dtype = _CACHE[kv_cache.dtype]
    c.batch, c.num_heads_kv, c.head_dim, c.page_size = B, Nk, D, page_size
    c.index_is_int64 = index == torch.int64
    c.kv_cache = kv_cache.data_ptr()
    c.num_pages = pages
    return c, keep


def _row_dtype(kv_cache, dtype):
    if dtype not in _ROWS:
        raise TypeError(f"unsupported dtype {dtype}")
    if kv_cache.dtype not in (dtype, torch.float8_e4m3fn):
        raise TypeError(f"{dtype} rows need a kv_cache of their type or of FP8 E4M3, got "
                        f"{kv_cache.dtype}")
    return _ROWS[dtype]


def _call(name, dev, *args):
    """One entry point on dev's current stream."""
    fn = getattr(_abi.lib(), name)
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        _abi.check(status, name)


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
    nearest even, saturating at +-448.

    status: an int32 tensor of one element that is set to 1 where offsets, lengths or page ids
    are found invalid on the device (nothing of such a sequence is written)."""
    c, keep = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale,
                     k_descale, v_descale, status)
    dev = kv_cache.device
    r = _abi.KVRows()
    if not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    r.dtype = _row_dtype(kv_cache, k.dtype)
    r.k_stride = _rows(k, "k", dev, k.dtype, c.num_heads_kv, c.head_dim)
    r.v_stride = _rows(v, "v", dev, k.dtype, c.num_heads_kv, c.head_dim)
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    r.k, r.v, r.seq_offsets = k.data_ptr(), v.data_ptr(), seq_offsets.data_ptr()
    r.total_tokens = k.shape[0]
    _call("hstu_kv_append", dev, ctypes.byref(c), ctypes.byref(r))
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
    c, keep = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale,
                     k_descale, v_descale, status)
    dev = kv_cache.device
    if (k is None) != (v is None):
        raise ValueError("k and v go together")
    if k is None:
        if total_tokens is None:
            raise ValueError("hstu_kv_read needs total_tokens, or k and v")
        if dtype is None:
            dtype = torch.bfloat16 if kv_cache.dtype == torch.float8_e4m3fn else kv_cache.dtype
        _row_dtype(kv_cache, dtype)
        shape = (int(total_tokens), c.num_heads_kv, c.head_dim)
        k = torch.empty(shape, dtype=dtype, device=dev)
        v = torch.empty(shape, dtype=dtype, device=dev)
    elif not isinstance(k, torch.Tensor):
        raise TypeError("k must be a torch.Tensor")
    elif dtype not in (None, k.dtype) or total_tokens not in (None, k.shape[0]):
        raise ValueError("dtype and total_tokens must be those of k")
    r = _abi.KVRows()
    r.dtype = _row_dtype(kv_cache, k.dtype)
    r.k_stride = _rows(k, "k", dev, k.dtype, c.num_heads_kv, c.head_dim)
    r.v_stride = _rows(v, "v", dev, k.dtype, c.num_heads_kv, c.head_dim)
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    r.k, r.v, r.seq_offsets = k.data_ptr(), v.data_ptr(), seq_offsets.data_ptr()
    r.total_tokens = k.shape[0]
    _call("hstu_kv_read", dev, ctypes.byref(c), ctypes.byref(r))
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
    c, keep = _cache(kv_cache, seq_offsets, page_offsets, page_ids, last_page_len, kv_scale,
                     k_descale, v_descale, status)
    dev = kv_cache.device
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    a = _abi.SoftmaxArgs()
    a.dtype = _row_dtype(kv_cache, q.dtype)
    a.q_stride = _rows(q, "q", dev, q.dtype, None, c.head_dim)
    T, Nq, D = q.shape
    if Nq % c.num_heads_kv:
        raise ValueError(f"q's heads ({Nq}) must be a multiple of the cache's ({c.num_heads_kv})")
    if out is None:
        out = torch.empty((T, Nq, D), dtype=q.dtype, device=dev)
        a.out = out.data_ptr()
    else:
        a.out = _tensor(out, "out", dev, q.dtype, q.shape)
    a.q, a.seq_offsets, a.total_tokens, a.num_heads_q = q.data_ptr(), seq_offsets.data_ptr(), T, Nq
    a.max_seqlen, a.max_seqlen_k = max_seqlen, max_seqlen_k
    a.causal, a.alpha = bool(causal), alpha
    lse = None
    if return_lse:
        lse = torch.empty((T, Nq), dtype=torch.float32, device=dev)
        a.lse = lse.data_ptr()
    need = ctypes.c_longlong(0)
    with torch.cuda.device(dev):
        _abi.check(_abi.lib().hstu_softmax_workspace(ctypes.byref(c), ctypes.byref(a),
                                                     ctypes.byref(need)),
                   "hstu_softmax_workspace")
    if need.value:
        workspace = torch.empty(need.value, dtype=torch.uint8, device=dev)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need.value
    _call("hstu_softmax_fwd", dev, ctypes.byref(c), ctypes.byref(a))
    return (out, lse) if return_lse else out
