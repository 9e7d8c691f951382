"""Plain 64-bit implementation of the 4-bit cache form (numpy, by the formulas of
include/hstu_kv.h): value = 2^(s - 127) * factor * code, E2M1 codes with E4M3 factors."""
import numpy as np
import torch

import kv_reference as R

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])


def row_exponent(x):
    """Smallest e >= -100 with max finite |x| <= 2688 * 2^e, over the last axis."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(a.shape, -100, dtype=np.int64)
    while True:
        big = a > 2688.0 * np.ldexp(1.0, e)
        if not big.any():
            return e
        e[big] += 1


def e2m1_code(m):
    """Codes of the nearest E2M1 values (ties to the even code, 6 at most) of x, signs in bit 3."""
    a, sign = np.abs(m), np.signbit(m)
    code = np.zeros(a.shape, dtype=np.uint8)
    for i, mid in enumerate((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)):
        code += (a >= mid) if i % 2 else (a > mid)
    return code + 8 * sign.astype(np.uint8)


def quantise(x):
    """x [..., D] in 64 bits -> codes [..., D], factors [..., D / 16] and exponents [...]."""
    e = row_exponent(x)
    y = np.clip(np.ldexp(np.asarray(x, dtype=np.float64), -e[..., None]), -2688.0, 2688.0)
    y = y.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    factor = R.e4m3_round(np.abs(y).max(-1) / 6)  # (NaN where an element is one)
    with np.errstate(invalid="ignore", divide="ignore"):
        m = np.where(factor[..., None] == 0, 0.0, y / factor[..., None])
    return e2m1_code(m).reshape(x.shape), factor, e


def pack(code):
    """Two codes a byte, the first in the low half."""
    return torch.tensor(code[..., 0::2] | code[..., 1::2] << 4)


def tensors(code, factor, e):
    """kv_cache, kv_group_scale and kv_scale of rows [pages, 2, Nk, page_size, ..]."""
    return pack(code), torch.tensor(factor).float().to(R.FP8), torch.tensor(e + 127).to(torch.uint8)


def values(cache, group, scale):
    """[pages, 2, page_size, Nk, D] in 64 bits (CPU tensors)."""
    b = cache.view(torch.uint8).numpy()
    code = np.stack([b & 15, b >> 4], -1).reshape(*b.shape[:-1], -1)
    with np.errstate(invalid="ignore"):
        x = E2M1[code].reshape(*code.shape[:-1], -1, 16) * R.values(group)[..., None]
        x = x.reshape(code.shape) * np.ldexp(1.0, scale.numpy().astype(np.int64) - 127)[..., None]
    return x.swapaxes(2, 3)
