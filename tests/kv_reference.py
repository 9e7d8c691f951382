"""Plain 64-bit implementations of the paged KV cache operators (numpy, by the formulas of
include/hstu_kv.h), and the input tables their tests share."""
import numpy as np
import torch

FP8 = torch.float8_e4m3fn
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {t: torch.finfo(t).eps / 2 for t in DTYPES.values()}


def e4m3_round(x):
    """Nearest E4M3 value, ties to even, saturating at +-448; NaN stays."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    e = np.frexp(np.maximum(a, 2.0 ** -6))[1] - 1  # the leading bit; subnormals share 2^-6's
    step = np.ldexp(1.0, e - 3)
    return np.copysign(np.minimum(np.round(a / step) * step, 448.0), x)


def row_exponent(x):
    """Smallest e >= -100 with max finite |x| <= 448 * 2^e, over the last axis."""
    a = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    e = np.full(a.shape, -100, dtype=np.int64)
    while True:
        big = a > 448.0 * np.ldexp(1.0, e)
        if not big.any():
            return e
        e[big] += 1


class Table:
    """Sequences of the given lengths in a paged cache (CPU tensors): a random permutation of
    pages, of which `spare` belong to no sequence."""

    def __init__(self, lengths, page_size, index=torch.int64, spare=3, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.page_size, self.index = [int(x) for x in lengths], page_size, index
        pages = [-(-n // page_size) for n in self.lengths]
        self.num_pages = sum(pages) + spare
        self.page_offsets = torch.tensor(np.concatenate([[0], np.cumsum(pages)]), dtype=index)
        self.page_ids = torch.randperm(self.num_pages, generator=g)[:sum(pages)].to(index)
        self.last_page_len = torch.tensor([n - (p - 1) * page_size if p else 1
                                           for n, p in zip(self.lengths, pages)], dtype=index)

    def rows(self, b):
        """Page and row in the page of every position of sequence b."""
        at = np.arange(self.lengths[b])
        first = int(self.page_offsets[b])
        return self.page_ids.numpy()[first + at // self.page_size].astype(np.int64), \
            at % self.page_size

    def args(self, dev):
        return dict(page_offsets=self.page_offsets.to(dev), page_ids=self.page_ids.to(dev),
                    last_page_len=self.last_page_len.to(dev))


def offsets(n, index=torch.int64):
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=index)


def values(x):
    """A CPU tensor's values in 64 bits (E4M3 too)."""
    return x.to(torch.float32).numpy().astype(np.float64) if x.dtype == FP8 else \
        x.double().numpy()


def cache_values(cache, scale=None, kd=None, vd=None):
    """[pages, 2, page_size, Nk, D] in 64 bits; kd, vd: one factor of every element of K, V."""
    x = values(cache)
    if scale is not None:
        x = x * np.ldexp(1.0, scale.numpy().astype(np.int64) - 127).swapaxes(2, 3)[..., None]
    return x


def softmax_rows(q, K, V, causal, alpha):
    """q [n, Nq, D], K, V [Lk, Nk, D] -> out, lse, weighted |v|, and the largest |alpha| |q| |k|
    (bound on a score) per row and head."""
    n, Nq, D = q.shape
    Lk, G = K.shape[0], Nq // K.shape[1]
    out, weight = np.zeros((n, Nq, D)), np.zeros((n, Nq, D))
    lse, size = np.full((n, Nq), -np.inf), np.zeros((n, Nq))
    for h in range(Nq):
        k, v = K[:, h // G], V[:, h // G]
        if not Lk or not n:
            continue
        x = alpha * (q[:, h] @ k.T)
        if causal:
            x = np.where(np.arange(Lk)[None, :] <= (Lk - n + np.arange(n))[:, None], x, -np.inf)
        top = x.max(1, keepdims=True)
        seen = np.isfinite(top[:, 0])
        p = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = p.sum(1, keepdims=True)
        total[total == 0] = 1.0
        out[:, h], weight[:, h] = p / total @ v, p / total @ np.abs(v)
        lse[seen, h] = top[seen, 0] + np.log(total[seen, 0])
        size[:, h] = abs(alpha) * np.linalg.norm(q[:, h], axis=1) * \
            np.linalg.norm(k, axis=1).max()
    return out, lse, weight, size
