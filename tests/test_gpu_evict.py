"""hstu_kv_weights, hstu_kv_select and hstu_kv_compact against plain 64-bit implementations: types,
cache forms, head layouts, lengths where tiles and pages end, rows that see nothing, ties, NaN and
infinite weights, budgets around the lengths, what must stay untouched, other streams and captured
graphs, tables that the device must reject, and the loop that a serving program runs.

Tolerance of an element of weights, from the roundings of the path: a score of D products in fp32
is off by at most (D + 8) 2^-24 |alpha| |q| |k| (bf16 queries over codes may drop 2^-38 of their
largest element besides, which is less), its product with alpha log2 e and that of lse with log2 e
by 2^-23 of them, their difference by 2^-24 of itself, at most |score| + |lse|; an exponential in
base 2 by 2^-21 relatively. An error d of an exponent moves its weight by (1 + d) d at most. n G
weights are summed in fp32. With S = sum p |alpha| |q| |k|, L = sum p |lse| and W = sum p,
  |error| <= 1.1 (D + 16) 2^-24 S + 2^-22 L + (2^-21 + n G 2^-24) W + 2^-24 |before| + 1e-30."""
import numpy as np
import pytest
import torch

import evict_reference as E
import kv4_reference as R4
import kv_reference as R
import test_gpu_kv4 as K4
import test_gpu_softmax as S
from hstu_dense_forward_gb300 import (HstuError, hstu_kv_append, hstu_kv_compact, hstu_kv_read, hstu_kv_select,
                                      hstu_kv_weights, hstu_softmax_fwd)

pytestmark = pytest.mark.gpu


def _cache(t, Nk, D, dt, mode, dev, seed):
    if mode == "fp4":
        return K4._filled(t, Nk, D, dev, seed)
    return S._filled(t, Nk, D, dt, mode, dev, seed)


def _used(t):
    """Which rows of which pages the sequences have."""
    used = np.zeros((t.num_pages, t.page_size), dtype=bool)
    for b in range(len(t.lengths)):
        page, row = t.rows(b)
        used[page, row] = True
    return used


def run_weights(dev, lengths, n, dtype, mode, Nq, Nk, D, ps, causal=True, accumulate=True,
                index=torch.int64, strided=False, seed=0, bounds=None, tail=2):
    dt = R.DTYPES[dtype]
    t = R.Table(lengths, ps, index, seed=seed)
    cache, vals, kw = _cache(t, Nk, D, dt, mode, dev, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    wide = torch.randn(sum(n) + tail, Nq + 3, D, generator=g).to(dt)
    wide[sum(n):] = float("nan")  # rows of no sequence
    wide = wide.to(dev)
    q = wide[:, 2:2 + Nq] if strided else wide[:, 2:2 + Nq].contiguous()
    alpha = D ** -0.5
    so = np.concatenate([[0], np.cumsum(n)])
    qv = R.values(q.cpu())
    lse = torch.full((sum(n) + tail, Nq), float("nan"))
    for b in range(len(n)):
        page, row = t.rows(b)
        x = R.softmax_rows(qv[so[b]:so[b + 1]], vals[page, 0, row], vals[page, 1, row], causal, alpha)[1]
        lse[so[b]:so[b + 1]] = torch.tensor(x).float()
    weights = torch.rand(t.num_pages, Nk, ps, generator=g).to(dev)
    before = weights.cpu().numpy().astype(np.float64)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sq, sk = bounds or (max(1, max(n)), max(1, max(lengths)))
    args = dict(max_seqlen=sq, max_seqlen_k=sk, causal=causal, alpha=alpha, accumulate=accumulate,
                status=status, **t.args(dev), **kw)
    offs = R.offsets(n, index).to(dev)
    other = weights.clone()
    assert hstu_kv_weights(q, lse.to(dev), cache, offs, weights, **args) is weights
    assert status.item() == 0
    hstu_kv_weights(q, lse.to(dev), cache, offs, other, **args)
    assert torch.equal(other, weights)  # the same bits
    got = weights.cpu().numpy().astype(np.float64)
    assert np.array_equal(got.swapaxes(1, 2)[~_used(t)], before.swapaxes(1, 2)[~_used(t)])
    for b in range(len(n)):
        page, row = t.rows(b)
        at = slice(so[b], so[b + 1])
        w, size, off = E.key_weights(qv[at], lse[at].double().numpy(), vals[page, 0, row], causal, alpha)
        old = before[page, :, row].T if accumulate else 0.0
        tol = 1.1 * (D + 16) * 2.0 ** -24 * size + 2.0 ** -22 * off + \
            (2.0 ** -21 + n[b] * (Nq // Nk) * 2.0 ** -24) * w + 2.0 ** -24 * np.abs(old + w) + 1e-30
        err = np.abs(got[page, :, row].T - (w + old))
        bad = ~(err <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:5], err[bad][:5], tol[bad][:5], w[bad][:5])


@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,ps,index", [
    ("bf16", "same", 8, 2, 128, 128, torch.int64), ("fp16", "same", 4, 4, 64, 32, torch.int32),
    ("bf16", "scale", 16, 4, 128, 128, torch.int32), ("fp16", "scale", 5, 1, 64, 256, torch.int64),
    ("bf16", "static", 6, 2, 128, 32, torch.int64), ("fp16", "cast", 3, 3, 96, 32, torch.int64),
    ("bf16", "fp4", 8, 2, 128, 128, torch.int64), ("fp16", "fp4", 12, 4, 96, 32, torch.int32),
    ("bf16", "fp4", 16, 1, 256, 32, torch.int64), ("fp16", "fp4", 4, 4, 32, 256, torch.int64),
    ("fp32", "same", 8, 2, 64, 32, torch.int64), ("fp32", "scale", 4, 1, 128, 128, torch.int32),
    ("fp32", "fp4", 20, 1, 256, 32, torch.int32),
    ("bf16", "same", 16, 1, 256, 128, torch.int64), ("bf16", "scale", 7, 1, 256, 32, torch.int64),
    ("fp16", "same", 12, 4, 16, 32, torch.int64), ("bf16", "scale", 32, 2, 80, 32, torch.int64),
])
def test_weights_of_single_tokens(cuda_device, dtype, mode, Nq, Nk, D, ps, index):
    for accumulate in (True, False):
        run_weights(cuda_device, S.TOKENS + [0, 70], [1] * (len(S.TOKENS)) + [0, 0], dtype, mode, Nq, Nk, D, ps,
                    index=index, seed=11, accumulate=accumulate)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,ps,strided", [
    ("bf16", "same", 8, 2, 128, 128, True), ("fp16", "same", 3, 1, 64, 32, False), ("bf16", "same", 4, 4, 96, 32, False),
    ("bf16", "scale", 4, 1, 128, 128, False), ("fp16", "scale", 4, 2, 64, 32, True), ("bf16", "static", 5, 1, 96, 256, False),
    ("fp16", "cast", 2, 2, 128, 32, False), ("fp32", "same", 4, 2, 64, 128, True), ("fp32", "scale", 2, 1, 48, 32, False),
    ("bf16", "same", 7, 1, 256, 128, True), ("fp16", "scale", 2, 2, 256, 32, False), ("fp16", "same", 2, 1, 144, 256, False),
    ("bf16", "fp4", 8, 2, 128, 128, True), ("fp16", "fp4", 6, 2, 64, 32, False), ("bf16", "fp4", 3, 1, 224, 256, False),
    ("fp32", "fp4", 4, 2, 96, 32, False), ("bf16", "same", 128, 1, 64, 32, False), ("fp16", "fp4", 40, 1, 32, 128, False),
])
def test_weights_of_chunks(cuda_device, dtype, mode, Nq, Nk, D, ps, strided, causal):
    run_weights(cuda_device, *S.CHUNK, dtype, mode, Nq, Nk, D, ps, causal=causal, seed=21, strided=strided)
    run_weights(cuda_device, *S.PROMPT, dtype, mode, Nq, Nk, D, ps, causal=causal, seed=22, accumulate=False,
                index=torch.int32)


@pytest.mark.parametrize("dtype,mode,n,Nq,D", [
    ("bf16", "same", 300, 4, 128), ("bf16", "scale", 300, 4, 128), ("fp16", "fp4", 200, 4, 64), ("bf16", "same", 7, 4, 128),
    ("fp16", "scale", 6, 4, 64), ("bf16", "same", 30, 4, 256), ("fp32", "same", 40, 4, 64), ("bf16", "fp4", 1, 4, 128)])
def test_weights_over_long_keys(cuda_device, dtype, mode, n, Nq, D):
    """Long keys parted among many CTAs, beside a short sequence, an empty one and one without queries."""
    run_weights(cuda_device, [7000, 3, 0, 600, 90], [n, 3, 0, n // 3, 0], dtype, mode, Nq, 2, D, 128, seed=101)
    run_weights(cuda_device, [4000, 3, 0, 600, 90], [n, 3, 0, n // 3, 0], dtype, mode, Nq, 2, D, 32, seed=102,
                bounds=(n + 100, 50000), accumulate=False)


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("fp16", "scale"), ("fp32", "same"), ("bf16", "fp4")])
def test_weights_with_more_queries_than_keys(cuda_device, dtype, mode):
    for causal in (True, False):
        run_weights(cuda_device, [3, 0, 40, 129], [10, 4, 41, 300], dtype, mode, 4, 2, 64, 32, causal=causal, seed=41)
        run_weights(cuda_device, [3, 0, 9], [5, 1, 8], dtype, mode, 2, 2, 64, 32, causal=causal, seed=42)


def test_weights_of_many_sequences(cuda_device):
    B = 300
    lengths = [(37 * b) % 400 + 20 for b in range(B)]
    for n in (1, 20):
        run_weights(cuda_device, lengths, [n] * B, "bf16", "same", 4, 2, 64, 32, seed=91)


def test_weights_without_queries(cuda_device):
    """No tokens at all: nothing to add; stored, 0 for every cached row."""
    dev = cuda_device
    t = R.Table([40, 0, 7], 32)
    cache, _, kw = _cache(t, 2, 64, torch.bfloat16, "same", dev, 3)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=dev)
    lse = torch.empty(0, 4, device=dev)
    w = torch.rand(t.num_pages, 2, 32, device=dev)
    before = w.clone()
    args = dict(max_seqlen=1, max_seqlen_k=64, **t.args(dev))
    so = torch.zeros(4, dtype=torch.int64, device=dev)
    hstu_kv_weights(q, lse, cache, so, w, **args)
    assert torch.equal(w, before)
    hstu_kv_weights(q, lse, cache, so, w, accumulate=False, **args)
    used = torch.tensor(_used(t)).to(dev)[:, None].expand(-1, 2, -1)
    assert (w[used] == 0).all() and torch.equal(w[~used], before[~used])


def test_weights_of_queries_without_heads(cuda_device):
    """Rows of no heads add nothing; stored, 0."""
    dev = cuda_device
    for dtype in (torch.bfloat16, torch.float32):
        t = R.Table([40, 0, 7], 32)
        cache, _, kw = _cache(t, 2, 64, dtype, "same", dev, 3)
        w = torch.rand(t.num_pages, 2, 32, device=dev)
        before = w.clone()
        args = dict(max_seqlen=3, max_seqlen_k=64, **t.args(dev))
        q, lse = torch.empty(6, 0, 64, dtype=dtype, device=dev), torch.empty(6, 0, device=dev)
        so = R.offsets([3, 0, 3]).to(dev)
        hstu_kv_weights(q, lse, cache, so, w, **args)
        assert torch.equal(w, before)
        hstu_kv_weights(q, lse, cache, so, w, accumulate=False, **args)
        used = torch.tensor(_used(t)).to(dev)[:, None].expand(-1, 2, -1)
        assert (w[used] == 0).all() and torch.equal(w[~used], before[~used])


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("fp16", "scale"), ("bf16", "fp4"), ("fp32", "same")])
@pytest.mark.parametrize("n", [8, 9, 17, 200])
def test_weights_of_many_queries_without_heads(cuda_device, dtype, mode, n):
    """However many tokens have no heads: nothing is reported, and 0 stored for every cached row."""
    dev, dt = cuda_device, R.DTYPES[dtype]
    t = R.Table([n + 40, n, 7], 32)
    cache, _, kw = _cache(t, 2, 64, dt, mode, dev, 3)
    lengths = [n, n, 3]
    q, lse = torch.empty(sum(lengths), 0, 64, dtype=dt, device=dev), torch.empty(sum(lengths), 0, device=dev)
    so = R.offsets(lengths).to(dev)
    used = torch.tensor(_used(t)).to(dev)[:, None].expand(-1, 2, -1)
    for accumulate in (True, False):
        w = torch.rand(t.num_pages, 2, 32, device=dev)
        before = w.clone()
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        hstu_kv_weights(q, lse, cache, so, w, max_seqlen=n, max_seqlen_k=n + 40, accumulate=accumulate, status=status,
                        **t.args(dev), **kw)
        assert status.item() == 0
        assert torch.equal(w[~used], before[~used])
        assert torch.equal(w[used], before[used] if accumulate else torch.zeros_like(w[used]))


@pytest.mark.parametrize("dtype,mode,n,Nq,Nk,D", [("bf16", "same", 2100, 4, 1, 128), ("fp16", "scale", 700, 16, 1, 64),
                                                  ("bf16", "fp4", 1500, 8, 2, 32), ("fp16", "same", 900, 8, 1, 256)])
def test_weights_of_few_prompts(cuda_device, dtype, mode, n, Nq, Nk, D):
    """Clusters of CTAs divide the query rows of a step of keys; a short sequence beside."""
    for causal in (True, False):
        run_weights(cuda_device, [n, 9], [n, 5], dtype, mode, Nq, Nk, D, 128, causal=causal, seed=111)


# ------------------------------------------------------------------ select
def check_select(dev, t, weights, budget, recent, bound=None):
    Nk, ps = weights.shape[1], t.page_size
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    before = weights.clone()
    kept, new = hstu_kv_select(weights, budget=budget, recent=recent, max_seqlen_k=bound or max(1, max(t.lengths)),
                               status=status, **t.args(dev))
    assert status.item() == 0 and kept.dtype == torch.int32 and kept.shape == (len(t.lengths), Nk, budget)
    assert torch.equal(weights.nan_to_num(nan=7.0), before.nan_to_num(nan=7.0))
    w = weights.cpu().numpy()
    ids = []
    for b, L in enumerate(t.lengths):
        page, row = t.rows(b)
        keep = min(L, budget)
        for hk in range(Nk):
            want = E.select(w[page, hk, row], budget, recent)
            got = kept[b, hk].tolist()
            assert got[:keep] == want and got[keep:] == [-1] * (budget - keep), (b, hk)
        pages = -(-keep // ps)
        first = int(t.page_offsets[b])
        ids += t.page_ids[first:first + pages].tolist()
        assert new["page_offsets"][b + 1].item() == len(ids)
        assert new["last_page_len"][b].item() == (keep - (pages - 1) * ps if pages else 1)
    assert new["page_offsets"][0].item() == 0
    assert new["page_ids"].tolist() == ids + [-1] * (t.page_ids.numel() - len(ids))
    assert all(new[k].dtype == t.index and new[k].shape == getattr(t, k).shape for k in new)
    return kept, new


LENGTHS = [0, 1, 31, 32, 33, 100, 127, 128, 129, 257, 1023, 1024, 1025, 2500, 5]


@pytest.mark.parametrize("ps,index,Nk", [(32, torch.int64, 3), (128, torch.int32, 2), (256, torch.int64, 1)])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (1, 9), (32, 0), (33, 32), (100, 16), (128, 128), (1024, 200),
                                           (1025, 5000), (3000, 0), (3000, 7)])
def test_select(cuda_device, ps, index, Nk, budget, recent):
    t = R.Table(LENGTHS, ps, index, seed=3)
    g = torch.Generator().manual_seed(budget)
    w = torch.exp(2 * torch.randn(t.num_pages, Nk, ps, generator=g))
    w[torch.rand(w.shape, generator=g) < 0.2] = 0
    check_select(cuda_device, t, w.to(cuda_device), budget, recent, 4096)


@pytest.mark.parametrize("kind", ["equal", "few", "signs", "odd", "close", "tiny"])
@pytest.mark.parametrize("budget,recent", [(40, 0), (300, 13), (1500, 100)])
def test_select_of_special_weights(cuda_device, kind, budget, recent):
    """All equal, few values, negative ones and both zeros, infinities and NaN, neighbours in fp32,
    values below fp32's normal range: ties go to the lower position."""
    t = R.Table(LENGTHS, 32, seed=4)
    g = torch.Generator().manual_seed(7)
    shape = (t.num_pages, 2, 32)
    few = torch.tensor({"equal": [0.5], "few": [1.0, 2.0, 3.0], "signs": [-1.0, -0.0, 0.0, 1.0, -2.5],
                        "odd": [float("inf"), float("-inf"), float("nan"), 0.0, 1.0, -1.0, -float("nan")],
                        "close": [1.0, 1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24, 1.0 + 2.0 ** -22],
                        "tiny": [0.0, 1e-45, 3e-45, 1e-39, 2e-38]}[kind])
    w = few[torch.randint(0, len(few), shape, generator=g)]
    check_select(cuda_device, t, w.to(cuda_device), budget, recent)


@pytest.mark.parametrize("length,budget,recent", [(20000, 4096, 256), (70000, 10000, 0), (150000, 75000, 1000)])
def test_select_of_long_sequences(cuda_device, length, budget, recent):
    t = R.Table([length, 3, length // 2 + 1, 0], 256, torch.int32, seed=5)
    g = torch.Generator().manual_seed(8)
    w = torch.exp(2 * torch.randn(t.num_pages, 2, 256, generator=g))
    w[torch.rand(w.shape, generator=g) < 0.4] = 0
    check_select(cuda_device, t, w.to(cuda_device), budget, recent)


def test_select_of_one_long_sequence_among_many(cuda_device):
    """Lists that a CTA each works on, one of more positions than its shared memory holds."""
    t = R.Table([70000] + [40] * 330, 128, seed=12)
    g = torch.Generator().manual_seed(10)
    w = torch.exp(2 * torch.randn(t.num_pages, 1, 128, generator=g))
    check_select(cuda_device, t, w.to(cuda_device), 30000, 100)


def test_select_of_many_sequences(cuda_device):
    B = 3000  # more than a CTA's threads
    t = R.Table([(13 * b) % 90 for b in range(B)], 32, torch.int32, seed=6)
    w = torch.rand(t.num_pages, 1, 32, generator=torch.Generator().manual_seed(9))
    check_select(cuda_device, t, w.to(cuda_device), 40, 5)


# ------------------------------------------------------------------ compact
def _lists(t, Nk, budget, seed, kind="random"):
    """kept [B, Nk, budget]: increasing positions, -1 behind them."""
    rng = np.random.default_rng(seed)
    kept = np.full((len(t.lengths), Nk, budget), -1, dtype=np.int32)
    for b, L in enumerate(t.lengths):
        for hk in range(Nk):
            m = min(L, budget)
            if kind == "random":
                m = min(m, int(rng.integers(0, budget + 1)) if hk else m)
                x = np.sort(rng.permutation(L)[:m])
            elif kind == "first":
                x = np.arange(m)
            elif kind == "last":
                x = np.arange(L - m, L)
            else:  # all but one early row
                x = np.delete(np.arange(L), 1)[:m] if L > 2 else np.arange(min(L, m))
            kept[b, hk, :len(x)] = x
    return kept


def check_compact(dev, t, Nk, D, mode, dt, kept, with_weights=True, seed=5, bound=None):
    ps = t.page_size
    cache, _, kw = _cache(t, Nk, D, dt, mode, dev, seed)
    kw = {k: v for k, v in kw.items() if "descale" not in k}
    w = torch.rand(t.num_pages, Nk, ps, device=dev) if with_weights else None
    tensors = [x for x in (cache, kw.get("kv_scale"), kw.get("kv_group_scale"), w) if x is not None]

    def numpy(x):
        return x.contiguous().view(torch.uint8).cpu().numpy().reshape(*x.shape[:-1], -1).copy()

    want = [numpy(x) for x in tensors]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    assert hstu_kv_compact(cache, torch.tensor(kept, device=dev), weights=w, status=status, max_seqlen_k=bound,
                           **t.args(dev), **kw) is cache
    assert status.item() == 0
    for i, x in enumerate(want):
        last = i == len(want) - 1 and with_weights
        # heads before rows, then any number of bytes
        rows = x.reshape(*tensors[i].shape[:-1], -1) if not (tensors[i] is kw.get("kv_scale") or last) else \
            x.reshape(*tensors[i].shape, -1)
        if tensors[i] is cache and mode != "fp4":
            rows = rows.swapaxes(2, 3)
        if last:
            rows = rows[:, None]
        old = rows.copy()
        for b in range(len(t.lengths)):
            page, row = t.rows(b)
            for hk in range(Nk):
                k = kept[b, hk][kept[b, hk] >= 0]
                rows[page[:len(k)], :, hk, row[:len(k)]] = old[page[k], :, hk, row[k]]
        if tensors[i] is cache and mode != "fp4":
            rows = rows.swapaxes(2, 3)
        assert np.array_equal(numpy(tensors[i]).reshape(-1), np.ascontiguousarray(rows).reshape(-1)), i


@pytest.mark.parametrize("kind", ["random", "last", "first", "hole"])
@pytest.mark.parametrize("dtype,mode,Nk,D,ps,index", [
    ("bf16", "same", 2, 128, 128, torch.int64), ("fp16", "same", 3, 16, 32, torch.int32), ("fp32", "same", 1, 256, 32, torch.int64),
    ("bf16", "scale", 4, 128, 128, torch.int32), ("bf16", "cast", 2, 16, 32, torch.int64), ("fp16", "scale", 1, 208, 256, torch.int64),
    ("bf16", "fp4", 2, 128, 128, torch.int64), ("bf16", "fp4", 1, 32, 32, torch.int32), ("fp32", "fp4", 3, 256, 256, torch.int64),
    ("bf16", "same", 1, 80, 32, torch.int64),
])
def test_compact(cuda_device, dtype, mode, Nk, D, ps, index, kind):
    t = R.Table(LENGTHS, ps, index, seed=3)
    for budget in (700, 33):
        check_compact(cuda_device, t, Nk, D, mode, R.DTYPES[dtype], _lists(t, Nk, budget, budget, kind),
                      with_weights=budget == 700, bound=None if budget == 33 else 2500)


@pytest.mark.parametrize("mode,D", [("same", 128), ("scale", 64), ("fp4", 128)])
@pytest.mark.parametrize("kind", ["random", "last", "hole"])
def test_compact_of_long_sequences(cuda_device, mode, D, kind):
    """Many rounds, whose sources and destinations overlap."""
    t = R.Table([30000, 5, 0, 17000], 128, torch.int32, seed=3)
    check_compact(cuda_device, t, 2, D, mode, torch.bfloat16, _lists(t, 2, 20000, 9, kind))


@pytest.mark.parametrize("length,budget", [(200000, 100000), (30000, 29990), (1150000, 1100000)])
def test_compact_of_lists_of_many_chunks(cuda_device, length, budget):
    """Rows of a kilobyte, of which few make a chunk: thousands of chunks, and more than 65536, whose
    sources are far away or next door."""
    dev, D, ps = cuda_device, 256, 256
    t = R.Table([length], ps, torch.int32, seed=3)
    g = torch.Generator(device=dev).manual_seed(4)
    cache = torch.randint(0, 1 << 30, (t.num_pages, 2, ps, 1, D), generator=g, device=dev, dtype=torch.int32).view(torch.float32)
    kept = torch.randperm(length, generator=g, device=dev)[:budget].sort().values
    page = t.page_ids.to(dev).long()
    want = cache.view(torch.int32).clone()
    to = torch.arange(budget, device=dev)
    want[page[to // ps], :, to % ps] = want[page[kept // ps], :, kept % ps]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    hstu_kv_compact(cache, kept.int().view(1, 1, -1), status=status, **t.args(dev))
    assert status.item() == 0 and torch.equal(cache.view(torch.int32), want)


def test_compact_again_is_no_change(cuda_device):
    """Lists that keep rows where they are move nothing."""
    t = R.Table([300, 64], 32)
    check_compact(cuda_device, t, 2, 64, "same", torch.bfloat16, _lists(t, 2, 300, 1, "first"))


@pytest.mark.parametrize("mode,D,budget", [("same", 128, 20), ("same", 128, 3000), ("fp4", 64, 3000), ("scale", 256, 3000)])
@pytest.mark.parametrize("at", [1, 17, 64, 128, 1000, 2999])
@pytest.mark.parametrize("kind", ["same again", "before", "ended", "behind"])
def test_lists_that_do_not_increase_end_there(cuda_device, mode, D, budget, at, kind):
    """Of short lists and of those that many CTAs move, with as good as anything behind the end."""
    if at >= budget:
        return
    dev, ps = cuda_device, 32
    t = R.Table([4000, 3500], ps, torch.int32, seed=3)
    whole = _lists(t, 1, budget, 4)
    bad, ended = whole.copy(), whole.copy()
    ended[1, 0, at:] = -1
    bad[1, 0, at] = {"same again": bad[1, 0, at - 1], "before": bad[1, 0, 0] - (bad[1, 0, 0] > 0), "ended": -1, "behind": 3500}[kind]
    if kind != "ended":
        bad[1, 0, at + 1:at + 7] = np.array([5, 5, 1 << 30, 70, -3, 0])[:max(0, budget - at - 1)]
    results = []
    for lists in (bad, ended):
        cache, _, kw = _cache(t, 1, D, torch.bfloat16, mode, dev, 5)
        w = torch.rand(t.num_pages, 1, ps, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        hstu_kv_compact(cache, torch.tensor(lists, device=dev), weights=w, status=status, **t.args(dev), **kw)
        assert status.item() == (lists is bad and kind != "ended")
        results.append([x.contiguous().view(torch.uint8) for x in (cache, w, *kw.values())])
    assert all(torch.equal(x, y) for x, y in zip(*results))


@pytest.mark.parametrize("budget", [10, 60, 3000])
@pytest.mark.parametrize("length", [0, 1, 7, 40])
def test_lists_that_go_on_behind_the_sequence(cuda_device, budget, length):
    """Reported, also where every position before is kept; the others' lists and the rows are as
    without what lies behind."""
    dev, ps = cuda_device, 32
    t = R.Table([3500, length, 50], ps, seed=3)
    m = min(length, budget)
    whole = _lists(t, 1, budget, 4, "first")
    bad = whole.copy()
    if m < budget:
        bad[1, 0, m:m + 3] = [max(length, 5), 70, 2][:budget - m]
    for more, good in ((bad, m == budget), (whole, True)):
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        cache, _, _ = _cache(t, 1, 64, torch.bfloat16, "same", dev, 5)
        w = torch.rand(t.num_pages, 1, ps, device=dev)
        before = [cache.clone().view(torch.uint8), w.clone()]
        hstu_kv_compact(cache, torch.tensor(more, device=dev), weights=w, status=status, **t.args(dev))
        assert status.item() == (not good)
        assert torch.equal(cache.view(torch.uint8), before[0]) and torch.equal(w, before[1])


def test_lists_and_tables_that_the_device_rejects(cuda_device):
    """Positions out of range and page ids out of range: no access outside, a status, the rest done."""
    dev = cuda_device
    t = R.Table([100, 40, 33], 32)
    cache, _, _ = _cache(t, 1, 64, torch.bfloat16, "same", dev, 5)
    for bad in (100, 1 << 30, -5):
        kept = torch.tensor(_lists(t, 1, 20, 1, "last")).to(dev)
        kept[1, 0, 3] = bad
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        hstu_kv_compact(cache.clone(), kept, status=status, **t.args(dev))
        assert (status.item() == 1) == (bad >= 0)
    kept = torch.tensor(_lists(t, 1, 20, 1, "last")).to(dev)
    w = torch.rand(t.num_pages, 1, 32, device=dev)
    so = R.offsets([1, 1, 1]).to(dev)
    q, lse = torch.ones(3, 1, 64, dtype=torch.bfloat16, device=dev), torch.zeros(3, 1, device=dev)
    good = t.args(dev)
    for change in (dict(page_ids=good["page_ids"] + t.num_pages), dict(last_page_len=good["last_page_len"] + 50),
                   dict(page_offsets=good["page_offsets"] + 5), dict(page_offsets=good["page_offsets"].flip(0)),
                   dict(page_ids=-1 - good["page_ids"])):
        args = {**good, **change}
        for call in (lambda s: hstu_kv_select(w, budget=30, recent=3, max_seqlen_k=128, status=s, **args),
                     lambda s: hstu_kv_compact(cache, kept, weights=w, status=s, **args),
                     lambda s: hstu_kv_weights(q, lse, cache, so, w, max_seqlen=1, max_seqlen_k=128, status=s, **args),
                     lambda s: hstu_kv_weights(q.repeat(20, 1, 1), lse.repeat(20, 1), cache, so * 20, w, max_seqlen=20,
                                               max_seqlen_k=128, status=s, **args)):
            status = torch.zeros(1, dtype=torch.int32, device=dev)
            call(status)
            assert status.item() == 1
    # sequences that share entries of page_ids: more of them than there is room for
    for index in (torch.int32, torch.int64):
        table = dict(page_offsets=torch.tensor([0, 8, 3, 8], dtype=index, device=dev),
                     page_ids=torch.arange(8, dtype=index, device=dev),
                     last_page_len=torch.tensor([32, 32, 32], dtype=index, device=dev))
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        kept, new = hstu_kv_select(torch.rand(8, 1, 32, device=dev), budget=256, max_seqlen_k=256, status=status, **table)
        assert status.item() == 1 and new["page_offsets"].tolist() == [0, 8, 8, 9]
        assert new["page_ids"].tolist() == list(range(8))
    # a length above its bound leaves the sequence out
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kept, new = hstu_kv_select(w, budget=30, max_seqlen_k=64, status=status, **good)
    assert status.item() == 1 and (kept[0] == -1).all() and new["page_offsets"].tolist() == [0, 0, 1, 2]


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("mode", ["same", "scale", "fp4"])
def test_a_serving_loop(cuda_device, mode):
    """A prompt, then tokens; the cache is shortened in between, and what attention gives over it is
    attention over the kept rows."""
    dev, Nq, Nk, D, ps, B = cuda_device, 4, 2, 64, 32, 3
    g = torch.Generator().manual_seed(1)
    pages = 60
    dt = torch.bfloat16
    if mode == "fp4":
        cache = torch.zeros(pages, 2, Nk, ps, D // 2, dtype=torch.uint8, device=dev)
        kw = dict(kv_scale=torch.zeros(pages, 2, Nk, ps, dtype=torch.uint8, device=dev),
                  kv_group_scale=torch.zeros(pages, 2, Nk, ps, D // 16, device=dev).to(R.FP8))
    else:
        cache = torch.zeros(pages, 2, ps, Nk, D, device=dev).to(dt if mode == "same" else R.FP8)
        kw = dict(kv_scale=torch.zeros(pages, 2, Nk, ps, dtype=torch.uint8, device=dev)) if mode == "scale" else {}
    free = torch.randperm(pages, generator=g).tolist()
    owned, lengths = [[] for _ in range(B)], [0] * B
    weights = torch.zeros(pages, Nk, ps, device=dev)
    kept_rows = [[[] for _ in range(Nk)] for _ in range(B)]  # (k, v) of every row that should be there

    def table():
        return dict(page_offsets=R.offsets([len(o) for o in owned]).to(dev),
                    page_ids=torch.tensor([p for o in owned for p in o], device=dev),
                    last_page_len=torch.tensor([L - (len(o) - 1) * ps if o else 1 for L, o in zip(lengths, owned)], device=dev))

    def step(n):
        for b in range(B):
            lengths[b] += n[b]
            while len(owned[b]) * ps < lengths[b]:
                owned[b].append(free.pop())
        q, k, v = (torch.randn(sum(n), h, D, generator=g).to(dt).to(dev) for h in (Nq, Nk, Nk))
        so, tab = R.offsets(n).to(dev), table()
        hstu_kv_append(k, v, so, cache, **tab, **kw)
        kr, vr = hstu_kv_read(cache, so, total_tokens=sum(n), dtype=dt, **tab, **kw)
        ends = np.concatenate([[0], np.cumsum(n)])
        for b in range(B):
            for h in range(Nk):
                kept_rows[b][h] += [(kr[i, h].double().cpu(), vr[i, h].double().cpu()) for i in range(ends[b], ends[b + 1])]
        bounds = dict(max_seqlen=max(n), max_seqlen_k=max(lengths))
        out, lse = hstu_softmax_fwd(q, cache, so, alpha=0.3, return_lse=True, **bounds, **tab, **kw)
        hstu_kv_weights(q, lse, cache, so, weights, alpha=0.3, **bounds, **tab, **kw)
        for b in range(B):
            for h in range(Nq):
                K, V = (torch.stack(x) for x in zip(*kept_rows[b][h // 2]))
                x = 0.3 * q[ends[b]:ends[b + 1], h].double().cpu() @ K.T
                i = torch.arange(n[b])[:, None]
                x[torch.arange(lengths[b])[None] > lengths[b] - n[b] + i] = -float("inf")
                want = torch.softmax(x, -1) @ V
                assert ((out[ends[b]:ends[b + 1], h].double().cpu() - want).abs() <= 0.02 * V.abs().max()).all()

    def shorten(budget, recent):
        kept, new = hstu_kv_select(weights, budget=budget, recent=recent, max_seqlen_k=max(lengths), **table())
        hstu_kv_compact(cache, kept, weights=weights, **table(), **kw)
        w = weights.cpu()
        for b in range(B):
            lengths[b] = min(lengths[b], budget)
            pages_left = -(-lengths[b] // ps)
            free.extend(owned[b][pages_left:])
            owned[b] = owned[b][:pages_left]
            for h in range(Nk):
                kept_rows[b][h] = [kept_rows[b][h][j] for j in kept[b, h].tolist() if j >= 0]
        for p in free:  # what a program does with pages that it uses again
            weights[p] = 0
        mine = table()
        assert all(torch.equal(new[k][:mine[k].numel()], mine[k]) for k in mine)
        assert torch.equal(w[mine["page_ids"].cpu()], weights[mine["page_ids"]].cpu())

    step([100, 37, 1])
    step([1, 1, 1])
    shorten(60, 8)
    step([1, 1, 1])
    step([40, 2, 70])
    shorten(50, 50)
    shorten(33, 0)
    step([1, 5, 1])


@pytest.mark.parametrize("mode,dtype,ps", [("same", "bf16", 32), ("scale", "bf16", 128), ("fp4", "fp16", 32), ("same", "fp32", 32),
                                           ("fp4", "bf16", 256)])
def test_weights_through_a_serving_loop(cuda_device, mode, dtype, ps):
    """What every key has received, from the step that appended it on, through shortened sequences and
    pages that are used again, against sums in 64 bits; nothing is cleared but by hstu_kv_append.

    Tolerance: each step's of the file's head, from the call's own lse, one 2^-24 of the sum per step."""
    dev, Nq, Nk, D, B, dt = cuda_device, 4, 2, 64, 3, R.DTYPES[dtype]
    g = torch.Generator().manual_seed(2)
    pages, alpha = 24 if ps < 256 else 8, 0.3
    if mode == "fp4":
        cache = torch.zeros(pages, 2, Nk, ps, D // 2, dtype=torch.uint8, device=dev)
        kw = dict(kv_scale=torch.zeros(pages, 2, Nk, ps, dtype=torch.uint8, device=dev),
                  kv_group_scale=torch.zeros(pages, 2, Nk, ps, D // 16, device=dev).to(R.FP8))
    else:
        cache = torch.zeros(pages, 2, ps, Nk, D, device=dev).to(dt if mode == "same" else R.FP8)
        kw = dict(kv_scale=torch.zeros(pages, 2, Nk, ps, dtype=torch.uint8, device=dev)) if mode == "scale" else {}
    weights = torch.full((pages, Nk, ps), 1e6, device=dev)  # what the pages' last users left
    free, owned, lengths = list(range(pages)), [[] for _ in range(B)], [0] * B
    keys = [np.zeros((0, Nk, D)) for _ in range(B)]   # as the cache holds them
    sums = [np.zeros((Nk, 0)) for _ in range(B)]
    tols = [np.zeros((Nk, 0)) for _ in range(B)]

    def table():
        return dict(page_offsets=R.offsets([len(o) for o in owned]).to(dev),
                    page_ids=torch.tensor([p for o in owned for p in o], device=dev),
                    last_page_len=torch.tensor([L - (len(o) - 1) * ps if o else 1 for L, o in zip(lengths, owned)], device=dev))

    def check():
        w = weights.cpu().numpy().astype(np.float64)
        for b in range(B):
            at = np.arange(lengths[b])
            got = w[np.array(owned[b], dtype=int)[at // ps], :, at % ps].T if lengths[b] else np.zeros((Nk, 0))
            bad = ~(np.abs(got - sums[b]) <= tols[b])
            assert not bad.any(), (b, np.argwhere(bad)[:5], got[bad][:5], sums[b][bad][:5])

    def step(n):
        for b in range(B):
            lengths[b] += n[b]
            while len(owned[b]) * ps < lengths[b]:
                owned[b].append(free.pop())
        q, k, v = (torch.randn(sum(n), h, D, generator=g).to(dt).to(dev) for h in (Nq, Nk, Nk))
        so, tab = R.offsets(n).to(dev), table()
        hstu_kv_append(k, v, so, cache, weights=weights, **tab, **kw)
        kr, _ = hstu_kv_read(cache, so, total_tokens=sum(n), dtype=dt if mode == "same" else torch.float32, **tab, **kw)
        bounds = dict(max_seqlen=max(n), max_seqlen_k=max(lengths), alpha=alpha)
        _, lse = hstu_softmax_fwd(q, cache, so, return_lse=True, **bounds, **tab, **kw)
        assert hstu_kv_weights(q, lse, cache, so, weights, **bounds, **tab, **kw) is weights
        ends = np.concatenate([[0], np.cumsum(n)])
        for b in range(B):
            at = slice(ends[b], ends[b + 1])
            keys[b] = np.concatenate([keys[b], R.values(kr[at].cpu())])
            pad = np.zeros((Nk, n[b]))
            w, size, off = E.key_weights(R.values(q[at].cpu()), lse[at].double().cpu().numpy(), keys[b], True, alpha)
            sums[b] = np.concatenate([sums[b], pad], 1) + w
            tols[b] = np.concatenate([tols[b], pad], 1) + 1.1 * (D + 16) * 2.0 ** -24 * size + 2.0 ** -22 * off + \
                (2.0 ** -21 + n[b] * (Nq // Nk) * 2.0 ** -24) * w + 2.0 ** -24 * sums[b] + 1e-30
        check()

    def shorten(budget, recent):
        kept, new = hstu_kv_select(weights, budget=budget, recent=recent, max_seqlen_k=max(lengths), **table())
        hstu_kv_compact(cache, kept, weights=weights, **table(), **kw)
        kept = kept.cpu().numpy()
        for b in range(B):
            lengths[b] = min(lengths[b], budget)
            left = -(-lengths[b] // ps)
            free.extend(owned[b][left:])
            owned[b] = owned[b][:left]
            rows = [kept[b, h, :lengths[b]] for h in range(Nk)]
            keys[b] = np.stack([keys[b][r, h] for h, r in enumerate(rows)], 1)
            sums[b] = np.stack([sums[b][h, r] for h, r in enumerate(rows)])
            tols[b] = np.stack([tols[b][h, r] for h, r in enumerate(rows)])
        assert new["page_offsets"].tolist() == table()["page_offsets"].tolist()
        check()

    step([100, 37, 1])
    step([1, 1, 1])
    shorten(60, 8)
    step([1, 1, 1])
    step([40, 2, 70])
    shorten(20, 5)  # (not whole pages)
    for _ in range(3):
        step([1, 3, 1])
    step([90, 1, 50])
    shorten(33, 0)
    step([1, 0, 1])


def test_append_clears_weights_of_the_rows_it_writes(cuda_device):
    """Those alone, of every cache form and both index types; not of sequences or pages that the device
    rejects, nor of rows of no sequence."""
    dev = cuda_device
    for dtype, mode, Nk, D, ps, index in (("bf16", "same", 3, 48, 32, torch.int32), ("fp16", "scale", 1, 256, 128, torch.int64),
                                          ("fp32", "cast", 2, 16, 256, torch.int64), ("bf16", "static", 4, 128, 32, torch.int32),
                                          ("bf16", "fp4", 5, 32, 32, torch.int64)):
        n = [1, 0, 40, 7, 130]
        t = R.Table([1, 50, 40, 90, 300], ps, index, seed=2)
        cache, _, kw = _cache(t, Nk, D, R.DTYPES[dtype], mode, dev, 3)
        k, v = (torch.randn(sum(n) + 2, Nk, D, device=dev).to(R.DTYPES[dtype]) for _ in range(2))
        w = torch.rand(t.num_pages, Nk, ps, device=dev) + 1
        want = w.clone()
        for b in range(len(n)):
            page, row = (torch.tensor(x[len(x) - n[b]:], device=dev) for x in t.rows(b))
            want[page, :, row] = 0
        untouched = cache.clone()
        hstu_kv_append(k, v, R.offsets(n, index).to(dev), untouched, **t.args(dev), **kw)
        hstu_kv_append(k, v, R.offsets(n, index).to(dev), cache, weights=w, **t.args(dev), **kw)
        assert torch.equal(w, want)
        assert torch.equal(cache.view(torch.uint8), untouched.view(torch.uint8))  # the rows are as without
        # (nothing of a sequence with a bad length, nor of a bad page)
        args = t.args(dev)
        args["last_page_len"][2] = 0
        args["page_ids"][-1] = -1
        w = torch.rand(t.num_pages, Nk, ps, device=dev) + 1
        want = w.clone()
        for b in (0, 3, 4):
            page, row = (torch.tensor(x[len(x) - n[b]:], device=dev) for x in t.rows(b))
            good = page != int(t.page_ids[-1])
            want[page[good], :, row[good]] = 0
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        hstu_kv_append(k, v, R.offsets(n, index).to(dev), cache, weights=w, status=status, **args, **kw)
        assert status.item() == 1 and torch.equal(w, want)
    for bad, error in ((w.half(), TypeError), (w[:1], ValueError), (w.cpu(), ValueError), (w.transpose(0, 2), ValueError)):
        with pytest.raises(error):
            hstu_kv_append(k, v, R.offsets(n, index).to(dev), cache, weights=bad, **t.args(dev), **kw)


def test_other_streams_and_captured_graphs(cuda_device):
    """The three calls on a stream of their own, two at once, and in a graph that is replayed."""
    dev = cuda_device
    t = R.Table([3000, 90, 700], 32)
    cache, _, _ = _cache(t, 2, 64, torch.bfloat16, "same", dev, 5)
    so, args = R.offsets([1, 1, 1]).to(dev), t.args(dev)
    q = torch.randn(3, 4, 64, device=dev, dtype=torch.bfloat16)
    lse = torch.full((3, 4), 6.0, device=dev)

    def work(cache, w):
        hstu_kv_weights(q, lse, cache, so, w, max_seqlen=1, max_seqlen_k=3000, alpha=0.1, **args)
        kept, new = hstu_kv_select(w, budget=500, recent=10, max_seqlen_k=3000, **args)
        hstu_kv_compact(cache, kept, weights=w, **args)
        return kept, new["page_ids"]

    states = [(cache.clone(), torch.rand(t.num_pages, 2, 32, device=dev)) for _ in range(4)]
    want = []
    for c, w in states:
        c, w = c.clone(), w.clone()
        want.append((*work(c, w), c, w))
    same = lambda x, y: torch.equal(x.nan_to_num(nan=3.0), y.nan_to_num(nan=3.0))  # noqa: E731
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for i in (0, 1):
        with torch.cuda.stream(streams[i]):
            c, w = (x.clone() for x in states[i])
            got.append((*work(c, w), c, w))
    torch.cuda.synchronize()
    for i in (0, 1):
        assert all(same(x.float(), y.float()) for x, y in zip(got[i], want[i]))
    c, w = (x.clone() for x in states[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept, ids = work(c, w)
    for i in (2, 3, 2):
        c.copy_(states[i][0])
        w.copy_(states[i][1])
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(x.float(), y.float()) for x, y in zip((kept, ids, c, w), want[i]))


@pytest.mark.parametrize("mode,dtype,pages", [("same", "bf16", 20000), ("fp4", "bf16", 70000), ("fp4", "fp32", 70000)])
def test_offsets_beyond_32_bits(cuda_device, mode, dtype, pages):
    """The last pages of a cache of more than 2^32 bytes (and 2^31 elements) do as the same pages of a
    small one."""
    dev, Nq, Nk, D, ps, dt = cuda_device, 8, 4, 128, 128, R.DTYPES[dtype]
    n = [1, 3, 130]
    t = R.Table([700, 90, 400], ps)
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(sum(n), h, D, generator=g).to(dt).to(dev) for h in (Nq, Nk, Nk))
    so = R.offsets(n).to(dev)
    small = K4._filled(t, Nk, D, dev, 5) if mode == "fp4" else S._filled(t, Nk, D, dt, mode, dev, 5)
    small = [small[0], *small[2].values(), torch.rand(t.num_pages, Nk, ps, device=dev)]

    def run(tensors, shift):
        cache, w = tensors[0], tensors[-1]
        kw = dict(zip(("kv_scale", "kv_group_scale"), tensors[1:-1]))
        args = t.args(dev)
        args["page_ids"] = args["page_ids"] + shift
        bounds = dict(max_seqlen=max(n), max_seqlen_k=max(t.lengths))
        hstu_kv_append(k, v, so, cache, **args, **kw)
        results = list(hstu_kv_read(cache, so, total_tokens=sum(n), dtype=dt, **args, **kw))
        out, lse = hstu_softmax_fwd(q, cache, so, alpha=0.1, return_lse=True, **bounds, **args, **kw)
        hstu_kv_weights(q, lse, cache, so, w, alpha=0.1, **bounds, **args, **kw)
        few = dict(max_seqlen=1, max_seqlen_k=max(t.lengths), alpha=0.1)
        one = torch.arange(4, device=dev)
        results += [out, lse, hstu_softmax_fwd(q[:3], cache, one, **few, **args, **kw)]
        hstu_kv_weights(q[:3], lse[:3], cache, one, w, **few, **args, **kw)
        kept, new = hstu_kv_select(w, budget=200, recent=9, max_seqlen_k=max(t.lengths), **args)
        hstu_kv_compact(cache, kept, weights=w, **args, **kw)
        used = torch.arange(t.num_pages, device=dev) + shift
        return [*results, kept, new["page_ids"] - shift * (new["page_ids"] >= 0)] + \
            [x[used].contiguous().view(torch.uint8) for x in tensors]

    shift = pages - t.num_pages
    large = []
    for x in small:
        y = torch.empty(pages, *x.shape[1:], dtype=x.dtype, device=dev)
        y[shift:] = x
        large.append(y)
    for x, y in zip(run(small, 0), run(large, shift)):
        assert torch.equal(x, y)


def test_empty_calls(cuda_device):
    dev = cuda_device
    w = torch.rand(4, 2, 32, device=dev)
    none = dict(page_offsets=torch.zeros(1, dtype=torch.int64, device=dev), page_ids=torch.zeros(0, dtype=torch.int64, device=dev),
                last_page_len=torch.zeros(0, dtype=torch.int64, device=dev))
    kept, new = hstu_kv_select(w, budget=3, max_seqlen_k=9, **none)
    assert kept.shape == (0, 2, 3) and new["page_offsets"].tolist() == [0]
    cache = torch.zeros(4, 2, 32, 2, 64, device=dev)
    assert hstu_kv_compact(cache, kept, **none) is cache
    t = R.Table([0, 0], 32)  # sequences without rows
    kept, new = hstu_kv_select(torch.rand(t.num_pages, 2, 32, device=dev), budget=3, max_seqlen_k=9, **t.args(dev))
    assert (kept == -1).all() and new["page_offsets"].tolist() == [0, 0, 0]
    hstu_kv_compact(torch.zeros(t.num_pages, 2, 32, 2, 64, device=dev), kept, **t.args(dev))


def test_refusals(cuda_device):
    dev = cuda_device
    t = R.Table([40, 10], 32)
    cache, _, _ = _cache(t, 2, 64, torch.bfloat16, "same", dev, 5)
    so, args = R.offsets([1, 1]).to(dev), t.args(dev)
    q, lse = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev), torch.zeros(2, 4, device=dev)
    w = torch.zeros(t.num_pages, 2, 32, device=dev)
    kw = dict(max_seqlen=1, max_seqlen_k=64, **args)
    hstu_kv_weights(q, lse, cache, so, w, **kw)
    for bad, error in ((dict(lse=lse.double()), TypeError), (dict(lse=lse[:1]), ValueError), (dict(lse=lse.cpu()), ValueError),
                       (dict(weights=w[:, :1]), ValueError), (dict(weights=w.half()), TypeError),
                       (dict(weights=w.transpose(1, 2)), ValueError), (dict(q=q.float()), TypeError),
                       (dict(q=q[:, :3]), ValueError), (dict(q=q[..., :32]), ValueError), (dict(q=None), TypeError),
                       (dict(lse=None), TypeError), (dict(max_seqlen=0), HstuError), (dict(alpha=-1.0), HstuError),
                       (dict(max_seqlen_k=1 << 40), HstuError)):
        a = {**dict(q=q, lse=lse, weights=w), **bad}
        with pytest.raises(error):
            hstu_kv_weights(a.pop("q"), a.pop("lse"), cache, so, a.pop("weights"), **{**kw, **a})
    for bad, error in ((dict(budget=0), ValueError), (dict(budget=1 << 31), ValueError), (dict(recent=-1), ValueError),
                       (dict(max_seqlen_k=0), ValueError), (dict(weights=w[0]), ValueError), (dict(weights=w.half()), TypeError),
                       (dict(weights=w.cpu()), ValueError), (dict(page_ids=args["page_ids"].int()), TypeError),
                       (dict(last_page_len=args["last_page_len"][:1]), ValueError), (dict(page_offsets=None), TypeError),
                       (dict(page_ids=args["page_ids"].cpu()), ValueError)):
        a = {**dict(weights=w, budget=8, max_seqlen_k=64, **args), **bad}
        with pytest.raises(error):
            hstu_kv_select(a.pop("weights"), **a)
    kept, _ = hstu_kv_select(w, budget=8, max_seqlen_k=64, **args)
    for bad, error in ((dict(kept=kept.long()), TypeError), (dict(kept=kept[:1]), ValueError), (dict(kept=kept[:, :1]), ValueError),
                       (dict(kept=kept.cpu()), ValueError), (dict(weights=w[:1]), ValueError), (dict(max_seqlen_k=0), ValueError),
                       (dict(kv_group_scale=w), ValueError), (dict(kept=None), ValueError)):
        a = {**dict(kept=kept, **args), **bad}
        with pytest.raises(error):
            hstu_kv_compact(cache, a.pop("kept"), **a)
