"""Paged KV caches of 4-bit codes: hstu_kv_append and hstu_kv_read against a plain 64-bit
implementation (exactly: quantisation has one result), and hstu_softmax_fwd over such caches with
the tolerance of test_gpu_softmax.py. Codes times factors are exact in fp16, so a 4-bit cache changes
that tolerance no more than an E4M3 one: weights of bf16 queries are bf16 or fp16 there (see
include/hstu_kv.h), whose half step is smaller."""
import numpy as np
import pytest
import torch

import kv4_reference as R4
import kv_reference as R
import test_gpu_softmax as S
from hstu_dense_forward_gb300 import HstuError, hstu_kv_append, hstu_kv_read, hstu_softmax_fwd

pytestmark = pytest.mark.gpu


def _empty(t, Nk, D, dev, seed=9):
    """A cache with something in every byte."""
    g = torch.Generator().manual_seed(seed)
    shape = (t.num_pages, 2, Nk, t.page_size)
    return (torch.randint(0, 256, (*shape, D // 2), generator=g, dtype=torch.uint8).to(dev),
            torch.rand(*shape, D // 16, generator=g).to(R.FP8).to(dev),
            torch.randint(100, 140, shape, generator=g, dtype=torch.uint8).to(dev))


def _expected(before, t, n, k, v):
    """Values after appending, and bytes of what must stay."""
    vals = R4.values(*(x.cpu() for x in before))
    so = np.concatenate([[0], np.cumsum(n)])
    for b in range(len(n)):
        page, row = t.rows(b)
        page, row = page[len(page) - n[b]:], row[len(row) - n[b]:]
        for plane, x in ((0, k), (1, v)):
            code, factor, e = R4.quantise(R.values(x[so[b]:so[b + 1]].cpu()))
            y = (R4.E2M1[code].reshape(*factor.shape, 16) * factor[..., None]).reshape(code.shape)
            vals[page, plane, row] = np.ldexp(y, e[..., None])
    return vals


def _rows(T, Nk, D, dtype, seed, dev, strided):
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, 3 * Nk, D, generator=g) * torch.exp2(torch.randn(T, 3 * Nk, 1, generator=g) * 3)
    wide *= torch.exp2(torch.randn(T, 3 * Nk, D // 16, generator=g) * 2).repeat_interleave(16, -1)
    wide = wide.to(dtype).to(dev)
    k, v = wide[:, Nk:2 * Nk], wide[:, 2 * Nk:]
    return (k, v) if strided else (k.contiguous(), v.contiguous())


CASES = [  # dtype, D, Nk, page size, index type, strided
    ("bf16", 128, 4, 128, torch.int64, True), ("fp16", 64, 3, 32, torch.int32, True),
    ("fp32", 256, 2, 256, torch.int64, False), ("bf16", 32, 5, 32, torch.int32, False),
    ("fp16", 96, 1, 128, torch.int64, False), ("fp32", 160, 7, 32, torch.int64, True),
    ("bf16", 224, 2, 256, torch.int32, False),
]


@pytest.mark.parametrize("dtype,D,Nk,ps,index,strided", CASES)
def test_append_and_read(cuda_device, dtype, D, Nk, ps, index, strided):
    dev, dt = cuda_device, R.DTYPES[dtype]
    lengths, n = [1, 0, ps, ps + 1, 3 * ps - 1, 77, 2], [1, 0, ps, 5, 2 * ps, 0, 2]
    t = R.Table(lengths, ps, index, seed=1)
    k, v = _rows(sum(n) + 2, Nk, D, dt, 2, dev, strided)  # two rows of no sequence
    cache, group, scale = before = _empty(t, Nk, D, dev)
    want = _expected(before, t, n, k, v)
    kw = dict(t.args(dev), kv_scale=scale, kv_group_scale=group)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    assert hstu_kv_append(k, v, R.offsets(n, index).to(dev), cache, status=status, **kw) is cache
    every = R4.values(cache.cpu(), group.cpu(), scale.cpu())
    assert np.array_equal(every, want)
    as_fp4 = cache.view(torch.float4_e2m1fn_x2) if hasattr(torch, "float4_e2m1fn_x2") else cache
    for m, c, out_dt in ((n, cache, dt), (lengths, as_fp4, torch.float32), (lengths, cache, torch.bfloat16)):
        so = np.concatenate([[0], np.cumsum(m)])
        got = hstu_kv_read(c, R.offsets(m, index).to(dev), total_tokens=sum(m), dtype=out_dt,
                           status=status, **kw)
        for plane, x in enumerate(got):
            for b in range(len(m)):
                page, row = t.rows(b)
                y = torch.tensor(every[page, plane, row][len(page) - m[b]:]).to(out_dt)
                assert torch.equal(x[so[b]:so[b + 1]].cpu(), y)
    assert hstu_kv_read(cache, R.offsets(n, index).to(dev), total_tokens=sum(n), **kw)[0].dtype == torch.bfloat16
    assert status.item() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantisation_at_its_edges(cuda_device, dtype):
    """Middles of two codes and their neighbours for every factor, rows of zeros, of the largest and
    smallest values, factors that round to 0, infinities and NaN."""
    dev, dt = cuda_device, R.DTYPES[dtype]
    rows = []
    # groups whose factor is f: largest 6 f; the others around the middles of the codes
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    for f in [1.0, 1.125, 1.25, 1.375, 1.5, 1.625, 1.75, 1.875, 2.0, 448.0 / 1024, 2.0 ** -9]:
        x = torch.tensor(np.concatenate([mids * f, -mids * f, [6 * f, 0.0]]), dtype=torch.float64).to(dt)
        for step in (0, 1, -1):  # the neighbour of the next larger, smaller magnitude
            y = (x.view(torch.int32 if dtype == "fp32" else torch.int16) + step).view(dt).clone()
            y[14], y[15] = 6 * f, 0
            rows.append(torch.cat([y, torch.tensor([2688.0] + [0.0] * 15, dtype=dt)]))
    big, small = torch.finfo(dt).max, torch.finfo(dt).tiny
    nan, inf = float("nan"), float("inf")
    for first, second in (([0.0], [0.0]), ([big], [1.0]), ([small], [small, -small / 2]), ([-0.0], [0.0]),
                          ([inf, 1.0], [2.0]), ([-inf, inf], [0.0]), ([nan, 1.0], [3.0, -1.0]),
                          ([2688.0], [2.6, 1.3]), ([2689.0], [-1.0]), ([1e-3], [1000.0]), ([big], [-inf])):
        row = torch.zeros(32, dtype=dt)
        row[:len(first)] = torch.tensor(first, dtype=torch.float64).to(dt)
        row[16:16 + len(second)] = torch.tensor(second, dtype=torch.float64).to(dt)
        rows.append(row)
    g = torch.Generator().manual_seed(3)
    rows += list((torch.randint(-448, 449, (500, 32), generator=g) / 8.0).to(dt))  # many ties
    x = torch.stack(rows)[:, None].to(dev)  # [T, 1, 32]
    T = x.shape[0]
    t = R.Table([T], 256)
    cache, group, scale = before = _empty(t, 1, 32, dev)
    with np.errstate(invalid="ignore"):
        want = _expected(before, t, [T], x, -x)
    kw = dict(t.args(dev), kv_scale=scale, kv_group_scale=group)
    hstu_kv_append(x, -x, R.offsets([T]).to(dev), cache, **kw)
    got = R4.values(cache.cpu(), group.cpu(), scale.cpu())
    assert np.array_equal(got, want, equal_nan=True)
    k, _ = hstu_kv_read(cache, R.offsets([T]).to(dev), total_tokens=T, dtype=torch.float32, **kw)
    page, row = t.rows(0)
    with np.errstate(over="ignore", invalid="ignore"):
        y = torch.tensor(want[page, 0, row]).float()
    assert torch.equal(k.cpu().nan_to_num(nan=1e33), y.nan_to_num(nan=1e33))


def _filled(t, Nk, D, dev, seed, sigma=1.0, spread=0.7):
    """A cache whose sequences hold random rows and whose other rows hold NaN factors and scales of
    255, with the values it stands for."""
    g = torch.Generator().manual_seed(seed)
    shape = (t.num_pages, 2, Nk, t.page_size, D)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randn(*shape[:-1], 1, generator=g) * spread) * sigma
    used = torch.zeros(t.num_pages, t.page_size, dtype=torch.bool)
    for b in range(len(t.lengths)):
        page, row = t.rows(b)
        used[torch.tensor(page), torch.tensor(row)] = True
    mask = used[:, None, None, :]
    cache, group, scale = R4.tensors(*R4.quantise(x.numpy().astype(np.float64)))
    vals = np.where(mask.swapaxes(2, 3)[..., None], R4.values(cache, group, scale), 0.0)
    group = torch.where(mask[..., None], group.float(), torch.nan).to(R.FP8)
    scale = torch.where(mask, scale, torch.tensor(255, dtype=torch.uint8))
    return cache.to(dev), vals, dict(kv_scale=scale.contiguous().to(dev), kv_group_scale=group.contiguous().to(dev))


def run_case(dev, lengths, n, dtype, Nq, Nk, D, ps, causal=True, index=torch.int64, strided=False,
             seed=0, tail=2, sigma=1.0, spread=0.7, bounds=None):
    dt = R.DTYPES[dtype]
    t = R.Table(lengths, ps, index, seed=seed)
    cache, vals, kw = _filled(t, Nk, D, dev, seed + 1, sigma, spread)
    g = torch.Generator().manual_seed(seed + 2)
    wide = torch.randn(sum(n) + tail, Nq + 3, D, generator=g).to(dt).to(dev)
    q = wide[:, 2:2 + Nq] if strided else wide[:, 2:2 + Nq].contiguous()
    out = torch.full((sum(n) + tail, Nq, D), 77.0, dtype=dt, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sq, sk = bounds or (max(1, max(n)), max(1, max(lengths)))
    _, lse = hstu_softmax_fwd(q, cache, R.offsets(n, index).to(dev), max_seqlen=sq, max_seqlen_k=sk,
                              causal=causal, alpha=D ** -0.5, out=out, return_lse=True, status=status,
                              **t.args(dev), **kw)
    assert status.item() == 0
    assert (out[len(out) - tail:] == 77.0).all()  # rows of no sequence
    S.check(t, n, q, vals, out, lse, causal, D ** -0.5, dt)


@pytest.mark.parametrize("dtype,Nq,Nk,D,ps,index", [
    ("bf16", 8, 2, 128, 128, torch.int64), ("fp16", 4, 4, 64, 32, torch.int32), ("bf16", 16, 1, 256, 256, torch.int64),
    ("fp16", 5, 1, 96, 256, torch.int32), ("bf16", 3, 3, 32, 32, torch.int64), ("fp16", 12, 4, 160, 128, torch.int64),
    ("bf16", 16, 4, 224, 32, torch.int32), ("fp32", 8, 2, 64, 32, torch.int64), ("fp32", 4, 1, 128, 128, torch.int32),
    ("fp32", 6, 2, 224, 32, torch.int64), ("bf16", 16, 1, 128, 32, torch.int64), ("fp16", 11, 1, 64, 128, torch.int64),
])
def test_single_tokens(cuda_device, dtype, Nq, Nk, D, ps, index):
    run_case(cuda_device, S.TOKENS, [1] * len(S.TOKENS), dtype, Nq, Nk, D, ps, index=index, seed=11)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Nq,Nk,D,ps,strided", [
    ("bf16", 8, 2, 128, 128, True), ("fp16", 3, 1, 64, 32, False), ("bf16", 4, 4, 96, 32, False),
    ("fp16", 2, 2, 256, 32, True), ("bf16", 7, 1, 224, 256, False), ("fp32", 4, 2, 64, 128, True),
    ("fp32", 2, 1, 160, 32, False), ("fp16", 5, 1, 32, 128, False),
])
def test_chunks(cuda_device, dtype, Nq, Nk, D, ps, strided, causal):
    run_case(cuda_device, *S.CHUNK, dtype, Nq, Nk, D, ps, causal=causal, seed=21, strided=strided)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,Nq,Nk,D,ps", [
    ("bf16", 8, 2, 128, 128), ("fp16", 6, 2, 64, 32), ("bf16", 3, 1, 32, 256), ("fp16", 4, 1, 192, 128),
    ("bf16", 4, 1, 96, 32)])
def test_prompts(cuda_device, dtype, Nq, Nk, D, ps, causal):
    run_case(cuda_device, *S.PROMPT, dtype, Nq, Nk, D, ps, causal=causal, seed=71)


# prompts of bf16 queries of 768 rows of a kv head in the mean and more, over pages turned into bf16
LONG = ([300, 1000, 70, 700, 40, 0], [300, 999, 70, 331, 0, 0])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Nq,Nk,D,ps,index", [(8, 2, 128, 128, torch.int64), (6, 2, 64, 32, torch.int32), (5, 1, 32, 256, torch.int64),
                                              (12, 3, 192, 128, torch.int32), (16, 4, 96, 32, torch.int64)])
def test_long_prompts(cuda_device, Nq, Nk, D, ps, index, causal):
    run_case(cuda_device, *LONG, "bf16", Nq, Nk, D, ps, causal=causal, index=index, seed=81, strided=Nk == 2)


def test_long_prompts_over_bad_pages(cuda_device):
    """Page ids outside the cache, in a sequence and behind the last: the others' outputs are right,
    and only ids that a sequence has are told."""
    dev = cuda_device
    t = R.Table([600, 600, 600], 128)
    n = [600, 600, 600]
    cache, vals, kw = _filled(t, 1, 64, dev, 5)
    q = torch.randn(1800, 4, 64, device=dev).to(torch.bfloat16)
    args = {**t.args(dev), **kw}
    args["page_ids"] = torch.cat([args["page_ids"], torch.tensor([-1, 1 << 40, -7], device=dev)])
    for bad in (False, True):
        if bad:
            args["page_ids"][7] = t.num_pages
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out, lse = hstu_softmax_fwd(q, cache, R.offsets(n).to(dev), max_seqlen=600, max_seqlen_k=600, alpha=0.125,
                                    return_lse=True, status=status, **args)
        assert status.item() == bad
        for b in (0, 2) if bad else (0, 1, 2):
            one = R.Table([600], 128)
            one.page_offsets, one.page_ids = torch.tensor([0, 5]), t.page_ids[5 * b:5 * b + 5]
            at = slice(600 * b, 600 * b + 600)
            S.check(one, [600], q[at], vals, out[at], lse[at], True, 0.125, torch.bfloat16)


def _check_weights_of(half_step, t, n, q, vals, got, alpha):
    """The tolerance of test_gpu_softmax.py with weights of this half step (u_p). fp16 weights stand
    beside the largest weight times its row's scale: 2^-25 of that times a row's codes, 2688 at most
    where the row of the largest has 1344, is 2^-24 max |v| a key."""
    so = np.concatenate([[0], np.cumsum(n)])
    for b in range(len(n)):
        page, row = t.rows(b)
        K, V = vals[page, 0, row], vals[page, 1, row]
        out, _, A, size = R.softmax_rows(R.values(q[so[b]:so[b + 1]].cpu()), K, V, True, alpha)
        ex, Lk = (out.shape[2] + 8) * 2.0 ** -24 * size, K.shape[0]
        tol = 2.0 ** -8 * np.abs(out) + (half_step + 2.0 ** -20 + Lk * 2.0 ** -24 + 2 * ex[..., None]) * A * 1.01
        tol = tol + Lk * 2.0 ** -24 * np.abs(V).max(initial=0) + 1e-30
        bad = ~(np.abs(got[so[b]:so[b + 1]].double().cpu().numpy() - out) <= tol)
        assert not bad.any(), (b, np.argwhere(bad)[:5])


@pytest.mark.parametrize("index", [torch.int32, torch.int64])
@pytest.mark.parametrize("lengths,n,Nq,Nk,D,ps", [([600, 0, 900, 300], [600, 0, 850, 0], 4, 1, 64, 128),
                                                 ([1000, 30], [1000, 1], 8, 2, 96, 32), ([900, 700], [880, 700], 6, 1, 160, 128)])
def test_pages_as_bf16_or_not(cuda_device, lengths, n, Nq, Nk, D, ps, index):
    """The choice does not look at entries of page_ids that no sequence has, of which there may be more
    than pages that fit the workspace; and a caller that declines it gets fp16 weights."""
    dev, alpha = cuda_device, D ** -0.5
    t = R.Table(lengths, ps, index, seed=4)
    cache, vals, kw = _filled(t, Nk, D, dev, 5)
    q = torch.randn(sum(n), Nq, D, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16).to(dev)
    args = dict(max_seqlen=max(n), max_seqlen_k=max(lengths), alpha=alpha, return_lse=True, **kw)
    table, so = t.args(dev), R.offsets(n, index).to(dev)
    page = 4 * ps * Nk * D
    more = torch.randint(-2, t.num_pages + 2, ((1 << 30) // page + 100,), device=dev).to(index)
    results = []
    for extra in (more[:0], more[:1], more):
        for expand in (True, False):
            status = torch.zeros(1, dtype=torch.int32, device=dev)
            ids = torch.cat([table["page_ids"], extra])
            out, lse = hstu_softmax_fwd(q, cache, so, expand=expand, status=status, **{**table, "page_ids": ids}, **args)
            assert status.item() == 0
            _check_weights_of(2.0 ** -8 if expand else 2.0 ** -11, t, n, q, vals, out, alpha)
            results.append((out, lse))
    for i in (2, 4):
        for j in (0, 1):
            assert all(torch.equal(x, y) for x, y in zip(results[i + j], results[j]))
    assert not torch.equal(results[0][0], results[1][0])


def test_pages_as_bf16_of_sequences_that_share_entries(cuda_device):
    """Of tables with more entries than pages that sequences can have, too; an invalid sequence between."""
    dev, D, ps = cuda_device, 64, 32
    t = R.Table([30 * ps], ps, seed=4)
    cache, vals, kw = _filled(t, 1, D, dev, 5)
    q = torch.randn(1600, 8, D, device=dev).to(torch.bfloat16)
    so = torch.tensor([0, 800, 800, 1600], device=dev)
    for extra in (0, 200):
        table = dict(page_offsets=torch.tensor([0, 25, 5, 30], device=dev),
                     page_ids=torch.cat([t.page_ids, torch.zeros(extra, dtype=torch.int64)]).to(dev),
                     last_page_len=torch.tensor([ps, ps, ps], device=dev))
        status = torch.zeros(1, dtype=torch.int32, device=dev)
        out = hstu_softmax_fwd(q, cache, so, max_seqlen=800, max_seqlen_k=25 * ps, alpha=0.125, status=status, **table, **kw)
        assert status.item() == 1  # (offsets decrease)
        for first, at in ((0, 0), (5, 800)):
            one = R.Table([800], ps)
            one.page_offsets, one.page_ids = torch.tensor([0, 25]), t.page_ids[first:first + 25]
            _check_weights_of(2.0 ** -8, one, [800], q[at:at + 800], vals, out[at:at + 800], 0.125)


@pytest.mark.parametrize("dtype,B,Nk,D", [("bf16", 1, 1, 64), ("fp16", 4, 2, 32), ("bf16", 4, 4, 32), ("fp16", 25, 1, 64),
                                          ("bf16", 7, 4, 32), ("bf16", 9, 4, 32), ("bf16", 3, 2, 256)])
def test_single_tokens_over_long_keys(cuda_device, dtype, B, Nk, D):
    """As many items as clusters of eight, clusters of two and single CTAs divide the keys of."""
    lengths = [40000, 100] + [2000 + 37 * b for b in range(B)]
    run_case(cuda_device, lengths[:B], [1] * B, dtype, 2 * Nk, Nk, D, 128, seed=61, bounds=(1, 40000))


@pytest.mark.parametrize("dtype,n,D", [("bf16", 300, 128), ("fp16", 200, 64), ("bf16", 30, 256), ("fp16", 6, 64),
                                       ("bf16", 3, 128), ("fp32", 3, 128)])
def test_items_over_many_ctas(cuda_device, dtype, n, D):
    run_case(cuda_device, [7000, 3, 0, 600], [n, 3, 0, n // 3], dtype, 4, 2, D, 128, seed=101)


@pytest.mark.parametrize("dtype,n,Nq,D", [("bf16", 1, 8, 128), ("fp16", 40, 4, 64), ("bf16", 300, 4, 128), ("fp16", 70, 4, 256)])
def test_rows_of_very_unlike_scales(cuda_device, dtype, n, Nq, D):
    """Row scales spread over 2^60 and more: rows keep exponents of their own."""
    run_case(cuda_device, [700, 300, 65], [n, min(n, 300), min(n, 65)], dtype, Nq, 2, D, 128, seed=31,
             sigma=0.01, spread=2.5)


def test_more_queries_than_keys(cuda_device):
    for causal in (True, False):
        run_case(cuda_device, [3, 0, 40, 129], [10, 4, 41, 300], "bf16", 4, 2, 64, 32, causal=causal, seed=41)
        run_case(cuda_device, [3, 0, 7], [5, 1, 8], "fp16", 2, 1, 128, 32, causal=causal, seed=42)


def test_loose_bounds_captured_and_replayed(cuda_device):
    """One graph of append and attention, replayed over caches that change in between; equal to
    calls that are not captured."""
    dev = cuda_device
    t = R.Table([130, 64, 257], 32)
    n = [1, 2, 1]
    cache, _, kw = _filled(t, 2, 128, dev, 5)
    g = torch.Generator().manual_seed(6)
    q, k, v = (torch.randn(4, h, 128, generator=g).to(torch.bfloat16).to(dev) for h in (8, 2, 2))
    so, args = R.offsets(n).to(dev), dict(t.args(dev), **kw)

    def step():
        hstu_kv_append(k, v, so, cache, **args)
        return hstu_softmax_fwd(q, cache, so, max_seqlen=16, max_seqlen_k=5000, alpha=0.1, **args)

    eager = step().clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = step()
    for i in range(3):
        q.normal_()
        k.normal_()
        graph.replay()
        got = out.clone()
        assert torch.equal(got, step())
    assert not torch.equal(got, eager)


def test_refusals(cuda_device):
    dev = cuda_device
    t = R.Table([40, 10], 32)
    cache, group, scale = _empty(t, 2, 64, dev)
    so = R.offsets([1, 1]).to(dev)
    k = torch.zeros(2, 2, 64, device=dev, dtype=torch.bfloat16)
    kw = dict(t.args(dev), kv_scale=scale, kv_group_scale=group)
    hstu_kv_append(k, k, so, cache, **kw)
    for change, error in ((dict(kv_group_scale=None), ValueError), (dict(kv_scale=None), ValueError),
                          (dict(kv_group_scale=group.float()), TypeError),
                          (dict(kv_group_scale=group[:, :, :, :, :2].contiguous()), ValueError),
                          (dict(kv_group_scale=group.cpu()), ValueError),
                          (dict(kv_scale=scale[1:]), ValueError),
                          (dict(k_descale=1.0, v_descale=1.0), ValueError)):
        with pytest.raises(error):
            hstu_kv_append(k, k, so, cache, **{**kw, **change})
        with pytest.raises(error):
            hstu_softmax_fwd(k, cache, so, max_seqlen=1, max_seqlen_k=64, **{**kw, **change})
    with pytest.raises(ValueError):  # head dim 48
        hstu_kv_append(k[..., :48].contiguous(), k[..., :48].contiguous(), so, cache[..., :24].contiguous(),
                       **{**kw, "kv_group_scale": group[..., :3].contiguous()})
    with pytest.raises(ValueError):  # group factors with another form
        hstu_kv_append(k, k, so, torch.zeros(t.num_pages, 2, 32, 2, 64, device=dev, dtype=torch.bfloat16),
                       **t.args(dev), kv_group_scale=group)
    with pytest.raises(ValueError):  # rows of another head dim
        hstu_kv_append(k[..., :32].contiguous(), k[..., :32].contiguous(), so, cache, **kw)
    bad = torch.zeros(1, dtype=torch.int32, device=dev)
    ids = kw["page_ids"].clone()
    ids[0] = t.num_pages
    hstu_kv_append(k, k, so, cache, status=bad, **{**kw, "page_ids": ids, "last_page_len": kw["last_page_len"] + 100})
    assert bad.item() == 1
