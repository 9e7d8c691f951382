"""hstu_kv_append and hstu_kv_read against plain 64-bit implementations: every cache type and
quantisation, head dims, page sizes and index types, rows that are slices of a wider tensor,
ragged and empty sequences, values where quantisation can go wrong, what must stay untouched,
tables that the device must reject, and the round trip into hstu_fwd."""
import numpy as np
import pytest
import torch

import kv_reference as R
import oracle
from hstu_dense_forward_gb300 import hstu_fwd, hstu_kv_append, hstu_kv_read

pytestmark = pytest.mark.gpu


def _rows(T, Nk, D, dtype, seed, dev, strided=False):
    """k, v [T, Nk, D] with rows of unlike sizes; strided: slices of [T, 3 Nk, D]."""
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(T, 3 * Nk, D, generator=g) * torch.exp2(torch.randn(T, 3 * Nk, 1, generator=g))
    wide = wide.to(dtype).to(dev)
    k, v = wide[:, Nk:2 * Nk], wide[:, 2 * Nk:]
    return (k, v) if strided else (k.contiguous(), v.contiguous())


def _empty_cache(t, Nk, D, dtype, fp8, dev, seed=9):
    g = torch.Generator().manual_seed(seed)
    cache = torch.randn(t.num_pages, 2, t.page_size, Nk, D, generator=g)
    cache = cache.to(R.FP8 if fp8 else dtype).to(dev)
    scale = torch.randint(100, 140, (t.num_pages, 2, Nk, t.page_size), generator=g,
                          dtype=torch.uint8).to(dev)
    return cache, scale


def _expected(before, scale, t, n, k, v, mode, kd=None, vd=None):
    """The cache's (and scales') values after appending."""
    cache, sc = R.values(before.cpu()), scale.cpu().numpy().copy()
    so = np.concatenate([[0], np.cumsum(n)])
    for b in range(len(n)):
        page, row = t.rows(b)
        page, row = page[len(page) - n[b]:], row[len(row) - n[b]:]
        for plane, x, f in ((0, k, kd), (1, v, vd)):
            y = R.values(x[so[b]:so[b + 1]].cpu())
            if mode == "scale":
                e = R.row_exponent(y)
                sc[page, plane, :, row] = e + 127
                y = R.e4m3_round(np.ldexp(y, -e[..., None]))
            elif mode == "static":
                y32 = y.astype(np.float32) / f[b].astype(np.float32)[None, :, None]
                y = R.e4m3_round(y32)
            elif mode == "cast":
                y = R.e4m3_round(y)
            cache[page, plane, row] = y
    return cache, sc


CASES = [  # dtype, mode, D, Nk, page size, index type, strided
    ("bf16", "copy", 128, 4, 128, torch.int64, False),
    ("bf16", "scale", 128, 4, 128, torch.int64, True),
    ("fp16", "scale", 64, 3, 32, torch.int32, True),
    ("fp32", "scale", 256, 2, 256, torch.int64, False),
    ("bf16", "cast", 48, 5, 32, torch.int32, False),
    ("fp16", "static", 128, 2, 128, torch.int64, True),
    ("fp32", "static", 16, 7, 32, torch.int64, True),
    ("fp32", "copy", 80, 1, 256, torch.int32, True),
    ("fp16", "copy", 240, 2, 32, torch.int32, False),
    ("bf16", "scale", 208, 1, 32, torch.int64, True),
]


@pytest.mark.parametrize("dtype,mode,D,Nk,ps,index,strided", CASES)
def test_append_and_read(cuda_device, dtype, mode, D, Nk, ps, index, strided):
    dev, dt = cuda_device, R.DTYPES[dtype]
    lengths = [1, 0, ps, ps + 1, 3 * ps - 1, 77, 2]
    n = [1, 0, ps, 5, 2 * ps, 0, 2]
    t = R.Table(lengths, ps, index, seed=1)
    k, v = _rows(sum(n) + 2, Nk, D, dt, 2, dev, strided)  # two rows of no sequence
    cache, scale = _empty_cache(t, Nk, D, dt, mode != "copy", dev)
    kw = dict(t.args(dev))
    kd = vd = None
    if mode == "scale":
        kw["kv_scale"] = scale
    if mode == "static":
        g = np.random.default_rng(3)
        kd, vd = (np.exp2(g.uniform(-9, -4, (len(n), Nk))).astype(np.float32) for _ in range(2))
        kw.update(k_descale=torch.tensor(kd, device=dev), v_descale=torch.tensor(vd, device=dev))
    want, want_scale = _expected(cache, scale, t, n, k, v, mode, kd, vd)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    so = R.offsets(n, index).to(dev)
    assert hstu_kv_append(k, v, so, cache, status=status, **kw) is cache
    assert status.item() == 0
    assert np.array_equal(R.values(cache.cpu()), want)  # quantisation is exact; the rest untouched
    assert np.array_equal(scale.cpu().numpy(), want_scale)
    # read back: the new rows, then every row, into all types the cache gives
    every = R.cache_values(cache.cpu(), scale.cpu() if mode == "scale" else None)
    for m, out_dt in ((n, dt), (lengths, torch.bfloat16 if mode != "copy" else dt)):
        so = np.concatenate([[0], np.cumsum(m)])
        got = hstu_kv_read(cache, R.offsets(m, index).to(dev), total_tokens=sum(m), dtype=out_dt,
                           status=status, **kw)
        for plane, x, f in ((0, got[0], kd), (1, got[1], vd)):
            assert x.shape == (sum(m), Nk, D) and x.dtype == out_dt
            for b in range(len(m)):
                page, row = t.rows(b)
                y = every[page, plane, row][len(page) - m[b]:]
                if f is not None:
                    y = y.astype(np.float32) * f[b][None, :, None]
                y = torch.tensor(y).float().to(out_dt)  # exact in fp32; one rounding
                assert torch.equal(x[so[b]:so[b + 1]].cpu(), y)
    assert status.item() == 0


def test_quantised_values_at_the_edges(cuda_device):
    """Row scales: zeros, one value at and just above 448 * 2^e, the smallest exponent, subnormals,
    infinities and NaN beside finite values; every tie of the E4M3 grid."""
    dev, D = cuda_device, 32
    rows = np.zeros((9, D), dtype=np.float32)
    rows[1, 3] = 448.0
    rows[2, 3] = np.nextafter(np.float32(448.0), np.float32(1e9))
    rows[3, :] = 2.0 ** -120
    rows[4, 0], rows[4, 1] = 1.0, 2.0 ** -140
    rows[5, :3] = [np.inf, -np.inf, 3.0]
    rows[6, :3] = [np.nan, 5.0, -7.0]
    rows[7, 0], rows[7, 1] = 3.0e38, -1.0
    rows[8, :] = 1.0 + np.arange(D) / 32.0  # between 1 and 2: ties at odd sixteenths
    x = torch.tensor(rows)[:, None, :].to(dev)
    t = R.Table([9], 32)
    cache, scale = _empty_cache(t, 1, D, torch.float32, True, dev)
    hstu_kv_append(x, x, R.offsets([9]).to(dev), cache, kv_scale=scale, **t.args(dev))
    page, row = t.rows(0)
    e = scale.cpu().numpy()[page, 0, 0, row].astype(int) - 127
    assert list(e) == list(R.row_exponent(rows.astype(np.float64)))
    assert e[0] == -100 and e[1] == 0 and e[2] == 1 and e[3] == -100 and e[7] == 120
    got = R.values(cache.cpu())[page, 0, row, 0]
    want = R.e4m3_round(np.ldexp(rows.astype(np.float64), -e[:, None]))
    assert np.array_equal(got, want, equal_nan=True)
    assert got[5, 0] == 448 and got[5, 1] == -448 and np.isnan(got[6, 0])
    k, v = hstu_kv_read(cache, R.offsets([9]).to(dev), total_tokens=9, dtype=torch.float32,
                        kv_scale=scale, **t.args(dev))
    assert torch.equal(k, v) or torch.isnan(k).any()
    assert np.array_equal(k[:, 0].cpu().numpy().astype(np.float64), np.ldexp(want, e[:, None]),
                          equal_nan=True)


def test_scalar_and_per_sequence_factors(cuda_device):
    dev = cuda_device
    t = R.Table([5, 40], 32)
    n = [5, 40]
    k, v = _rows(45, 2, 32, torch.bfloat16, 4, dev)
    for kf, vf in ((0.03125, 0.25), (torch.tensor([0.01], device=dev), torch.tensor([3.0], device=dev)),
                   (torch.tensor([0.01, 0.2], device=dev), torch.tensor([3.0, 0.5], device=dev))):
        cache, scale = _empty_cache(t, 2, 32, torch.bfloat16, True, dev)
        wide = lambda f: np.broadcast_to(  # noqa: E731
            np.float32(f) if not isinstance(f, torch.Tensor) else f.cpu().numpy().reshape(-1, 1),
            (2, 2))
        want, _ = _expected(cache, scale, t, n, k, v, "static", wide(kf), wide(vf))
        hstu_kv_append(k, v, R.offsets(n).to(dev), cache, k_descale=kf, v_descale=vf, **t.args(dev))
        assert np.array_equal(R.values(cache.cpu()), want)


def test_read_into_given_rows_leaves_the_rest(cuda_device):
    dev = cuda_device
    t = R.Table([7, 0, 33], 32)
    cache, _ = _empty_cache(t, 2, 64, torch.float16, False, dev)
    wide = torch.full((40, 6, 64), 7.5, dtype=torch.float16, device=dev)
    k, v = wide[:, 1:3], wide[:, 4:]
    n = [3, 0, 33]
    hstu_kv_read(cache, R.offsets(n).to(dev), k=k, v=v, **t.args(dev))
    for b, at in ((0, 0), (2, 3)):
        page, row = t.rows(b)
        for plane, x in ((0, k), (1, v)):
            want = cache.cpu()[page, plane, row][len(page) - n[b]:]
            assert torch.equal(x[at:at + n[b]].cpu(), want)
    assert (wide[36:] == 7.5).all() and (wide[:, 0] == 7.5).all() and (wide[:, 3] == 7.5).all()


BAD = [  # what is wrong, and the sequences that must be left out
    ("offset decreases", {1, 2}), ("offset past the rows", {2}), ("last page too long", {1}),
    ("last page empty", {1}), ("more new rows than the sequence has", {1}),
    ("page offsets past page_ids", {2}),
]


def _break(what, t, n):
    so, po, last = R.offsets(n), t.page_offsets.clone(), t.last_page_len.clone()
    if what == "offset decreases":
        so[2] = so[1] - 1
    elif what == "offset past the rows":
        so[3] = so[3] + 100000
    elif what == "last page too long":
        last[1] = 33
    elif what == "last page empty":
        last[1] = 0
    elif what == "more new rows than the sequence has":
        last[1] = 2  # 34 positions for 40 rows
    elif what == "page offsets past page_ids":
        po[3] += 1
    return so, po, last


@pytest.mark.parametrize("what,bad", BAD)
def test_invalid_tables_write_nothing(cuda_device, what, bad):
    dev = cuda_device
    n, t = [10, 40, 20], R.Table([10, 50, 20], 32, seed=5)
    k, v = _rows(70, 2, 32, torch.bfloat16, 6, dev)
    cache, _ = _empty_cache(t, 2, 32, torch.bfloat16, False, dev)
    before = cache.clone()
    so, po, last = (x.to(dev) for x in _break(what, t, n))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = dict(page_offsets=po, page_ids=t.page_ids.to(dev), last_page_len=last)
    hstu_kv_append(k, v, so, cache, status=status, **kw)
    assert status.item() == 1
    hstu_kv_append(k, v, so, cache, **kw)  # without a status word: still in bounds
    for b in bad:
        page, row = t.rows(b)
        assert torch.equal(cache.cpu()[page, :, row], before.cpu()[page, :, row])
    page, row = t.rows(0)
    assert torch.equal(cache.cpu()[page, 0, row], k[:10].cpu())
    status.zero_()
    out = torch.full((70, 2, 32), 3.0, dtype=torch.bfloat16, device=dev)
    hstu_kv_read(cache, so, k=out, v=out.clone(), status=status, **kw)
    assert status.item() == 1 and torch.equal(out[:10], k[:10])


@pytest.mark.parametrize("bad_id", [-1, 1 << 20, -(1 << 40), (1 << 40)])
def test_invalid_page_ids_skip_their_rows(cuda_device, bad_id):
    dev = cuda_device
    t = R.Table([100], 32, seed=5)
    ids = t.page_ids.clone()
    ids[1] = bad_id
    k, v = _rows(100, 1, 16, torch.float16, 6, dev)
    cache, _ = _empty_cache(t, 1, 16, torch.float16, False, dev)
    before = cache.clone()
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = dict(t.args(dev), page_ids=ids.to(dev))
    hstu_kv_append(k, v, R.offsets([100]).to(dev), cache, status=status, **kw)
    assert status.item() == 1
    page, row = t.rows(0)
    assert torch.equal(cache.cpu()[page[32:64], :, row[32:64]], before.cpu()[page[32:64], :, row[32:64]])
    assert torch.equal(cache.cpu()[page[64:], 0, row[64:]], k[64:].cpu())
    out = torch.full_like(k, 9.0)
    hstu_kv_read(cache, R.offsets([100]).to(dev), k=out, v=out.clone(), **kw)
    assert (out[32:64] == 9.0).all() and torch.equal(out[:32], k[:32])


def test_empty_calls(cuda_device):
    dev = cuda_device
    t = R.Table([5], 32)
    cache, _ = _empty_cache(t, 2, 32, torch.bfloat16, False, dev)
    none = torch.empty(0, 2, 32, dtype=torch.bfloat16, device=dev)
    before = cache.clone()
    hstu_kv_append(none, none, R.offsets([0]).to(dev), cache, **t.args(dev))
    assert torch.equal(cache, before)
    e = R.Table([], 32)
    hstu_kv_append(none, none, R.offsets([]).to(dev), cache, **e.args(dev))
    k, v = hstu_kv_read(cache, R.offsets([]).to(dev), total_tokens=0, **e.args(dev))
    assert k.shape == v.shape == (0, 2, 32)


@pytest.mark.parametrize("fp8", [False, True])
def test_appended_rows_feed_hstu_fwd(cuda_device, fp8):
    """Rows appended (bf16, or E4M3 with per-head factors) and then attended to by hstu_fwd as
    its cached history, against the oracle on the cache's values."""
    dev, ps, Nk, D = cuda_device, 128, 2, 64
    hist, new = [300, 128, 5], [20, 40, 3]
    t = R.Table(hist, ps, seed=8)
    kh, vh = _rows(sum(hist), Nk, D, torch.bfloat16, 9, dev, strided=True)
    dt = R.FP8 if fp8 else torch.bfloat16
    cache = torch.zeros(t.num_pages, 2, ps, Nk, D, device=dev).to(dt)
    kw = {}
    if fp8:
        f = torch.rand(3, Nk, device=dev) * 0.05 + 0.01
        kw = dict(k_descale=f, v_descale=f * 2)
    hstu_kv_append(kh, vh, R.offsets(hist).to(dev), cache, **t.args(dev), **kw)
    g = torch.Generator().manual_seed(10)
    q, k, v = ((torch.randn(sum(new), Nk, D, generator=g) * (20 if fp8 else 0.5)).to(dt).to(dev)
               for _ in range(3))
    fwd = dict(kw, q_descale=kw["k_descale"]) if fp8 else {}
    out = hstu_fwd(q, k, v, R.offsets(new).to(dev), max_seqlen=64, max_seqlen_k=512, alpha=0.1,
                   seq_offsets_k=R.offsets(new).to(dev), kv_cache=cache, **t.args(dev), **fwd)
    qd, kd, vd, cd = (R.values(x.cpu()) for x in (q, k, v, cache))
    if fp8:
        so = np.concatenate([[0], np.cumsum(new)])
        fk, fv = f.cpu().double().numpy(), 2 * f.cpu().double().numpy()
        for b in range(3):
            page, row = t.rows(b)
            cd[page, 0, row] *= fk[b][:, None]
            cd[page, 1, row] *= fv[b][:, None]
            for x, m in ((qd, fk), (kd, fk), (vd, fv)):
                x[so[b]:so[b + 1]] *= m[b][:, None]
    so = R.offsets(new)
    ref = oracle.hstu_fwd(torch.tensor(qd), torch.tensor(kd), torch.tensor(vd), so,
                          seq_offsets_k=so, kv_cache=torch.tensor(cd), page_offsets=t.page_offsets,
                          page_ids=t.page_ids, last_page_len=t.last_page_len,
                          mask_type=oracle.MASK_CAUSAL, alpha=0.1, silu_scale=1.0 / 512,
                          max_seqlen=512, nthreads=4)
    err = np.max(np.abs(out.double().cpu().numpy() - ref)) / np.max(np.abs(ref))
    assert err <= (2.0 ** -4 if fp8 else 2e-2)  # hstu_fwd's own bounds (test_gpu_kv.py)
