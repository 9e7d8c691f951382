"""hstu_softmax_fwd against a plain 64-bit implementation: types, cache forms, head layouts,
head dims, page sizes, lengths from none to long ones, rows that see no key, what the unused
rows of pages hold, key ranges worked on in parts, strides, other streams and captured graphs,
and tables that the device must reject.

Tolerance of an output element, from the roundings of the path: the weights p_j are rounded to
q's type when that has 16 bits (half a step u_p = u relative, and half of the smallest fp16 value
absolutely; E4M3 keys and values are exact in 16 bits, so an E4M3 cache changes nothing: bf16
weights lie within 2^-8 of their values, which is what the product with V can be off by), the
output to its type (u), and a score of D products in fp32 is off by at most
(D + 8) 2^-24 alpha |q| |k|, which moves a weight and the sum by as much relatively each. With
A = sum_j p_j |v_j| / sum_j p_j:
  |error| <= u |out| + u_p A + (2 (D + 8) 2^-24 alpha |q| |k| + 2^-20 + Lk 2^-24) A
             + Lk 2^-25 max|v|  (16-bit weights)."""
import numpy as np
import pytest
import torch

import kv_reference as R
from hstu_dense_forward_gb300 import HstuError, hstu_kv_append, hstu_kv_read, hstu_softmax_fwd

pytestmark = pytest.mark.gpu


def _filled(t, Nk, D, dtype, mode, dev, seed, sigma=1.0):
    """A cache whose sequences hold random rows and whose other rows hold NaN (E4M3: NaN codes,
    scales of 255), with the values it stands for."""
    g = torch.Generator().manual_seed(seed)
    shape = (t.num_pages, 2, t.page_size, Nk, D)
    x = torch.randn(shape, generator=g) * torch.exp2(torch.randn(*shape[:-1], 1, generator=g) * 0.7)
    x *= sigma
    used = torch.zeros(t.num_pages, t.page_size, dtype=torch.bool)
    for b in range(len(t.lengths)):
        page, row = t.rows(b)
        used[torch.tensor(page), torch.tensor(row)] = True
    mask = used[:, None, :, None, None]
    kw = {}
    if mode == "same":
        cache = torch.where(mask, x, torch.nan).to(dtype)
        vals = R.values(torch.where(mask, x, 0.0).to(dtype))
    elif mode == "scale":
        e = R.row_exponent(x.numpy().astype(np.float64))
        codes = R.e4m3_round(np.ldexp(x.numpy().astype(np.float64), -e[..., None]))
        cache = torch.where(mask, torch.tensor(codes).float(), torch.nan).to(R.FP8)
        scale = torch.tensor((e + 127).swapaxes(2, 3)).to(torch.uint8)
        scale = torch.where(used[:, None, None, :], scale, torch.tensor(255, dtype=torch.uint8))
        kw["kv_scale"] = scale.contiguous().to(dev)
        vals = np.where(mask.numpy(), np.ldexp(codes, e[..., None]), 0.0)
    else:
        cache = torch.where(mask, x * 60.0, torch.nan).clamp(-448, 448).to(R.FP8)
        vals = np.where(mask.numpy(), R.values(cache), 0.0)
        if mode == "static":
            f = torch.rand(len(t.lengths), Nk, generator=g) * 0.02 + 0.01
            kw.update(k_descale=f.to(dev), v_descale=(2 * f).to(dev))
            for b in range(len(t.lengths)):
                page, row = t.rows(b)
                for plane in (0, 1):
                    vals[page, plane, row] *= ((1 + plane) * f[b]).double().numpy()[:, None]
        else:  # plain cast
            pass
    return cache.to(dev), vals, kw


def check(t, n, q, vals, got, lse, causal, alpha, dtype):
    so = np.concatenate([[0], np.cumsum(n)])
    u = R.HALF_STEP[dtype]
    up = 0.0 if dtype == torch.float32 else u
    qv = R.values(q.cpu())
    for b in range(len(n)):
        page, row = t.rows(b)
        K, V = vals[page, 0, row], vals[page, 1, row]
        out, ls, A, size = R.softmax_rows(qv[so[b]:so[b + 1]], K, V, causal, alpha)
        D, Lk = out.shape[2], K.shape[0]
        ex = (D + 8) * 2.0 ** -24 * size
        tol = u * np.abs(out) + (up + 2.0 ** -20 + Lk * 2.0 ** -24 + 2 * ex[..., None]) * A * 1.01
        if up and Lk:
            tol = tol + Lk * 2.0 ** -25 * np.abs(V).max()
        x = got[so[b]:so[b + 1]].double().cpu().numpy()
        bad = ~(np.abs(x - out) <= tol + 1e-30)
        assert not bad.any(), (b, np.argwhere(bad)[:5], x[bad][:5], out[bad][:5], tol[bad][:5])
        if lse is not None:
            y = lse[so[b]:so[b + 1]].double().cpu().numpy()
            assert np.array_equal(np.isneginf(y), np.isneginf(ls))
            fin = np.isfinite(ls)
            tol = 2 * ex + 2.0 ** -20 + (Lk + 8) * 2.0 ** -24 + np.abs(np.where(fin, ls, 0)) * 2.0 ** -22
            assert (np.abs(y - np.where(fin, ls, 0))[fin] <= tol[fin]).all()


def run_case(dev, lengths, n, dtype, mode, Nq, Nk, D, ps, causal=True, index=torch.int64,
             strided=False, alpha=None, seed=0, bounds=None, lse=True, tail=2, sigma=1.0):
    dt = R.DTYPES[dtype]
    t = R.Table(lengths, ps, index, seed=seed)
    cache, vals, kw = _filled(t, Nk, D, dt, mode, dev, seed + 1, sigma)
    g = torch.Generator().manual_seed(seed + 2)
    wide = torch.randn(sum(n) + tail, Nq + 3, D, generator=g).to(dt).to(dev)
    q = wide[:, 2:2 + Nq] if strided else wide[:, 2:2 + Nq].contiguous()
    alpha = D ** -0.5 if alpha is None else alpha
    out = torch.full((sum(n) + tail, Nq, D), 77.0, dtype=dt, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    sq, sk = bounds or (max(1, max(n)), max(1, max(lengths)))
    r = hstu_softmax_fwd(q, cache, R.offsets(n, index).to(dev), max_seqlen=sq, max_seqlen_k=sk,
                         causal=causal, alpha=alpha, out=out, return_lse=lse, status=status,
                         **t.args(dev), **kw)
    assert status.item() == 0
    assert (r[0] if lse else r) is out
    if tail:
        assert (out[-tail:] == 77.0).all()  # rows of no sequence
    check(t, n, q, vals, out, r[1] if lse else None, causal, alpha, dt)


# one token per sequence, over the lengths where tiles and pages end
TOKENS = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500]


@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,ps,index", [
    ("bf16", "same", 8, 2, 128, 128, torch.int64), ("fp16", "same", 4, 4, 64, 32, torch.int32),
    ("bf16", "scale", 16, 4, 128, 128, torch.int32), ("fp16", "scale", 5, 1, 64, 256, torch.int64),
    ("bf16", "static", 6, 2, 128, 32, torch.int64), ("fp16", "cast", 3, 3, 96, 32, torch.int64),
    ("fp32", "same", 8, 2, 64, 32, torch.int64), ("fp32", "scale", 4, 1, 128, 128, torch.int32),
    ("bf16", "same", 16, 1, 256, 128, torch.int64), ("bf16", "scale", 7, 1, 256, 32, torch.int64),
    ("fp16", "same", 12, 4, 16, 32, torch.int64), ("bf16", "same", 4, 4, 208, 256, torch.int64),
    ("bf16", "scale", 32, 2, 80, 32, torch.int64), ("fp16", "static", 4, 4, 176, 128, torch.int32),
])
def test_single_tokens(cuda_device, dtype, mode, Nq, Nk, D, ps, index):
    run_case(cuda_device, TOKENS, [1] * len(TOKENS), dtype, mode, Nq, Nk, D, ps, index=index, seed=11)


# chunks: lengths and new rows around tile and page edges, sequences without rows
CHUNK = ([0, 1, 5, 64, 129, 128, 300, 257, 400, 33], [0, 1, 5, 17, 129, 128, 1, 200, 0, 3])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,ps", [
    ("bf16", "same", 8, 2, 128, 128), ("fp16", "same", 3, 1, 64, 32), ("bf16", "same", 4, 4, 128, 32),
    ("bf16", "scale", 4, 1, 128, 128), ("fp16", "scale", 4, 2, 64, 32), ("bf16", "static", 5, 1, 96, 256),
    ("fp16", "cast", 2, 2, 128, 32), ("fp32", "same", 4, 2, 64, 128), ("fp32", "scale", 2, 1, 48, 32),
    ("bf16", "same", 7, 1, 256, 128), ("fp16", "scale", 2, 2, 256, 32), ("fp16", "same", 2, 1, 144, 256),
    ("bf16", "scale", 3, 3, 16, 32),
])
def test_chunks(cuda_device, dtype, mode, Nq, Nk, D, ps, causal):
    run_case(cuda_device, *CHUNK, dtype, mode, Nq, Nk, D, ps, causal=causal, seed=21)


# prompts: 256 rows of a kv head in the mean and more, which run in pairs of row tiles; pairs whose
# second tile is empty or partly filled, sequences of a few rows among them
PROMPT = ([300, 129, 70, 700, 4, 0, 1000], [300, 64, 70, 331, 1, 0, 65])


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,ps", [
    ("bf16", "same", 8, 2, 128, 128), ("fp16", "same", 6, 2, 64, 32), ("bf16", "scale", 8, 2, 128, 32),
    ("fp16", "scale", 4, 1, 64, 128), ("bf16", "static", 5, 1, 96, 256), ("bf16", "same", 4, 1, 256, 32),
    ("bf16", "scale", 3, 1, 32, 128), ("fp16", "cast", 7, 1, 128, 128), ("bf16", "scale", 4, 1, 256, 256),
])
def test_prompts(cuda_device, dtype, mode, Nq, Nk, D, ps, causal):
    run_case(cuda_device, *PROMPT, dtype, mode, Nq, Nk, D, ps, causal=causal, seed=71)


@pytest.mark.parametrize("dtype,mode,Nq,Nk,D,n,bound", [
    ("bf16", "same", 8, 2, 128, 75, 0), ("fp16", "same", 16, 4, 64, 70, 0), ("bf16", "scale", 8, 2, 128, 70, 0),
    ("fp16", "scale", 8, 2, 64, 66, 0), ("bf16", "same", 16, 4, 256, 20, 0), ("bf16", "same", 4, 4, 128, 30, 0),
    ("bf16", "scale", 4, 4, 80, 30, 0), ("fp16", "scale", 16, 4, 256, 20, 0), ("bf16", "same", 8, 2, 128, 75, 5000),
    ("fp16", "same", 16, 4, 64, 70, 5000), ("fp16", "same", 8, 8, 48, 30, 0), ("bf16", "same", 12, 4, 128, 25, 600),
])
def test_many_sequences(cuda_device, dtype, mode, Nq, Nk, D, n, bound):
    """More row tiles than CTAs can share out; with a loose bound on the keys, too."""
    g = torch.Generator().manual_seed(n)
    B = 70
    new = torch.randint(n // 2, n + n // 2, (B,), generator=g).tolist()
    new[3], new[-1] = 0, 1
    lengths = [m + h for m, h in zip(new, torch.randint(0, 200, (B,), generator=g).tolist())]
    lengths[5], new[5] = 0, 0
    run_case(cuda_device, lengths, new, dtype, mode, Nq, Nk, D, 32, seed=81,
             bounds=(max(new), bound) if bound else None)


@pytest.mark.parametrize("n", [1, 5, 20])
def test_more_sequences_than_a_table_holds(cuda_device, n):
    B = 600
    lengths = [(7 * b) % 61 + n for b in range(B)]
    run_case(cuda_device, lengths, [n] * B, "bf16", "same", 4, 1, 64, 32, seed=91)


@pytest.mark.parametrize("dtype,mode,n,Nq,D", [("bf16", "same", 300, 4, 128), ("bf16", "scale", 300, 4, 128),
                                               ("fp16", "same", 270, 4, 64), ("fp16", "scale", 200, 4, 64),
                                               ("bf16", "same", 7, 4, 128), ("fp16", "scale", 6, 4, 64),
                                               ("bf16", "same", 30, 4, 256)])
def test_items_over_many_ctas(cuda_device, dtype, mode, n, Nq, D):
    """Few items with long keys: the keys of one are parted among more CTAs than a warp's eight
    parts, beside a short sequence and an empty one."""
    run_case(cuda_device, [7000, 3, 0, 600], [n, 3, 0, n // 3], dtype, mode, Nq, 2, D, 128, seed=101)


@pytest.mark.parametrize("dtype,mode,G", [("bf16", "same", 1), ("fp16", "scale", 2), ("fp32", "same", 1),
                                          ("bf16", "scale", 16), ("fp16", "same", 24), ("bf16", "same", 128)])
def test_more_queries_than_keys(cuda_device, dtype, mode, G):
    """Causal rows before the first key see none (out 0, lse -inf); without a mask every row sees
    all keys, of any number; no keys at all."""
    lengths, n = [3, 0, 40, 129], [10, 4, 41, 300]
    for causal in (True, False):
        run_case(cuda_device, lengths, n, dtype, mode, 2 * G, 2, 64, 32, causal=causal, seed=31)


@pytest.mark.parametrize("dtype,mode,n,D", [("bf16", "same", 1, 128), ("fp16", "scale", 1, 64),
                                            ("bf16", "scale", 3, 128), ("fp32", "same", 2, 64),
                                            ("bf16", "same", 40, 128), ("bf16", "scale", 70, 128),
                                            ("fp16", "same", 33, 256), ("bf16", "scale", 1, 256)])
def test_long_keys_in_ranges(cuda_device, dtype, mode, n, D):
    """Few rows over long keys: the keys are split over CTAs and joined. One sequence is short
    (fewer ranges), one is empty, and the bounds are loose."""
    run_case(cuda_device, [9001, 150, 0, 4097], [n, n, 0, n], dtype, mode, 4, 2, D, 128, seed=41,
             bounds=(max(64, n), 20000))


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("fp16", "scale"), ("fp32", "same"), ("bf16", "scale")])
@pytest.mark.parametrize("n", [1, 50])
def test_strided_queries(cuda_device, dtype, mode, n):
    run_case(cuda_device, [200, 70], [n, n], dtype, mode, 6, 2, 64, 32, strided=True, seed=51)


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("bf16", "scale"), ("fp16", "same")])
@pytest.mark.parametrize("n", [1, 60])
def test_large_scores(cuda_device, dtype, mode, n):
    """Scores of some hundreds: the running maximum moves in steps far beyond what a 16-bit weight
    holds, and nearly all weights vanish."""
    run_case(cuda_device, [700, 300], [n, n], dtype, mode, 4, 2, 128, 128, alpha=1.0, seed=61, sigma=8.0)


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("bf16", "scale")])
def test_increasing_scores(cuda_device, dtype, mode):
    """Keys that grow along the sequence: every tile raises the maximum."""
    dev, ps, D = cuda_device, 128, 64
    L = 1000
    t = R.Table([L], ps)
    g = torch.Generator().manual_seed(3)
    d = torch.randn(D, generator=g)
    k = (d[None] / d.norm() * torch.linspace(0, 40, L)[:, None])[:, None, :]
    v = torch.randn(L, 1, D, generator=g)
    q = (d / d.norm() * 3.0).expand(70, 2, D).contiguous()
    k, v, q = (x.to(torch.bfloat16).to(dev) for x in (k, v, q))
    fp8 = mode == "scale"
    cache = torch.zeros(t.num_pages, 2, ps, 1, D, device=dev).to(R.FP8 if fp8 else torch.bfloat16)
    scale = torch.zeros(t.num_pages, 2, 1, ps, dtype=torch.uint8, device=dev) if fp8 else None
    hstu_kv_append(k, v, R.offsets([L]).to(dev), cache, kv_scale=scale, **t.args(dev))
    vals = R.cache_values(cache.cpu(), None if scale is None else scale.cpu())
    for n in (1, 70):
        got = hstu_softmax_fwd(q[:n], cache, R.offsets([n]).to(dev), max_seqlen=n, max_seqlen_k=L,
                               kv_scale=scale, **t.args(dev))
        check(t, [n], q[:n], vals, got, None, True, 1.0, torch.bfloat16)


def test_values_of_unlike_sizes(cuda_device):
    """Row scales from 2^-40 to 2^30 in one sequence, and a row of zeros (the smallest scale) that
    takes most of the weight."""
    dev, ps, D, L = cuda_device, 32, 64, 300
    g = torch.Generator().manual_seed(5)
    k = torch.randn(L, 1, D, generator=g)
    v = torch.randn(L, 1, D, generator=g) * torch.exp2(torch.randint(-40, 30, (L, 1, 1), generator=g).float())
    v[17] = 0
    k[17] *= 3
    t = R.Table([L], ps)
    cache = torch.zeros(t.num_pages, 2, ps, 1, D, device=dev).to(R.FP8)
    scale = torch.zeros(t.num_pages, 2, 1, ps, dtype=torch.uint8, device=dev)
    k, v = k.to(torch.bfloat16).to(dev), v.to(torch.bfloat16).to(dev)
    hstu_kv_append(k, v, R.offsets([L]).to(dev), cache, kv_scale=scale, **t.args(dev))
    vals = R.cache_values(cache.cpu(), scale.cpu())
    for n in (1, 40):
        q = k[17].expand(n, 4, D).contiguous()
        got, lse = hstu_softmax_fwd(q, cache, R.offsets([n]).to(dev), max_seqlen=n, max_seqlen_k=L,
                                    alpha=0.05, kv_scale=scale, return_lse=True, causal=False,
                                    **t.args(dev))
        check(t, [n], q, vals, got, lse, False, 0.05, torch.bfloat16)


@pytest.mark.parametrize("what", ["offset decreases", "too many queries", "too many keys",
                                  "last page too long", "page id"])
@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("fp16", "scale"), ("fp32", "same")])
@pytest.mark.parametrize("n", [1, 40])
def test_invalid_tables(cuda_device, what, dtype, mode, n):
    """The bad sequence is left out (a bad page id: unspecified outputs), the others are right, and
    the status word says so."""
    dev, dt = cuda_device, R.DTYPES[dtype]
    lengths, m = [90, 100, 80], [n, n, n]
    t = R.Table(lengths, 32, seed=7)
    cache, vals, kw = _filled(t, 2, 64, dt, mode, dev, 8)
    q = torch.randn(3 * n, 4, 64, generator=torch.Generator().manual_seed(9)).to(dt).to(dev)
    so, args = R.offsets(m), t.args(torch.device("cpu"))
    sq, sk = n, 100
    if what == "offset decreases":
        so[2] = so[1] - 1
    elif what == "too many queries":
        so[2] += 1
        so[3] += 1
        q = torch.cat([q, q[:1]])
    elif what == "too many keys":
        sk = 99
    elif what == "last page too long":
        args["last_page_len"][1] = 33
    else:
        args["page_ids"][int(args["page_offsets"][1]) + 1] = 1 << 30
    out = torch.full(q.shape, 5.0, dtype=dt, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    hstu_softmax_fwd(q, cache, so.to(dev), max_seqlen=sq, max_seqlen_k=sk, alpha=0.1, out=out,
                     status=status, **{k: x.to(dev) for k, x in args.items()}, **kw)
    assert status.item() == 1
    one = R.Table([90], 32, seed=7)
    one.page_ids = t.page_ids[:3]
    check(one, [n], q[:n], vals, out[:n], None, True, 0.1, dt)
    if what == "last page too long" or what == "too many keys":
        assert (out[n:2 * n] == 5.0).all()


@pytest.mark.parametrize("n,mode", [(1, "same"), (1, "scale"), (60, "same"), (60, "scale")])
def test_other_stream_and_graph(cuda_device, n, mode):
    """A call on a side stream equals one on the default stream bit for bit; two graphs captured
    from the same call replay side by side, on new inputs, and give those inputs' results."""
    dev = cuda_device
    t = R.Table([3000, 700], 128, seed=3)
    cache, vals, kw = _filled(t, 2, 128, torch.bfloat16, mode, dev, 4)
    so, args = R.offsets([n, n]).to(dev), t.args(dev)
    call = lambda x: hstu_softmax_fwd(x, cache, so, max_seqlen=n, max_seqlen_k=3000, alpha=0.1,  # noqa: E731
                                      **args, **kw)
    q = [torch.randn(2 * n, 4, 128, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).to(dev)
         for i in range(4)]
    want = [call(x).clone() for x in q]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = call(q[0])
    torch.cuda.synchronize()
    assert torch.equal(got, want[0])
    inputs = [q[0].clone(), q[1].clone()]
    graphs, outs = [], []
    for x in inputs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(x))
        graphs.append(g)
    inputs[0].copy_(q[2])
    inputs[1].copy_(q[3])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[2]) and torch.equal(outs[1], want[3])


@pytest.mark.parametrize("mode", ["same", "scale"])
def test_calls_at_once(cuda_device, mode):
    """Calls of every kernel on streams of their own, enqueued in turn, equal the calls alone bit
    for bit."""
    dev = cuda_device
    calls = []
    for lengths, n, Nq, D in (([150] * 70, [40] * 70, 8, 128), ([3000, 2500], [70, 300], 4, 128),
                              ([400] * 20, [300] * 20, 8, 64), ([900] * 40, [1] * 40, 4, 128),
                              ([60] * 90, [30] * 90, 16, 64)):
        t = R.Table(lengths, 32, seed=Nq)
        cache, _, kw = _filled(t, 2, D, torch.bfloat16, mode, dev, D)
        g = torch.Generator().manual_seed(9)
        q = torch.randn(sum(n), Nq, D, generator=g).bfloat16().to(dev)
        so = R.offsets(n).to(dev)
        kw.update(t.args(dev), max_seqlen=max(n), max_seqlen_k=max(lengths), alpha=0.1)
        calls.append((q, cache, so, kw, torch.cuda.Stream()))
    alone = [hstu_softmax_fwd(q, cache, so, **kw) for q, cache, so, kw, _ in calls]
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for i, (q, cache, so, kw, stream) in enumerate(calls):
            with torch.cuda.stream(stream):
                got.append((i, hstu_softmax_fwd(q, cache, so, **kw)))
    torch.cuda.synchronize()
    for i, x in got:
        assert torch.equal(x, alone[i])


@pytest.mark.parametrize("mode", ["same", "scale"])
def test_serving_run(cuda_device, mode):
    """As a user runs them: a prompt in two chunks, then single tokens, each step appended and
    attended to, over one growing table; every step against the whole sequence so far, and the
    rows read back at the end are what was appended."""
    dev, ps, Nk, Nq, D = cuda_device, 32, 2, 4, 64
    fp8 = mode == "scale"
    steps = [[70, 5], [40, 90], [1, 1], [1, 1], [1, 0], [1, 1]]
    total = np.sum(steps, axis=0)
    full = R.Table(total, ps, seed=12)
    g = torch.Generator().manual_seed(13)
    qkv = torch.randn(int(total.sum()), Nq + 2 * Nk, D, generator=g).to(torch.bfloat16).to(dev)
    cache = torch.zeros(full.num_pages, 2, ps, Nk, D, device=dev).to(R.FP8 if fp8 else torch.bfloat16)
    scale = torch.zeros(full.num_pages, 2, Nk, ps, dtype=torch.uint8, device=dev) if fp8 else None
    at, length = 0, np.zeros(2, dtype=int)
    for n in steps:
        x = qkv[at:at + sum(n)]
        at, length = at + sum(n), length + n
        t = R.Table(length, ps)  # the first pages of the full table
        own = [full.page_ids[int(full.page_offsets[b]):][:-(-int(length[b]) // ps)] for b in range(2)]
        t.page_ids = torch.cat(own)
        so = R.offsets(n).to(dev)
        hstu_kv_append(x[:, Nq:Nq + Nk], x[:, Nq + Nk:], so, cache, kv_scale=scale, **t.args(dev))
        got = hstu_softmax_fwd(x[:, :Nq], cache, so, max_seqlen=max(n), max_seqlen_k=256, alpha=0.125,
                               kv_scale=scale, **t.args(dev))
        vals = R.cache_values(cache.cpu(), None if scale is None else scale.cpu())
        check(t, n, x[:, :Nq], vals, got, None, True, 0.125, torch.bfloat16)
    k, v = hstu_kv_read(cache, R.offsets(total).to(dev), total_tokens=int(total.sum()), kv_scale=scale,
                        **full.args(dev))
    row = 0
    for b in range(2):
        at = 0
        for n in steps:
            base = at + (n[0] if b else 0)
            x = qkv[base:base + n[b], Nq:Nq + Nk].float()
            y = k[row:row + n[b]].float()
            if fp8:  # half a step of E4M3 below 448, relative to the row's largest value
                assert ((x - y).abs() <= x.abs() * 2.0 ** -4 + x.abs().amax(-1, keepdim=True) * 2.0 ** -17).all()
            else:
                assert torch.equal(x, y)
            at, row = at + sum(n), row + n[b]


def test_empty_calls(cuda_device):
    dev = cuda_device
    t = R.Table([5], 32)
    cache, _, _ = _filled(t, 2, 64, torch.bfloat16, "same", dev, 1)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=dev)
    out, lse = hstu_softmax_fwd(q, cache, R.offsets([0]).to(dev), max_seqlen=1, max_seqlen_k=5,
                                return_lse=True, **t.args(dev))
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_bad_sizes_are_refused(cuda_device):
    dev = cuda_device
    t = R.Table([5], 32)
    cache, _, _ = _filled(t, 2, 64, torch.bfloat16, "same", dev, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=dev)
    so, kw = R.offsets([1]).to(dev), dict(max_seqlen=1, max_seqlen_k=5, **t.args(dev))
    for bad in (dict(alpha=0.0), dict(alpha=-1.0), dict(alpha=float("nan")), dict(max_seqlen=0),
                dict(max_seqlen_k=0)):
        with pytest.raises(HstuError):
            hstu_softmax_fwd(q, cache, so, **{**kw, **bad})
    with pytest.raises(ValueError):
        hstu_softmax_fwd(q[:, :3], cache, so, **kw)
    with pytest.raises(TypeError):
        hstu_softmax_fwd(q.half(), cache, so, **kw)
    with pytest.raises(HstuError):  # rows off the 16-byte grid
        hstu_softmax_fwd(torch.zeros(9 * 64, dtype=torch.bfloat16, device=dev)[1:257].view(1, 4, 64),
                         cache, so, **kw)
