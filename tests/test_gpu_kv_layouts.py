"""The paged KV cache operators where indexes pass 32 bits, where rows stand in front of the first
sequence, where no sequence has a page, with static factors of every granularity, and captured into a
graph as a process's first call. Tolerances: those of test_gpu_softmax; copies are exact."""
import subprocess
import sys

import numpy as np
import pytest
import torch

import kv_reference as R
from hstu_dense_forward_gb300 import hstu_kv_append, hstu_kv_read, hstu_softmax_fwd
from test_gpu_softmax import _filled, check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("bf16", True), ("fp32", False), ("fp32", True)])
def test_cache_and_rows_beyond_32_bits(cuda_device, dtype, fp8, n):
    """A cache of more than 2^32 elements of which the last pages are used, and rows of q, k and v
    2^25 elements apart."""
    dev, dt, ps, Nk, Nq, D = cuda_device, R.DTYPES[dtype], 256, 8, 8, 256
    lengths = [300, 70]
    t = R.Table(lengths, ps)
    pages = (1 << 32) // (2 * ps * Nk * D) + 10
    cache = torch.empty(pages, 2, ps, Nk, D, device=dev, dtype=R.FP8 if fp8 else dt)
    args = t.args(dev)
    args["page_ids"] = pages - 1 - args["page_ids"]
    if fp8:
        args["kv_scale"] = torch.empty(pages, 2, Nk, ps, dtype=torch.uint8, device=dev)
    g = torch.Generator().manual_seed(1)
    T, stride = sum(lengths), 1 << 25
    kv = torch.randn(2, T, Nk, D, generator=g).to(dt).to(dev)
    hstu_kv_append(kv[0], kv[1], R.offsets(lengths).to(dev), cache, **args)
    # the last 2 n rows again, far apart
    wide = torch.empty((2 * n - 1) * stride + 3 * Nk * D, dtype=dt, device=dev)
    assert (2 * n - 1) * stride > 1 << 31 or n == 1
    rows = [wide[i * Nk * D:].as_strided((2 * n, Nk, D), (stride, D, 1)) for i in range(3)]
    q = torch.randn(2 * n, Nq, D, generator=g).to(dt)
    rows[0].copy_(q.to(dev))
    last = torch.cat([torch.arange(300 - n, 300), torch.arange(370 - n, 370)]).to(dev)
    for i in (0, 1):
        rows[1 + i].copy_(kv[i, last])
    hstu_kv_append(rows[1], rows[2], R.offsets([n, n]).to(dev), cache, **args)
    k, v = hstu_kv_read(cache, R.offsets(lengths).to(dev), total_tokens=T, dtype=torch.float32 if fp8 else dt, **args)
    used = cache[args["page_ids"]].cpu()
    vals = R.cache_values(used, args["kv_scale"][args["page_ids"]].cpu() if fp8 else None)
    one = R.Table(lengths, ps)
    one.page_ids = torch.arange(one.page_ids.numel())  # places in `used`
    for b, at in ((0, 0), (1, 300)):
        page, row = one.rows(b)
        for plane, x in ((0, k), (1, v)):
            assert np.array_equal(R.values(x[at:at + lengths[b]].cpu()), vals[page, plane, row])
        if not fp8:
            assert torch.equal(k[at:at + lengths[b]], kv[0, at:at + lengths[b]])
    out = hstu_softmax_fwd(rows[0], cache, R.offsets([n, n]).to(dev), max_seqlen=n, max_seqlen_k=300, alpha=0.06,
                           **args)
    check(one, [n, n], q, vals, out, None, True, 0.06, dt)


@pytest.mark.parametrize("n", [1, 7, 60])
@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("bf16", "scale"), ("fp32", "same"), ("fp32", "scale")])
def test_rows_in_front_of_the_first_sequence(cuda_device, dtype, mode, n):
    """seq_offsets[0] > 0: the rows before it belong to no sequence."""
    dev, dt, lead = cuda_device, R.DTYPES[dtype], 5
    lengths = [700, 3000, 64]
    t = R.Table(lengths, 32, seed=3)
    cache, vals, kw = _filled(t, 2, 64, dt, mode, dev, 4)
    q = torch.randn(lead + 3 * n + 2, 4, 64, generator=torch.Generator().manual_seed(5)).to(dt).to(dev)
    so = (R.offsets([n] * 3) + lead).to(dev)
    out = torch.full(q.shape, 5.0, dtype=dt, device=dev)
    hstu_softmax_fwd(q, cache, so, max_seqlen=n, max_seqlen_k=3000, alpha=0.1, out=out, **t.args(dev), **kw)
    assert (out[:lead] == 5.0).all() and (out[-2:] == 5.0).all()
    check(t, [n] * 3, q[lead:-2], vals, out[lead:-2], None, True, 0.1, dt)
    k, v = (torch.full((lead + 3 * n + 2, 2, 64), 5.0, dtype=dt, device=dev) for _ in range(2))
    hstu_kv_read(cache, so, k=k, v=v, **t.args(dev), **kw)
    for x in (k, v):
        assert (x[:lead] == 5.0).all() and (x[-2:] == 5.0).all()
    before = cache.view(torch.uint8).clone()
    hstu_kv_append(k, v, so, cache, **t.args(dev), **kw)  # what was read, to where it was
    if mode == "same":
        assert torch.equal(cache.view(torch.uint8), before)


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("fp16", "scale"), ("fp32", "same")])
@pytest.mark.parametrize("n", [1, 40, 300])
def test_no_sequence_has_a_page(cuda_device, dtype, mode, n):
    dev, dt = cuda_device, R.DTYPES[dtype]
    t = R.Table([0, 0], 32)
    cache, _, kw = _filled(t, 2, 64, dt, mode, dev, 6)
    q = torch.randn(2 * n, 4, 64).to(dt).to(dev)
    for causal in (True, False):
        out, lse = hstu_softmax_fwd(q, cache, R.offsets([n, n]).to(dev), max_seqlen=n, max_seqlen_k=500,
                                    causal=causal, return_lse=True, **t.args(dev), **kw)
        assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("n", [1, 8, 40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_one_factor_and_one_per_sequence(cuda_device, dtype, n):
    dev, dt, lengths = cuda_device, R.DTYPES[dtype], [330, 400, 301]
    t = R.Table(lengths, 32, seed=2)
    cache, vals, _ = _filled(t, 2, 64, dt, "cast", dev, 7)
    q = torch.randn(3 * n, 4, 64, generator=torch.Generator().manual_seed(8)).to(dt).to(dev)
    for kf, vf in ((0.02, -0.03), (torch.tensor([0.02], device=dev), torch.tensor(0.5, device=dev).reshape(1)),
                   (torch.tensor([0.02, -0.01, 0.03], device=dev), torch.tensor([0.5, 3.0, -0.1], device=dev))):
        got = hstu_softmax_fwd(q, cache, R.offsets([n] * 3).to(dev), max_seqlen=n, max_seqlen_k=400, alpha=0.1,
                               k_descale=kf, v_descale=vf, **t.args(dev))
        x = vals.copy()
        for b in range(3):
            page, row = t.rows(b)
            for plane, f in ((0, kf), (1, vf)):
                f = f.cpu().double().numpy() if isinstance(f, torch.Tensor) else np.array([np.float32(f)])
                x[page, plane, row] *= float(f[b if f.size == 3 else 0])
        check(t, [n] * 3, q, x, got, None, True, 0.1, dt)


CAPTURE = """
import sys
sys.path[:0] = {path!r}
import torch
import kv_reference as R
from hstu_dense_forward_gb300 import hstu_kv_append, hstu_kv_read, hstu_softmax_fwd
dev, n, fp8 = torch.device("cuda", 0), {n}, {fp8}
t = R.Table([900, 2000], 32)
cache = torch.zeros(t.num_pages, 2, 32, 2, 64, device=dev).to(R.FP8 if fp8 else torch.bfloat16)
args = t.args(dev)
if fp8:
    args["kv_scale"] = torch.full((t.num_pages, 2, 2, 32), 127, dtype=torch.uint8, device=dev)
k, v, q = (torch.randn(2 * n, h, 64, device=dev).bfloat16() for h in (2, 2, 4))
so = R.offsets([n, n]).to(dev)
def step():
    hstu_kv_append(k, v, so, cache, **args)
    out = hstu_softmax_fwd(q, cache, so, max_seqlen=n, max_seqlen_k=2000, **args)
    return (out, *hstu_kv_read(cache, so, total_tokens=2 * n, **args))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    a = step()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(a, step()))
print("same")
"""


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 60])
def test_first_call_of_a_process_is_captured(cuda_device, n, fp8):
    code = CAPTURE.format(path=sys.path, n=n, fp8=fp8)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
