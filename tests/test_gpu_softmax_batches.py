"""hstu_softmax_fwd over batches of unlike sequences: an invalid sequence in the middle (the ones
around it are right, its own rows are left as they were), one prompt among single tokens, bounds far
above the lengths. Tolerances: those of test_gpu_softmax."""
import pytest
import torch

import kv_reference as R
from hstu_dense_forward_gb300 import HstuError, hstu_softmax_fwd
from test_gpu_softmax import _filled, check, run_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("what", ["too many queries", "too many keys", "last page too long", "last page empty",
                                  "pages decrease"])
@pytest.mark.parametrize("dtype,mode,Nq,D", [("bf16", "same", 4, 128), ("bf16", "scale", 4, 128),
                                             ("fp16", "same", 4, 64), ("fp16", "scale", 4, 64),
                                             ("bf16", "same", 2, 256), ("fp32", "same", 4, 64),
                                             ("fp32", "scale", 4, 64)])
@pytest.mark.parametrize("lengths,n", [
    ([90, 100, 80, 0, 33], [1, 1, 1, 0, 1]),            # few rows
    ([90, 100, 80, 0, 60], [40, 40, 40, 0, 7]),         # a tile each
    ([3000, 2500, 2700, 0, 600], [300, 290, 300, 0, 20])])  # key tiles shared among CTAs, joined
def test_invalid_sequence_among_others(cuda_device, what, dtype, mode, Nq, D, lengths, n):
    dev, dt = cuda_device, R.DTYPES[dtype]
    t = R.Table(lengths, 32, seed=7)
    cache, vals, kw = _filled(t, 2, D, dt, mode, dev, 8)
    q = torch.randn(sum(n), Nq, D, generator=torch.Generator().manual_seed(9)).to(dt).to(dev)
    args, m = {k: x.clone() for k, x in t.args(torch.device("cpu")).items()}, list(n)
    sq, sk = max(n), max(lengths)
    if what == "too many queries":
        m[1] += sq - m[1] + 1
        q = torch.cat([q, q[:m[1] - n[1]]])
    elif what == "too many keys":
        pages = -(-sk // 32) + 1  # one more than the bound has, all of them valid ids
        first, last = int(args["page_offsets"][1]), int(args["page_offsets"][2])
        ids, more = args["page_ids"], pages - (last - first)
        args["page_ids"] = torch.cat([ids[:last], ids[:1].repeat(more), ids[last:]])
        args["page_offsets"][2:] += more
    elif what == "last page too long":
        args["last_page_len"][1] = 33
    elif what == "last page empty":
        args["last_page_len"][1] = 0
    else:  # sequence 1 ends before it begins, and sequence 2 has more pages than its own
        args["page_offsets"][2] = args["page_offsets"][1] - 1
    out = torch.full(q.shape, 5.0, dtype=dt, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    hstu_softmax_fwd(q, cache, R.offsets(m).to(dev), max_seqlen=sq, max_seqlen_k=sk, alpha=0.1, out=out,
                     status=status, **{k: x.to(dev) for k, x in args.items()}, **kw)
    assert status.item() == 1
    at = 0
    for b, rows in enumerate(m):
        x = out[at:at + rows]
        if b == 1:
            assert (x == 5.0).all()
        elif not (what == "pages decrease" and b == 2):
            one = R.Table([lengths[b]], 32)
            first = int(t.page_offsets[b])
            one.page_ids = t.page_ids[first:first + -(-lengths[b] // 32)]
            check(one, [rows], q[at:at + rows], vals, x, None, True, 0.1, dt)
        at += rows


@pytest.mark.parametrize("bounds", [None, (4096, 20000)])
@pytest.mark.parametrize("dtype,mode,Nq,Nk,D", [
    ("bf16", "same", 8, 2, 128), ("bf16", "scale", 8, 2, 128), ("fp16", "same", 4, 4, 64),
    ("fp16", "scale", 4, 1, 64), ("bf16", "static", 4, 2, 128), ("fp16", "cast", 2, 2, 256),
    ("fp32", "same", 4, 2, 64), ("fp32", "scale", 4, 2, 64)])
def test_one_prompt_among_single_tokens(cuda_device, dtype, mode, Nq, Nk, D, bounds):
    """What a server's step is, and what a captured one with loose bounds is."""
    lengths = [(37 * b) % 400 + 1 for b in range(30)] + [700] + [(53 * b) % 300 + 1 for b in range(20)]
    n = [1] * 30 + [200] + [1] * 20
    run_case(cuda_device, lengths, n, dtype, mode, Nq, Nk, D, 32, bounds=bounds, seed=111)


@pytest.mark.parametrize("dtype,mode", [("bf16", "same"), ("bf16", "scale"), ("fp32", "same")])
def test_single_tokens_under_loose_bounds(cuda_device, dtype, mode):
    lengths = [(37 * b) % 400 + 1 for b in range(40)]
    run_case(cuda_device, lengths, [1] * 40, dtype, mode, 8, 2, 128, 32, bounds=(1 << 24, 1 << 30), seed=121)


@pytest.mark.parametrize("bad", [dict(max_seqlen=1 << 31), dict(max_seqlen_k=1 << 31), dict(max_seqlen=-(1 << 40)),
                                 dict(alpha=1e39), dict(alpha=-1e300), dict(alpha=float("inf"))])
def test_sizes_beyond_the_abi_are_refused(cuda_device, bad):
    dev = cuda_device
    t = R.Table([5], 32)
    cache, _, _ = _filled(t, 2, 64, torch.bfloat16, "same", dev, 1)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16, device=dev)
    kw = dict(max_seqlen=1, max_seqlen_k=5, **t.args(dev))
    with pytest.raises(HstuError):
        hstu_softmax_fwd(q, cache, R.offsets([1]).to(dev), **{**kw, **bad})
