"""Single tokens over batches of long sequences of unlike lengths, which the CTAs take by length: attention
and attention weights against the plain 64-bit implementations, with sequences without keys or queries,
many of one length, invalid ones, and up to as many sequences as are put in order. Tolerances: those of
test_gpu_softmax and test_gpu_evict."""
import numpy as np
import pytest
import torch

import kv_reference as R
import test_gpu_evict as EV
import test_gpu_kv4 as K4
import test_gpu_softmax as S
from hstu_dense_forward_gb300 import hstu_kv_weights, hstu_softmax_fwd

pytestmark = pytest.mark.gpu


def _lengths(B, seed, most=6000):
    """Unlike ones, a quarter of the mean length, some empty, the longest first, in the middle or last."""
    rng = np.random.default_rng(seed)
    x = rng.integers(0, most, B)
    x[rng.permutation(B)[:B // 4]] = most // 2
    x[rng.permutation(B)[:3]] = 0
    x[[0, B // 2, B - 1][seed % 3]] = most
    # what the order needs: two items an SM, 2048 keys and a longest one that is a quarter longer
    assert x.mean() >= 2200 and 1.25 * x.mean() * 1.02 <= most
    return [int(v) for v in x]


CASES = [("bf16", "same", 160, 2, 32, 32, torch.int64), ("fp16", "same", 256, 2, 16, 128, torch.int32),
         ("bf16", "scale", 255, 2, 32, 256, torch.int32), ("fp16", "cast", 81, 4, 16, 32, torch.int64),
         ("bf16", "same", 39, 8, 80, 128, torch.int64), ("bf16", "fp4", 40, 8, 32, 32, torch.int32)]


@pytest.mark.parametrize("dtype,mode,B,Nk,D,ps,index", CASES)
def test_attention_of_single_tokens(cuda_device, dtype, mode, B, Nk, D, ps, index):
    lengths = _lengths(B, B)
    n = [1] * B
    n[B // 3] = 0
    n = [min(x, L) for x, L in zip(n, lengths)]
    if mode == "fp4":
        K4.run_case(cuda_device, lengths, n, dtype, 2 * Nk, Nk, D, ps, index=index, seed=3)
    else:
        S.run_case(cuda_device, lengths, n, dtype, mode, Nk, Nk, D, ps, index=index, seed=3)


@pytest.mark.parametrize("dtype,mode,B,Nk,D,ps,index", CASES)
def test_weights_of_single_tokens(cuda_device, dtype, mode, B, Nk, D, ps, index):
    lengths = _lengths(B, B + 1)
    n = [min(1, L) for L in lengths]
    n[B // 3] = 0
    EV.run_weights(cuda_device, lengths, n, dtype, mode, Nk, Nk, D, ps, index=index, seed=4)


@pytest.mark.parametrize("mode", ["same", "scale"])
def test_invalid_sequences_among_them(cuda_device, mode):
    """Bad last lengths, a length above the bound and offsets that decrease: reported, the rows of those
    sequences left, the others' as in a batch without them."""
    dev, B, Nk, D, ps = cuda_device, 160, 2, 32, 32
    lengths = _lengths(B, 5)
    t = R.Table(lengths, ps, seed=1)
    cache, _, kw = S._filled(t, Nk, D, torch.bfloat16, mode, dev, 2)
    q = torch.randn(B, 2 * Nk, D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev)
    so, good = torch.arange(B + 1, device=dev), t.args(dev)
    bad = {k: x.clone() for k, x in good.items()}
    longest = max(lengths)
    out_of = [i for i in (7, 70, 111) if lengths[i] > 0]
    for i in out_of:
        bad["last_page_len"][i] = (0, 33, -5)[i % 3]
    results, weights = [], []
    for args, ok in ((good, True), (bad, False)):
        status = torch.zeros(2, dtype=torch.int32, device=dev)
        out = torch.full_like(q, 7.0)
        _, lse = hstu_softmax_fwd(q, cache, so, max_seqlen=1, max_seqlen_k=longest, out=out, return_lse=True,
                                  status=status[:1], **args, **kw)
        w = torch.ones(t.num_pages, Nk, ps, device=dev)
        if ok:
            every = lse
        hstu_kv_weights(q, every, cache, so, w, max_seqlen=1, max_seqlen_k=longest, status=status[1:], **args, **kw)
        assert status.tolist() == [int(not ok)] * 2
        results.append(out)
        weights.append(w)
    keep = torch.ones(B, dtype=torch.bool, device=dev)
    keep[out_of] = False
    assert torch.equal(results[1][keep], results[0][keep]) and (results[1][~keep] == 7.0).all()
    pages = torch.cat([good["page_ids"][good["page_offsets"][i]:good["page_offsets"][i + 1]] for i in out_of])
    rest = torch.ones(t.num_pages, dtype=torch.bool, device=dev)
    rest[pages] = False
    assert torch.equal(weights[1][rest], weights[0][rest]) and (weights[1][pages] == 1).all()
