"""hstu_softmax_fwd over E4M3 caches with row scales of very unlike sizes: rows far above the others
(with and without weight, seen and hidden by the causal mask), rows of zeros (the smallest scale)
beside large ones, queries of zeros, keys and queries at opposite ends of the range.

Tolerance, from the roundings of the path. Codes times powers of two are exact, so keys and values
are; a bf16 query becomes fp16 times a power of two of its row, exact but for elements below 2^-38 of
the row's largest. A score of D products in fp32 is off by ex_j = (D + 8) 2^-24 alpha |q| |k_j|, which
moves weight j by as much relatively (p_j: the normalised weights, A = sum_j p_j |v_j|). Weights are
rounded to fp16: by half a step, 2^-11, relatively, and by 2^-25 absolutely in the unit of the
references. That unit times the largest code is at most twice (references are whole powers of two)
the largest p_j 448 2^(e_j), e_j the row scale's exponent, and 448 2^(e_j) at most twice the largest
magnitude in row j: the absolute part is at most Lk 2^-25 * 2 * 2 B = Lk 2^-23 B, B the largest
p_j max|v_j|. A row of zeros is no reason to treat its key tile (128 keys at most) row by row, so its
score enters the reference with the largest scale of the tile: in B it counts like the largest row
less than 128 rows away. The output is rounded to its type, relatively by u, and absolutely by half of the
smallest value (fp16: 2^-25).
  |error| <= u |out| + (2^-11 + 2^-20 + Lk 2^-24) A + sum_j p_j ex_j |v_j| + (sum_j p_j ex_j) A
             + Lk 2^-23 B
fp32 queries: the same without the weights' roundings."""
import numpy as np
import pytest
import torch

import kv_reference as R
from hstu_dense_forward_gb300 import hstu_softmax_fwd

pytestmark = pytest.mark.gpu


def quantised(k, v, ps, dev, seed=0):
    """k, v [L, Nk, D] (64 bits) as one sequence of an E4M3 cache with row scales: arguments of a
    call and the values that the cache stands for."""
    L, Nk, D = k.shape
    t = R.Table([L], ps, seed=seed)
    page, row = t.rows(0)
    cache = np.full((t.num_pages, 2, ps, Nk, D), np.nan)
    scale = np.full((t.num_pages, 2, Nk, ps), 255, dtype=np.uint8)
    vals = []
    for plane, x in ((0, k), (1, v)):
        e = R.row_exponent(x)
        codes = R.e4m3_round(np.ldexp(x, -e[..., None]))
        cache[page, plane, row] = codes
        scale[page, plane, :, row] = e + 127
        vals.append(np.ldexp(codes, e[..., None]))
    kw = dict(t.args(dev), kv_scale=torch.tensor(scale).to(dev))
    return torch.tensor(cache).float().to(R.FP8).to(dev), kw, vals[0], vals[1]


def check(q, K, V, got, lse, causal, alpha, sharp=False, weight_bits=11):
    """Output and lse of the last n positions against 64 bits, with the tolerance above. sharp: every
    key scores exactly the most or far less than that, so that its errors move no weight. The weights
    are rounded to weight_bits bits."""
    dt, q = got.dtype, R.values(q.cpu())
    n, Nq, D = q.shape
    Lk, G = K.shape[0], Nq // K.shape[1]
    up = 0.0 if dt == torch.float32 else 2.0 ** -weight_bits
    u = R.HALF_STEP[dt]
    got, lse = got.double().cpu().numpy(), lse.double().cpu().numpy()
    seen = np.arange(Lk)[None, :] <= ((Lk - n + np.arange(n))[:, None] if causal else Lk)
    for h in range(Nq):
        k, v = K[:, h // G], V[:, h // G]
        x = np.where(seen, alpha * (q[:, h] @ k.T), -np.inf)
        top = x.max(1, keepdims=True)
        assert np.isfinite(top).all()
        p = np.exp(x - top)
        total = p.sum(1, keepdims=True)
        p /= total
        out, A = p @ v, p @ np.abs(v)
        ex = (D + 8) * 2.0 ** -24 * alpha * np.linalg.norm(q[:, h], axis=1)[:, None] * \
            np.linalg.norm(k, axis=1)[None, :]
        e1, e0 = (p * ex) @ np.abs(v), (p * ex).sum(1)
        if sharp:
            assert ((x == top) | (x < top - 4 * ex - 60.0)).all()
            e1, e0 = 0.0 * e1, 0.0 * e0
        size = np.abs(v).max(1)
        near = np.array([size[max(0, j - 127):j + 128].max() for j in range(Lk)])
        B = (p * np.where(size == 0.0, near, size)).max(1)
        tol = u * np.abs(out) + (up + 2.0 ** -20 + Lk * 2.0 ** -24 + e0[:, None]) * A * 1.01 + \
            e1 * 1.01 + (Lk * 2.0 ** -23 * B[:, None] if up else 0.0) + \
            (2.0 ** -25 if dt == torch.float16 else 0.0)
        bad = ~(np.abs(got[:, h] - out) <= tol + 1e-37)
        if dt == torch.float16:  # rounds to infinity from 65520 on
            bad &= ~((got[:, h] == np.copysign(np.inf, out)) & (np.abs(out) + tol >= 65520.0))
        assert not bad.any(), (h, int(bad.sum()), np.argwhere(bad)[:4], got[:, h][bad][:4], out[bad][:4],
                               tol[bad][:4])
        ls = top[:, 0] + np.log(total[:, 0])
        tol = 1.01 * (p * ex).sum(1) + 2.0 ** -20 + (Lk + 8) * 2.0 ** -24 + np.abs(ls) * 2.0 ** -22
        bad = ~(np.abs(lse[:, h] - ls) <= tol)
        assert not bad.any(), (h, np.argwhere(bad)[:4], lse[:, h][bad][:4], ls[bad][:4], tol[bad][:4])


def run(dev, q, k, v, causal, alpha, ps=32, seed=0, sharp=False):
    """q [n, Nq, D] (its type), k, v [L, Nk, D] (numpy)."""
    cache, kw, K, V = quantised(k, v, ps, dev, seed)
    n, q = q.shape[0], q.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got, lse = hstu_softmax_fwd(q, cache, R.offsets([n]).to(dev), max_seqlen=n, max_seqlen_k=k.shape[0],
                                causal=causal, alpha=alpha, return_lse=True, status=status, **kw)
    assert status.item() == 0
    check(q, K, V, got, lse, causal, alpha, sharp)


def directed(n, Nq, D, dtype, seed, size=3.0, noise=0.3):
    """Queries near size * d, and the unit vector d: a key c * d scores about alpha * size * c."""
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(D, generator=g)
    d /= d.norm()
    q = size * d + noise * torch.randn(n, Nq, D, generator=g)
    return q.to(dtype), d.double().numpy()


ROWS = [1, 16, 17, 300]  # query rows of a kv head: both sides of the kernels' borders


@pytest.mark.parametrize("up", [4, 8, 12, 20, 30, 60])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256), ("fp32", 64)])
def test_large_value_row_without_weight(cuda_device, dtype, D, n, up):
    """One value row 2^up above 699 others, with a weight of about e^-60."""
    q, d = directed(n, 1, D, R.DTYPES[dtype], 1)
    g = np.random.default_rng(2)
    k, v = g.standard_normal((700, 1, D)), g.standard_normal((700, 1, D))
    k[333, 0] = -60.0 / (3.0 * D ** -0.5) * d
    v[333] = np.ldexp(v[333], up)
    run(cuda_device, q, k, v, False, D ** -0.5)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 128), ("bf16", 64), ("fp32", 128)])
def test_value_row_with_all_the_weight_below_a_large_one(cuda_device, dtype, D, n):
    """Nearly all weight on one value row 2^28 below another one of its tile, which has none."""
    q, d = directed(n, 2, D, R.DTYPES[dtype], 3)
    g = np.random.default_rng(4)
    k, v = 0.1 * g.standard_normal((90, 1, D)), g.standard_normal((90, 1, D))
    k[40, 0], k[50, 0] = 40.0 / (3.0 * D ** -0.5) * d, -90.0 / (3.0 * D ** -0.5) * d
    v[50] = np.ldexp(v[50], 28)
    run(cuda_device, q, k, v, False, D ** -0.5)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("up", [16, 24, 40])
@pytest.mark.parametrize("dtype,D,n,L", [("bf16", 128, 300, 300), ("fp16", 64, 300, 415), ("bf16", 256, 40, 100),
                                         ("bf16", 128, 16, 200), ("fp32", 64, 100, 100), ("bf16", 64, 120, 120)])
def test_large_rows_that_the_mask_hides(cuda_device, which, up, dtype, D, n, L):
    """Late tokens whose keys or values are 2^up above the others': rows in front of them do not
    see them, and what those get may not depend on them."""
    q, _ = directed(n, 2, D, R.DTYPES[dtype], 5, noise=1.0)
    g = np.random.default_rng(6)
    k, v = g.standard_normal((L, 1, D)), g.standard_normal((L, 1, D))
    for at in (L - 3, L - min(n, 20)):
        x = k if which == "k" else v
        x[at] = np.ldexp(x[at], up)
    run(cuda_device, q, k, v, True, D ** -0.5)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 300), ("fp16", 64, 70), ("bf16", 256, 40), ("bf16", 128, 1)])
def test_keys_and_values_of_every_size(cuda_device, dtype, D, n, causal):
    """Keys over 2^-60 to 1 and values over 2^-30 to 2^8, every row of its own size."""
    q, _ = directed(n, 2, D, R.DTYPES[dtype], 7, noise=1.0)
    g = np.random.default_rng(8)
    k, v = g.standard_normal((500, 2, D)), g.standard_normal((500, 2, D))
    k = np.ldexp(k, g.integers(-60, 1, (500, 2, 1)))
    v = np.ldexp(v, g.integers(-30, 9, (500, 2, 1)))
    run(cuda_device, q, k, v, causal, D ** -0.5)


@pytest.mark.parametrize("order", ["zeros first", "zeros last", "mixed"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype,up", [("bf16", 38), ("bf16", 90), ("fp32", 38), ("fp16", 0)])
def test_zero_values_beside_large_ones(cuda_device, dtype, up, n, order):
    """Value rows of zeros (scale 2^-100) that hold most of the weight beside rows of some 2^up: the
    former count in the sum all the same."""
    L, D = 400, 64
    q, d = directed(n, 1, D, R.DTYPES[dtype], 9, noise=0.05)
    g = np.random.default_rng(10)
    v = np.ldexp(g.standard_normal((L, 1, D)), up)
    at = np.arange(200) if order == "zeros first" else np.arange(200, 400) if order == "zeros last" else \
        g.permutation(L)[:200]
    v[at] = 0.0
    k = 0.1 * g.standard_normal((L, 1, D))
    k[at] += 3.0 / (3.0 * D ** -0.5) * d  # scores of 3 for rows of zeros, of 0 for the others
    run(cuda_device, q, k, v, False, D ** -0.5)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_only_zero_values(cuda_device, dtype, n):
    """9000 value rows of zeros, with scores that lie 5 above the first tile's: out 0, lse finite."""
    L, D = 9000, 64
    q, d = directed(n, 1, D, R.DTYPES[dtype], 11, noise=0.01)
    k = 0.01 * np.random.default_rng(12).standard_normal((L, 1, D))
    k[128:] += 5.0 / (3.0 * D ** -0.5) * d
    run(cuda_device, q, k, np.zeros((L, 1, D)), False, D ** -0.5, ps=128)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("keys", [0.0, 2.0 ** -20, 2.0 ** -60, 1.0])
@pytest.mark.parametrize("queries", [0.0, 2.0 ** -40, 2.0 ** -110])
@pytest.mark.parametrize("dtype,D,n,L", [("bf16", 128, 40, 333), ("bf16", 64, 300, 300), ("fp16", 128, 40, 333),
                                         ("bf16", 256, 40, 70), ("bf16", 128, 300, 333), ("bf16", 128, 1, 70)])
def test_zero_and_tiny_queries(cuda_device, dtype, D, n, L, queries, keys, causal):
    """Rows of padding: the mean of the values that they see."""
    q, _ = directed(n, 2, D, R.DTYPES["fp32"], 13)
    q = (q * queries).to(R.DTYPES[dtype])
    q[n // 2] = 0
    g = np.random.default_rng(14)
    k, v = keys * g.standard_normal((L, 1, D)), g.standard_normal((L, 1, D))
    run(cuda_device, q, k, v, causal, D ** -0.5)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_keys_and_small_queries(cuda_device, dtype, n):
    """Queries of some 2^-115 over keys of some 2^115: scores of ordinary size."""
    q, _ = directed(n, 2, 128, R.DTYPES["fp32"], 15, noise=1.0)
    q = (q * 2.0 ** -115).to(R.DTYPES[dtype])
    g = np.random.default_rng(16)
    k, v = np.ldexp(g.standard_normal((300, 1, 128)), 115), g.standard_normal((300, 1, 128))
    run(cuda_device, q, k, v, True, 128 ** -0.5)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_scores_of_hundreds_of_millions(cuda_device, dtype, n):
    """Three equal keys, far from each other, take all the weight, with scores that 24 bits hold to a
    few units only; their values are of unlike sizes."""
    L, D = 300, 64
    q, d = directed(n, 1, D, R.DTYPES[dtype], 17, size=2e4, noise=0.0)
    g = np.random.default_rng(18)
    c = g.uniform(-1.0, 0.5, L)
    c[[20, 170, 290]] = 1.0
    v = np.ldexp(g.standard_normal((L, 1, D)), g.integers(-2, 3, (L, 1, 1)))
    v[128:256] *= 2.0 ** -8
    run(cuda_device, q, (1e4 * c)[:, None, None] * d, v, False, 1.0, sharp=True)


@pytest.mark.parametrize("kf,vf", [(-0.02, 0.03), (0.02, -0.03), (-0.02, -0.03)])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D,n", [("bf16", 128, 300), ("fp16", 128, 300), ("fp16", 64, 40), ("bf16", 256, 40),
                                       ("bf16", 64, 300), ("bf16", 128, 1), ("fp32", 64, 40), ("fp32", 64, 1)])
def test_negative_static_factors(cuda_device, dtype, D, n, causal, kf, vf):
    """Static factors of either sign, per head."""
    dev, L, ps = cuda_device, 400, 32
    q, _ = directed(n, 2, D, R.DTYPES[dtype], 19, noise=1.0)
    g = np.random.default_rng(20)
    t = R.Table([L], ps)
    page, row = t.rows(0)
    cache, vals = np.full((t.num_pages, 2, ps, 1, D), np.nan), []
    for plane, f in ((0, kf), (1, vf)):
        cache[page, plane, row] = R.e4m3_round(60.0 * g.standard_normal((L, 1, D)))
        vals.append(cache[page, plane, row] * float(np.float32(f)))
    got, lse = hstu_softmax_fwd(q.to(dev), torch.tensor(cache).float().to(R.FP8).to(dev), R.offsets([n]).to(dev),
                                max_seqlen=n, max_seqlen_k=L, causal=causal, alpha=D ** -0.5, return_lse=True,
                                k_descale=torch.full((1, 1), kf, device=dev),
                                v_descale=torch.full((1, 1), vf, device=dev), **t.args(dev))
    check(q, *vals, got, lse, causal, D ** -0.5)


@pytest.mark.parametrize("size", [1e5, 1e7, 1e9])
@pytest.mark.parametrize("dtype,cache,D,n,L", [
    ("bf16", "same", 128, 300, 900), ("bf16", "same", 128, 17, 900), ("bf16", "same", 64, 300, 900),
    ("bf16", "same", 256, 40, 900), ("bf16", "same", 128, 1, 900), ("fp16", "same", 128, 300, 900),
    ("fp16", "same", 64, 20, 900), ("fp32", "same", 64, 40, 900), ("bf16", "e4m3", 128, 300, 900),
    ("fp16", "e4m3", 64, 20, 900), ("bf16", "e4m3", 256, 40, 900), ("bf16", "e4m3", 128, 1, 900)])
def test_scores_beyond_24_bits(cuda_device, dtype, cache, D, n, L, size):
    """Scores of up to some `size`^2 / 10: one key takes all the weight, whatever a product's rounding."""
    dev, dt, ps = cuda_device, R.DTYPES[dtype], 32
    if dt == torch.float16:
        size = min(size, 4e4)
    q, d = directed(n, 1, D, dt, 21, size=size, noise=0.0)
    g = np.random.default_rng(22)
    c = g.uniform(-1.0, 0.5, L)
    c[[20, 170, 700]] = 1.0
    k, v = (size * c)[:, None, None] * d, g.standard_normal((L, 1, D))
    if cache == "e4m3":
        run(dev, q, k, v, False, 0.5, sharp=True)
        return
    t = R.Table([L], ps)
    page, row = t.rows(0)
    rows = torch.full((t.num_pages, 2, ps, 1, D), torch.nan, dtype=dt)
    rows[page, 0, row], rows[page, 1, row] = torch.tensor(k).to(dt), torch.tensor(v).to(dt)
    got, lse = hstu_softmax_fwd(q.to(dev), rows.to(dev), R.offsets([n]).to(dev), max_seqlen=n, max_seqlen_k=L,
                                causal=False, alpha=0.5, return_lse=True, **t.args(dev))
    K, V = (R.values(rows[page, plane, row]) for plane in (0, 1))
    check(q, K, V, got, lse, False, 0.5, sharp=True, weight_bits=8 if dt == torch.bfloat16 else 11)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D,Nq,Nk,n", [
    ("bf16", 128, 4, 2, 300), ("fp16", 64, 4, 2, 300), ("bf16", 256, 2, 2, 40), ("bf16", 64, 4, 1, 30),
    ("fp16", 128, 2, 2, 20), ("bf16", 128, 4, 2, 1), ("fp16", 64, 8, 1, 2), ("fp32", 64, 4, 2, 40),
    ("fp32", 64, 4, 2, 1)])
def test_unlike_sizes_over_many_ctas(cuda_device, dtype, D, Nq, Nk, n, causal):
    """A long sequence whose keys are parted among CTAs: stretches of ordinary rows, of outliers, of zeros
    and of rows of every size, in every order."""
    L = 6100
    q, d = directed(n, Nq, D, R.DTYPES[dtype], 23, noise=1.0)
    g = np.random.default_rng(24)
    k, v = g.standard_normal((L, Nk, D)), g.standard_normal((L, Nk, D))
    at = 0
    while at < L:
        end, kind = at + int(g.integers(1, 400)), g.integers(0, 6)
        if kind == 1:
            v[at:end] = 0.0
        elif kind == 2:
            v[at:end] = np.ldexp(v[at:end], g.integers(-24, 9, v[at:end].shape[:2])[..., None])
        elif kind == 3:
            k[at:end] = np.ldexp(k[at:end], g.integers(-40, 2, k[at:end].shape[:2])[..., None])
        elif kind == 4:
            v[at] = np.ldexp(v[at], 12)
            k[at, 0] = -30.0 / (3.0 * D ** -0.5) * d
        elif kind == 5:
            k[at:end] = v[at:end] = 0.0
        at = end
    run(cuda_device, q, k, v, causal, D ** -0.5, ps=128)


@pytest.mark.parametrize("ahead", [5.0, 15.0, 40.0])
@pytest.mark.parametrize("zeros", ["one", "many", "tile"])
@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("fp16", 64), ("bf16", 256), ("fp32", 64)])
def test_zero_values_with_nearly_all_the_weight(cuda_device, dtype, D, n, zeros, ahead):
    """Value rows of zeros whose scores lie far above the others': what the others give keeps its bits."""
    L = 500
    q, d = directed(n, 1, D, R.DTYPES[dtype], 25, noise=0.05)
    g = np.random.default_rng(26)
    k, v = 0.3 * g.standard_normal((L, 1, D)), g.standard_normal((L, 1, D))
    at = {"one": [200], "many": g.permutation(L)[:150], "tile": np.arange(128, 256)}[zeros]
    v[at] = 0.0
    k[at] += ahead / (3.0 * D ** -0.5) * d
    run(cuda_device, q, k, v, False, D ** -0.5, ps=128)
