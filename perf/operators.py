"""Cases of the paged KV cache operators: writing new rows (quantising them to E4M3 where the
cache holds it), reading a sequence's rows back, and softmax attention of a chunk of new tokens
over the cache.

The cache is the one that hstu_fwd reads: kv_cache [num_pages, 2, page_size, Nk, D] (plane 0
keys, plane 1 values) with page_offsets [B+1], page_ids and last_page_len [B]. A sequence's
length Lk is (pages - 1) * page_size + last_page_len, or 0 without pages. The n new rows of a
sequence (seq_offsets) are its last n positions.

E4M3 caches with kv_scale [num_pages, 2, Nk, page_size] (uint8): the value of an element is
code * 2^(kv_scale - 127), where 2^e is the smallest power of two that brings the largest
magnitude of the row (D values of one head) to 448 or less, and e at least -100.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = torch.float8_e4m3fn
EXP_MIN = -100


def listed():
    base = {"dtype": "bf16", "cache": "same", "D": 128, "page": 128, "index": "int64", "strided": False, "mix": 1}
    attn = {"op": "attn", **base, "causal": True}
    append = {"op": "append", **base, "cache": "e4m3", "strided": True}
    read = {"op": "read", **base, "whole": True}
    return [
        # one user's next token after a short history: latency
        {"name": "attn_one_token", **attn, "B": 1, "Nq": 8, "Nk": 2, "hist_lo": 900, "hist_hi": 900, "new_lo": 1, "new_hi": 1},
        # a batch that generates one token per sequence from E4M3 caches
        {"name": "attn_tokens_e4m3", **attn, "cache": "e4m3", "index": "int32", "B": 128, "Nq": 16, "Nk": 4,
         "hist_lo": 1024, "hist_hi": 4096, "new_lo": 1, "new_hi": 1},
        # one token each for four very long histories: few rows, many keys
        {"name": "attn_tokens_long", **attn, "page": 256, "B": 4, "Nq": 8, "Nk": 2,
         "hist_lo": 90000, "hist_hi": 120000, "new_lo": 1, "new_hi": 1},
        # the candidates of a ranking batch over cached histories, each seeing all of them (no GQA)
        {"name": "attn_candidates", **attn, "causal": False, "B": 128, "Nq": 4, "Nk": 4,
         "hist_lo": 1024, "hist_hi": 4096, "new_lo": 32, "new_hi": 256},
        # chunks of new tokens over E4M3 caches, q a slice of a fused projection
        {"name": "attn_chunk_e4m3", **attn, "cache": "e4m3", "strided": True, "B": 16, "Nq": 8, "Nk": 2,
         "hist_lo": 500, "hist_hi": 8000, "new_lo": 100, "new_hi": 512},
        # a long prompt's second half: the largest case, bound by the products
        {"name": "attn_prefill", **attn, "B": 4, "Nq": 16, "Nk": 4, "hist_lo": 4096, "hist_hi": 4096, "new_lo": 4096, "new_hi": 4096},
        # fp16, head dim 64, three query heads to a key head, ragged chunks, sequences without a history or a row
        {"name": "attn_ragged_fp16", **attn, "dtype": "fp16", "D": 64, "page": 32, "index": "int32", "B": 24, "Nq": 12, "Nk": 4,
         "hist_lo": 0, "hist_hi": 1500, "new_lo": 0, "new_hi": 333},
        # fp32: a verification run of a small model
        {"name": "attn_fp32", **attn, "dtype": "fp32", "D": 64, "page": 32, "B": 3, "Nq": 4, "Nk": 2,
         "hist_lo": 0, "hist_hi": 400, "new_lo": 17, "new_hi": 65},
        # one new token per sequence written to E4M3 caches: latency
        {"name": "append_tokens_e4m3", **append, "B": 128, "Nk": 4, "hist_lo": 1024, "hist_hi": 4096, "new_lo": 1, "new_hi": 1},
        # prompts written to E4M3 caches from slices of a fused projection: bandwidth
        {"name": "append_prompts_e4m3", **append, "B": 32, "Nk": 8, "hist_lo": 0, "hist_hi": 100, "new_lo": 500, "new_hi": 4000},
        # the short histories of a few users read back: latency
        {"name": "read_small", **read, "dtype": "fp16", "page": 32, "D": 64, "B": 5, "Nk": 2,
         "hist_lo": 0, "hist_hi": 300, "new_lo": 1, "new_hi": 40},
        # the E4M3 histories of a ranking batch read back as bf16: bandwidth
        {"name": "read_e4m3", **read, "cache": "e4m3", "B": 128, "Nk": 4, "hist_lo": 1024, "hist_hi": 4096, "new_lo": 32, "new_hi": 256},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, Nk = rng.choice(["attn", "attn", "attn", "append", "read"]), rng.choice([1, 2, 4, 8])
    hist = rng.choice([_spread(rng, 1, 100), _spread(rng, 100, 8000), _spread(rng, 8000, 120000)])
    new = rng.choice([1, _spread(rng, 2, 16), _spread(rng, 17, 300), _spread(rng, 300, 4096)])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"]), "cache": rng.choice(["same", "e4m3"]),
            "D": rng.choice([64, 128, 128, 256, 16 * rng.randint(1, 16)]), "page": rng.choice([32, 128, 256]),
            "index": rng.choice(["int32", "int64"]), "strided": rng.random() < 0.4, "mix": rng.randrange(1 << 20),
            "B": _spread(rng, 1, 160), "Nk": Nk, "hist_lo": rng.choice([0, hist // 4, hist]), "hist_hi": hist,
            "new_lo": rng.choice([0, new, new]), "new_hi": new}
    if op == "attn":
        case |= {"Nq": Nk * rng.choice([1, 2, 3, 4, 5, 8, 16]), "causal": rng.random() < 0.75}
    elif op == "read":
        case["whole"] = rng.random() < 0.8
    # at most the cost of the operator's largest listed case (for fp32 attention, a fifth of it)
    while True:
        keys = case["B"] * (case["hist_hi"] + case["new_hi"])
        scores = case.get("Nq", 0) * case["new_hi"] * keys
        fp32 = op == "attn" and case["dtype"] == "fp32"
        if keys * Nk * case["D"] <= (1e8 if fp32 else 2.5e8) and scores <= (2e8 if fp32 else 2e9) and scores * case["D"] <= 2.5e11:
            return case
        if case["B"] > 1:
            case["B"] //= 2
        else:
            case |= {k: case[k] // 2 for k in ("hist_lo", "hist_hi", "new_lo")} | {"new_hi": max(1, case["new_hi"] // 2)}


def _lengths(case):
    """Rows in the cache before the new ones, and new rows, of each sequence."""
    rng = random.Random(case["mix"])
    return [[rng.randint(case[k + "_lo"], case[k + "_hi"]) for _ in range(case["B"])] for k in ("hist", "new")]


def work(case):
    hist, new = _lengths(case)
    size = TYPES[case["dtype"]].itemsize
    row = case["Nk"] * (case["D"] + 1) if case["cache"] == "e4m3" else case["Nk"] * case["D"] * size  # of one plane of the cache
    cached, added = sum(hist) + sum(new), sum(new)
    if case["op"] == "append":
        return {"bytes": 2 * added * (case["Nk"] * case["D"] * size + row), "flops": 0}
    if case["op"] == "read":
        return {"bytes": 2 * (cached if case["whole"] else added) * (case["Nk"] * case["D"] * size + row), "flops": 0}
    pairs = sum(n * (h + n) - (n * (n - 1) // 2 if case["causal"] else 0) for h, n in zip(hist, new))
    seen = sum(h + n for h, n in zip(hist, new) if n)
    return {"bytes": 2 * added * case["Nq"] * case["D"] * size + 2 * seen * row, "flops": 4 * case["D"] * case["Nq"] * pairs}


def _quantise(x):
    """Codes and biased exponents of rows x [..., D]."""
    x = x.float()
    fraction, exponent = torch.frexp(x.abs().amax(-1))  # fraction in [0.5, 1); 448 is 0.875 * 2^9
    e = torch.where(fraction > 0.875, exponent - 8, exponent - 9)
    e = torch.where(fraction == 0, EXP_MIN, e).clamp(min=EXP_MIN).to(torch.int32)
    inverse = ((127 - e) << 23).view(torch.float32)  # 2^-e
    return (x * inverse[..., None]).clamp(-448, 448).to(FP8), (e + 127).to(torch.uint8)


def _scale(kv_scale):
    """2^(kv_scale - 127)."""
    return (kv_scale.to(torch.int32) << 23).view(torch.float32)


def _power(e):
    """2^e in 64 bits (torch.pow is a rounding off, which would move ties)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


class _State:
    pass


def prepare(case, seed):
    s, dev, dt = _State(), "cuda", TYPES[case["dtype"]]
    g = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    index = getattr(torch, case["index"])
    hist, new = (torch.tensor(x) for x in _lengths(case))
    Nk, D, ps, Nq = case["Nk"], case["D"], case["page"], case.get("Nq", 2 * case["Nk"])
    s.case, length = case, hist + new
    pages = (length + ps - 1) // ps
    total = int(pages.sum())

    def offsets(n):
        return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)]).to(dev, index)

    s.page_offsets = offsets(pages)
    s.page_ids = torch.randperm(total + 4, generator=host)[:total].to(dev, index)  # four pages belong to no sequence
    s.last_page_len = torch.where(pages > 0, length - (pages - 1) * ps, 1).to(dev, index)
    s.seq_offsets = offsets(length if case.get("whole") else new)
    s.rows = int((length if case.get("whole") else new).sum())
    s.max_seqlen, s.max_seqlen_k = max(1, int(new.max())), max(1, int(length.max()))
    s.alpha = 1.0 / math.sqrt(D)
    # rows of unlike sizes, as the keys and values of a model have
    values = torch.randn(total + 4, 2, ps, Nk, D, generator=g, device=dev, dtype=dt)
    values *= torch.exp2(torch.randn(total + 4, 2, ps, Nk, 1, generator=g, device=dev, dtype=dt) * 0.5)
    s.kv_scale = None
    if case["cache"] == "e4m3":
        s.kv_cache, scale = _quantise(values)
        s.kv_scale = scale.transpose(2, 3).contiguous()
    else:
        s.kv_cache = values.to(dt)
    # a fused projection's rows [T, Nq + 2 Nk, D], or tensors of their own
    fused = torch.randn(int(new.sum()), Nq + 2 * Nk, D, generator=g, device=dev).to(dt)
    s.q, s.k, s.v = fused[:, :Nq], fused[:, Nq:Nq + Nk], fused[:, Nq + Nk:]
    if not case["strided"]:
        s.q, s.k, s.v = (x.contiguous() for x in (s.q, s.k, s.v))
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"attn": _attn, "append": _append, "read": _read}[s.case["op"]](s)


def _run_own(s):
    import hstu_dense_forward_gb300 as hstu
    table = dict(page_offsets=s.page_offsets, page_ids=s.page_ids, last_page_len=s.last_page_len, kv_scale=s.kv_scale)
    if s.case["op"] == "append":
        hstu.hstu_kv_append(s.k, s.v, s.seq_offsets, s.kv_cache, **table)
        return {"kv_cache": s.kv_cache, "kv_scale": s.kv_scale}
    if s.case["op"] == "read":
        k, v = hstu.hstu_kv_read(s.kv_cache, s.seq_offsets, total_tokens=s.rows, dtype=TYPES[s.case["dtype"]], **table)
        return {"k": k, "v": v}
    return {"out": hstu.hstu_softmax_fwd(s.q, s.kv_cache, s.seq_offsets, max_seqlen=s.max_seqlen, max_seqlen_k=s.max_seqlen_k,
                                         causal=s.case["causal"], alpha=s.alpha, **table)}


def _sequence_lengths(s):
    pages = s.page_offsets.diff()
    return torch.where(pages > 0, (pages - 1) * s.case["page"] + s.last_page_len, 0)


def _places(s, rows):
    """Sequence, page and row in the page of the rows 0 .. rows - 1 that seq_offsets counts."""
    t = torch.arange(rows, device="cuda", dtype=s.seq_offsets.dtype)
    b = torch.searchsorted(s.seq_offsets, t, right=True) - 1
    position = _sequence_lengths(s)[b] - s.seq_offsets[b + 1] + t
    return b, s.page_ids[s.page_offsets[b] + position // s.case["page"]].long(), position % s.case["page"]


def _append(s):
    _, page, row = _places(s, s.rows)
    for plane, x in ((0, s.k), (1, s.v)):
        if s.kv_scale is None:
            s.kv_cache[page, plane, row] = x
        else:
            codes, scale = _quantise(x)
            s.kv_cache.view(torch.uint8)[page, plane, row] = codes.view(torch.uint8)
            s.kv_scale[page, plane, :, row] = scale
    return {"kv_cache": s.kv_cache, "kv_scale": s.kv_scale}


def _gather(s, page, plane, row):
    """The rows of one plane, in 32 bits."""
    if s.kv_scale is None:
        return s.kv_cache[page, plane, row].float()
    codes = s.kv_cache.view(torch.uint8)[page, plane, row].view(FP8).float()
    return codes * _scale(s.kv_scale[page, plane, :, row])[..., None]


def _read(s):
    _, page, row = _places(s, s.rows)
    dt = TYPES[s.case["dtype"]]
    return {"k": _gather(s, page, 0, row).to(dt), "v": _gather(s, page, 1, row).to(dt)}


def _attn(s):
    ps, Nq, Nk, D = s.case["page"], s.case["Nq"], s.case["Nk"], s.case["D"]
    B, Lq, Lk, G = s.case["B"], s.max_seqlen, s.max_seqlen_k, Nq // Nk
    if not s.rows:
        return {"out": torch.empty_like(s.q)}
    length, n = _sequence_lengths(s)[:, None], s.seq_offsets.diff()[:, None]
    i, j = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    real = j < length  # [B, Lk]
    slot = (s.page_offsets[:-1, None] + j // ps).clamp(max=s.page_ids.numel() - 1)
    page, row = s.page_ids[slot].long(), (j % ps).expand(B, Lk)
    K, V = (_gather(s, page, plane, row).masked_fill_(~real[..., None, None], 0).permute(0, 2, 1, 3) for plane in (0, 1))
    Q = s.q[(s.seq_offsets[:-1, None] + i).clamp(max=s.rows - 1).long()].float()  # [B, Lq, Nq, D]
    Q = Q.view(B, Lq, Nk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Nk, G * Lq, D)
    x = torch.matmul(Q, K.transpose(2, 3)).mul_(s.alpha).view(B, Nk, G, Lq, Lk)
    seen = real[:, None, :] & ((j <= length[:, None] - n[:, None] + i[:, None]) | (not s.case["causal"]))  # [B, Lq, Lk]
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill_(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Nk, G * Lq, Lk), V).view(B, Nk, G, Lq, D) / total.masked_fill_(total == 0, 1)
    b = torch.searchsorted(s.seq_offsets, torch.arange(s.rows, device="cuda", dtype=s.seq_offsets.dtype), right=True) - 1
    t = torch.arange(s.rows, device="cuda") - s.seq_offsets[b]
    return {"out": o.permute(0, 3, 1, 2, 4)[b, t].reshape(s.rows, Nq, D).to(s.q.dtype)}


def _sequence(s, b):
    """Keys and values [Lk, Nk, D] of sequence b in 64 bits, and the pages and rows that hold them."""
    ps, first, last = s.case["page"], int(s.page_offsets[b]), int(s.page_offsets[b + 1])
    length = (last - first - 1) * ps + int(s.last_page_len[b]) if last > first else 0
    ids = s.page_ids[first:last].long()
    planes = []
    for plane in (0, 1):
        x = s.kv_cache[ids, plane] if s.kv_scale is None else s.kv_cache.view(torch.uint8)[ids, plane].view(FP8)
        x = x.to(torch.float64)
        if s.kv_scale is not None:
            x = x * _power(s.kv_scale[ids, plane].to(torch.int64) - 127).transpose(1, 2)[..., None]
        planes.append(x.flatten(0, 1)[:length])
    return planes, ids, length


def exact(case, seed):
    s = prepare(case, seed)
    ends = [int(x) for x in s.seq_offsets]
    if case["op"] == "read":
        k, v = (torch.zeros(s.rows, case["Nk"], case["D"], dtype=torch.float64, device="cuda") for _ in range(2))
        for b in range(case["B"]):
            (K, V), _, length = _sequence(s, b)
            n = ends[b + 1] - ends[b]
            k[ends[b]:ends[b + 1]], v[ends[b]:ends[b + 1]] = K[length - n:], V[length - n:]
        return {"k": k, "v": v}
    if case["op"] == "append":
        cache = s.kv_cache.to(torch.float64)
        for b in range(case["B"]):
            _, ids, length = _sequence(s, b)
            n = ends[b + 1] - ends[b]
            at = torch.arange(length - n, length, device="cuda")
            for plane, new in ((0, s.k), (1, s.v)):
                x = new[ends[b]:ends[b + 1]].to(torch.float64)
                if s.kv_scale is not None:
                    largest = x.abs().amax(-1, keepdim=True).clamp(min=448 * 2.0 ** EXP_MIN)
                    e = torch.ceil(torch.log2(largest / 448))
                    e = torch.where(largest > 448 * _power(e), e + 1, e)  # log2 rounds too
                    e = torch.where(largest <= 448 * _power(e - 1), e - 1, e).clamp(min=EXP_MIN)
                    x = x / _power(e)
                    # E4M3 has three bits below the leading one, and 2^-9 below 2^-6
                    step = _power(torch.frexp(x.abs().clamp(min=2.0 ** -6)).exponent - 4)
                    x = torch.round(x / step) * step
                cache[ids[at // case["page"]], plane, at % case["page"]] = x
        return {"kv_cache": cache, "kv_scale": None}
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    G = case["Nq"] // case["Nk"]
    for b in range(case["B"]):
        (K, V), _, length = _sequence(s, b)
        n = ends[b + 1] - ends[b]
        j = torch.arange(length, device="cuda")
        for h in range(case["Nq"]):
            for i0 in range(0, n, 2048):
                i = torch.arange(i0, min(n, i0 + 2048), device="cuda")
                x = s.alpha * (s.q[ends[b] + i, h].to(torch.float64) @ K[:, h // G].T)
                if case["causal"]:
                    x = torch.where(j[None, :] <= (length - n + i)[:, None], x, -math.inf)
                out[ends[b] + i, h] = torch.softmax(x, -1) @ V[:, h // G]
    return {"out": out}
