"""Cases of the operators that let a paged KV cache hold longer histories: caches of 4-bit values
(written, read back, attended over with a softmax), the attention weight that every cached key has
received, and the eviction of the keys that received least.

The page table is the one of the other cache operators: page_offsets [B+1], page_ids and
last_page_len [B]; a sequence's length Lk is (pages - 1) * page_size + last_page_len, or 0 without
pages, and the n new rows of a sequence (seq_offsets) are its last n positions.

4-bit caches: kv_cache [num_pages, 2, Nk, page_size, D / 2] holds E2M1 codes, element 2 i in the low
half of byte i; kv_group_scale [num_pages, 2, Nk, page_size, D / 16] one E4M3 factor per sixteen
elements; kv_scale [num_pages, 2, Nk, page_size] (uint8) a power of two per row and head. The value of
an element is 2^(kv_scale - 127) * factor * code. e is the smallest exponent, at least -100, for which
the row's largest magnitude is 2688 * 2^e or less (448 * 6, both formats' largest); a factor is a
sixth of its elements' largest magnitude over 2^e rounded to E4M3, a code the element over 2^e and
the factor rounded to E2M1 (nearest, ties to even, 6 at most).

The weight of key j of kv head hk is the sum of exp(alpha q k_j - lse) over the queries and their
heads of hk that see j, in weights [num_pages, Nk, page_size]. Eviction keeps, of every sequence and
kv head, min(Lk, budget) rows: the `recent` last, and those of the largest weights among the others
(of equal ones the earlier), in the order in which they were, as the sequence's first rows.
"""
import math
import random

import torch

own = False

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
FP8 = torch.float8_e4m3fn
EXP_MIN = -100
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    base = {"dtype": "bf16", "cache": "fp4", "D": 128, "page": 128, "index": "int64", "strided": False, "mix": 1}
    attn = {"op": "attn", **base, "causal": True}
    append = {"op": "append", **base, "strided": True}
    read = {"op": "read", **base}
    weights = {"op": "weights", **base, "causal": True, "accumulate": True}
    evict = {"op": "evict", **base, "cache": "same", "new_lo": 0, "new_hi": 0}
    return [
        # one user's next token after a short history: latency
        {"name": "attn_one_token_fp4", **attn, "B": 1, "Nq": 8, "Nk": 2, "hist_lo": 900, "hist_hi": 900, "new_lo": 1, "new_hi": 1},
        # a batch that generates one token per sequence
        {"name": "attn_tokens_fp4", **attn, "index": "int32", "B": 128, "Nq": 16, "Nk": 4,
         "hist_lo": 1024, "hist_hi": 4096, "new_lo": 1, "new_hi": 1},
        # chunks of new tokens, q a slice of a fused projection
        {"name": "attn_chunk_fp4", **attn, "strided": True, "B": 16, "Nq": 8, "Nk": 2,
         "hist_lo": 500, "hist_hi": 8000, "new_lo": 100, "new_hi": 512},
        # one new token per sequence written, and read as the cache now holds it: latency
        {"name": "append_tokens_fp4", **append, "B": 128, "Nk": 4, "hist_lo": 1024, "hist_hi": 4096, "new_lo": 1, "new_hi": 1},
        # prompts written from slices of a fused projection, and read as the cache now holds them (so that
        # the layer's own attention sees what later steps will see): bandwidth
        {"name": "append_prompts_fp4", **append, "B": 32, "Nk": 8, "hist_lo": 0, "hist_hi": 100, "new_lo": 500, "new_hi": 4000},
        # the short histories of a few users read back: latency
        {"name": "read_small_fp4", **read, "dtype": "fp16", "page": 32, "D": 64, "B": 5, "Nk": 2,
         "hist_lo": 0, "hist_hi": 300, "new_lo": 1, "new_hi": 40},
        # the histories of a ranking batch read back as bf16: bandwidth
        {"name": "read_fp4", **read, "B": 128, "Nk": 4, "hist_lo": 1024, "hist_hi": 4096, "new_lo": 32, "new_hi": 256},
        # while a batch generates: each step's token adds its weights, over E4M3 caches
        {"name": "weights_tokens_e4m3", **weights, "cache": "e4m3", "index": "int32", "B": 128, "Nq": 16, "Nk": 4,
         "hist_lo": 1024, "hist_hi": 4096, "new_lo": 1, "new_hi": 1},
        # the last tokens of long prompts decide what is kept of them
        {"name": "weights_window", **weights, "cache": "same", "accumulate": False, "B": 8, "Nq": 8, "Nk": 2,
         "hist_lo": 4000, "hist_hi": 16000, "new_lo": 64, "new_hi": 64},
        # every token of long prompts adds its weights: the largest case, bound by products and exponentials
        {"name": "weights_prompt", **weights, "cache": "same", "B": 4, "Nq": 16, "Nk": 4, "hist_lo": 0, "hist_hi": 0, "new_lo": 4096, "new_hi": 4096},
        # a few short histories shortened, fp16, small pages: latency
        {"name": "evict_small", **evict, "dtype": "fp16", "page": 32, "D": 64, "index": "int32", "B": 5, "Nk": 2,
         "hist_lo": 0, "hist_hi": 300, "budget": 100, "recent": 16},
        # the long histories of a batch halved or more: bandwidth
        {"name": "evict_histories", **evict, "B": 32, "Nk": 4, "hist_lo": 4096, "hist_hi": 16000, "budget": 4096, "recent": 256},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, Nk = rng.choice(["attn", "attn", "append", "read", "weights", "weights", "evict", "evict"]), rng.choice([1, 2, 4, 8])
    hist = rng.choice([_spread(rng, 1, 100), _spread(rng, 100, 8000), _spread(rng, 8000, 100000)])
    new = rng.choice([1, _spread(rng, 2, 16), _spread(rng, 17, 300), _spread(rng, 300, 4096)])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp16", "fp32"]), "cache": "fp4",
            "D": rng.choice([64, 128, 128, 256, 32 * rng.randint(1, 8)]), "page": rng.choice([32, 128, 256]),
            "index": rng.choice(["int32", "int64"]), "strided": rng.random() < 0.4, "mix": rng.randrange(1 << 20),
            "B": _spread(rng, 1, 160), "Nk": Nk, "hist_lo": rng.choice([0, hist // 4, hist]), "hist_hi": hist,
            "new_lo": rng.choice([0, new, new]), "new_hi": new}
    if op in ("weights", "evict"):
        case["cache"] = rng.choice(["same", "e4m3", "fp4"])
        if case["cache"] != "fp4" and rng.random() < 0.3:
            case["D"] = 16 * rng.randint(1, 16)
    if op in ("attn", "weights"):
        case |= {"Nq": Nk * rng.choice([1, 2, 3, 4, 5, 8, 16]), "causal": rng.random() < 0.75}
    if op == "weights":
        case["accumulate"] = rng.random() < 0.7
    if op == "evict":
        case |= {"new_lo": 0, "new_hi": 0, "budget": _spread(rng, max(1, hist // 8), hist)}
        case["recent"] = rng.choice([0, rng.randint(0, case["budget"]), _spread(rng, 1, 64)])
    # at most the cost of the operator's largest listed case (for fp32 products, a fifth of it)
    while True:
        keys = case["B"] * (case["hist_hi"] + case["new_hi"])
        scores = case.get("Nq", 0) * case["new_hi"] * keys
        fp32 = case["dtype"] == "fp32" and "Nq" in case
        if keys * Nk * case["D"] <= (5e7 if fp32 else 1.5e8) and scores <= (2e8 if fp32 else 1e9) and scores * case["D"] <= 1.2e11:
            break
        if case["B"] > 1:
            case["B"] //= 2
        else:
            case |= {k: case[k] // 2 for k in ("hist_lo", "hist_hi", "new_lo")} | {"new_hi": max(min(1, case["new_hi"]), case["new_hi"] // 2)}
    part = "hist" if op == "evict" else "new"
    if not any(_lengths(case)[op != "evict"]):  # some sequence has rows
        case[part + "_lo"] = case[part + "_hi"] = max(1, case[part + "_hi"])
    return case


def _lengths(case):
    """Rows in the cache before the new ones, and new rows, of each sequence."""
    rng = random.Random(case["mix"])
    return [[rng.randint(case[k + "_lo"], case[k + "_hi"]) for _ in range(case["B"])] for k in ("hist", "new")]


def work(case):
    hist, new = _lengths(case)
    size, Nk, D = TYPES[case["dtype"]].itemsize, case["Nk"], case["D"]
    # bytes of one row, in one plane of the cache and in a tensor
    cached = Nk * {"same": D * size, "e4m3": D + 1, "fp4": D // 2 + D // 16 + 1}[case["cache"]]
    plain = Nk * D * size
    lengths = 3 * case["B"] * (4 if case["index"] == "int32" else 8)
    if case["op"] == "append":
        return {"bytes": lengths + 2 * sum(new) * (2 * plain + cached), "flops": 0}
    if case["op"] == "read":
        return {"bytes": lengths + 2 * (sum(hist) + sum(new)) * (plain + cached), "flops": 0}
    if case["op"] == "evict":
        moved = sum(case["budget"] for h in hist if h > case["budget"])
        return {"bytes": lengths + 4 * Nk * (sum(hist) + case["B"] * case["budget"]) + 2 * 2 * moved * cached, "flops": 0}
    pairs = sum(n * (h + n) - (n * (n - 1) // 2 if case["causal"] else 0) for h, n in zip(hist, new))
    seen = sum(h + n for h, n in zip(hist, new) if n)
    queries = sum(new) * case["Nq"]
    if case["op"] == "attn":
        return {"bytes": lengths + 2 * queries * D * size + 2 * seen * cached, "flops": 4 * D * case["Nq"] * pairs}
    return {"bytes": lengths + queries * (D * size + 4) + seen * (cached + Nk * (8 if case["accumulate"] else 4)), "flops": 2 * D * case["Nq"] * pairs}


def _power(e, dtype=torch.float32):
    """2^e (torch.pow is a rounding off, which would move ties)."""
    if dtype is torch.float32:
        return ((e.to(torch.int32) + 127) << 23).view(torch.float32)
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exponent(x, largest):
    """The smallest e >= EXP_MIN for which the largest magnitude of rows x is largest * 2^e or less."""
    fraction, exponent = torch.frexp(x.abs().amax(-1))  # fraction in [0.5, 1)
    top, log = math.frexp(largest)
    e = torch.where(fraction > top, exponent - log + 1, exponent - log)
    return torch.where(fraction == 0, EXP_MIN, e).clamp(min=EXP_MIN).to(torch.int32)


def _quantise8(x):
    """E4M3 codes and biased exponents of rows x [..., D]."""
    x = x.float()
    e = _exponent(x, 448.0)
    return (x * _power(-e)[..., None]).clamp(-448, 448).to(FP8), (e + 127).to(torch.uint8)


def _quantise4(x):
    """Packed E2M1 codes, E4M3 factors and biased exponents of rows x [..., D]."""
    x = x.float()
    e = _exponent(x, 2688.0)
    x = (x * _power(-e)[..., None]).unflatten(-1, (-1, 16))
    group = (x.abs().amax(-1) / 6).to(FP8)
    m = x.abs() / group.float()[..., None]  # (a factor of 0: its elements become 0)
    m.masked_fill_(group.float()[..., None] == 0, 0)
    code = (m > 0.25).to(torch.uint8)
    for middle in (m >= 0.75, m > 1.25, m >= 1.75, m > 2.5, m >= 3.5, m > 5):
        code += middle
    code = (code + 8 * (x < 0).to(torch.uint8)).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, group, (e + 127).to(torch.uint8)


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
    s.page_ids = torch.randperm(total + 4, generator=host)[:max(1, total)].to(dev, index)  # four pages belong to no sequence
    s.last_page_len = torch.where(pages > 0, length - (pages - 1) * ps, 1).to(dev, index)
    whole = case["op"] == "read"
    s.seq_offsets = offsets(length if whole else new)
    s.rows = int((length if whole else new).sum())
    s.max_seqlen, s.max_seqlen_k = max(1, int(new.max())), max(1, int(length.max()))
    s.alpha = 1.0 / math.sqrt(D)
    s.e2m1 = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=dev)
    # rows of unlike sizes, as the keys and values of a model have
    values = torch.randn(total + 4, 2, ps, Nk, D, generator=g, device=dev, dtype=dt)
    values *= torch.exp2(torch.randn(total + 4, 2, ps, Nk, 1, generator=g, device=dev, dtype=dt) * 0.5)
    s.kv_scale = s.kv_group_scale = None
    if case["cache"] == "e4m3":
        s.kv_cache, scale = _quantise8(values)
        s.kv_scale = scale.transpose(2, 3).contiguous()
    elif case["cache"] == "fp4":
        s.kv_cache, s.kv_group_scale, s.kv_scale = _quantise4(values.transpose(2, 3).contiguous())
    else:
        s.kv_cache = values
    # a fused projection's rows [T, Nq + 2 Nk, D], or tensors of their own
    fused = torch.randn(int(new.sum()), Nq + 2 * Nk, D, generator=g, device=dev).to(dt)
    s.q, s.k, s.v = fused[:, :Nq], fused[:, Nq:Nq + Nk], fused[:, Nq + Nk:]
    if not case["strided"]:
        s.q, s.k, s.v = (x.contiguous() for x in (s.q, s.k, s.v))
    if case["op"] in ("weights", "evict"):
        # what earlier steps have added up: a few keys have most of it, some nothing
        w = torch.randn(total + 4, Nk, ps, generator=g, device=dev).mul_(2).exp_()
        s.weights = w.masked_fill_(torch.rand(total + 4, Nk, ps, generator=g, device=dev) < 0.05, 0)
    if case["op"] == "weights":
        s.lse = _lse(s)  # the step's attention has returned it
    if case["op"] == "evict":
        s.kept_offsets = offsets(length.clamp(max=case["budget"]))
        s.kept_rows = int(s.kept_offsets[-1])
    return s


def run(s):
    if own:
        return _run_own(s)
    return {"attn": _attn, "append": _append, "read": _read, "weights": _weights, "evict": _evict}[s.case["op"]](s)


def _run_own(s):
    import hstu_dense_forward_gb300 as hstu
    case = s.case
    table = dict(page_offsets=s.page_offsets, page_ids=s.page_ids, last_page_len=s.last_page_len)
    scales = dict(kv_scale=s.kv_scale, kv_group_scale=s.kv_group_scale)
    if case["op"] in ("append", "read"):
        if case["op"] == "append":
            hstu.hstu_kv_append(s.k, s.v, s.seq_offsets, s.kv_cache, **table, **scales)
        k, v = hstu.hstu_kv_read(s.kv_cache, s.seq_offsets, total_tokens=s.rows, dtype=TYPES[case["dtype"]], **table, **scales)
        return {"k": k, "v": v}
    if case["op"] == "attn":
        return {"out": hstu.hstu_softmax_fwd(s.q, s.kv_cache, s.seq_offsets, max_seqlen=s.max_seqlen, max_seqlen_k=s.max_seqlen_k,
                                             causal=case["causal"], alpha=s.alpha, **table, **scales)}
    if case["op"] == "weights":
        return {"weights": hstu.hstu_kv_weights(s.q, s.lse, s.kv_cache, s.seq_offsets, s.weights, max_seqlen=s.max_seqlen,
                                                max_seqlen_k=s.max_seqlen_k, causal=case["causal"], alpha=s.alpha,
                                                accumulate=case["accumulate"], **table, **scales)}
    kept, shorter = hstu.hstu_kv_select(s.weights, budget=case["budget"], recent=case["recent"], max_seqlen_k=s.max_seqlen_k, **table)
    hstu.hstu_kv_compact(s.kv_cache, kept, **table, **scales)
    out = {"kept": kept, **shorter}
    if case["cache"] == "fp4":
        out["k"], out["v"] = hstu.hstu_kv_read(s.kv_cache, s.kept_offsets, total_tokens=s.kept_rows, dtype=TYPES[case["dtype"]], **shorter, **scales)
    else:
        out |= {"kv_cache": s.kv_cache, "kv_scale": s.kv_scale}
    return out


def _sequence_lengths(s):
    pages = s.page_offsets.diff()
    return torch.where(pages > 0, (pages - 1) * s.case["page"] + s.last_page_len, 0)


def _places(s, rows):
    """Sequence, page and row in the page of the rows 0 .. rows - 1 that seq_offsets counts."""
    t = torch.arange(rows, device="cuda", dtype=s.seq_offsets.dtype)
    b = torch.searchsorted(s.seq_offsets, t, right=True) - 1
    position = _sequence_lengths(s)[b] - s.seq_offsets[b + 1] + t
    return b, s.page_ids[s.page_offsets[b] + position // s.case["page"]].long(), position % s.case["page"]


def _all_places(s):
    """Page and row in the page of the positions 0 .. max_seqlen_k - 1 of every sequence [B, Lk], and whether it has them."""
    j = torch.arange(s.max_seqlen_k, device="cuda")
    slot = (s.page_offsets[:-1, None] + j // s.case["page"]).clamp(max=s.page_ids.numel() - 1)
    return s.page_ids[slot].long(), (j % s.case["page"]).expand(slot.shape), j < _sequence_lengths(s)[:, None]


def _append(s):
    _, page, row = _places(s, s.rows)
    for plane, x in ((0, s.k), (1, s.v)):
        codes, group, scale = _quantise4(x)
        s.kv_cache[page, plane, :, row] = codes
        s.kv_group_scale.view(torch.uint8)[page, plane, :, row] = group.view(torch.uint8)
        s.kv_scale[page, plane, :, row] = scale
    return _read(s)


def _gather(s, page, plane, row):
    """The rows of one plane, in 32 bits."""
    if s.case["cache"] == "same":
        return s.kv_cache[page, plane, row].float()
    scale = _power(s.kv_scale[page, plane, :, row].to(torch.int32) - 127)[..., None]
    if s.case["cache"] == "e4m3":
        return s.kv_cache.view(torch.uint8)[page, plane, row].view(FP8).float() * scale
    codes = s.kv_cache[page, plane, :, row].to(torch.int32)
    values = s.e2m1[torch.stack([codes & 15, codes >> 4], -1).flatten(-2)].unflatten(-1, (-1, 16))
    group = s.kv_group_scale.view(torch.uint8)[page, plane, :, row].view(FP8).float()
    return (values * group[..., None]).flatten(-2) * scale


def _read(s):
    _, page, row = _places(s, s.rows)
    dt = TYPES[s.case["dtype"]]
    return {"k": _gather(s, page, 0, row).to(dt), "v": _gather(s, page, 1, row).to(dt)}


def _scores(s):
    """alpha q k [B, Nk, G, Lq, Lk], -inf where a query does not see a key, and the keys' places."""
    Nq, Nk, D = s.case["Nq"], s.case["Nk"], s.case["D"]
    B, Lq, Lk, G = s.case["B"], s.max_seqlen, s.max_seqlen_k, Nq // Nk
    page, row, real = _all_places(s)
    length, n = _sequence_lengths(s)[:, None], s.seq_offsets.diff()[:, None]
    i, j = torch.arange(Lq, device="cuda"), torch.arange(Lk, device="cuda")
    K = _gather(s, page, 0, row).masked_fill_(~real[..., None, None], 0).permute(0, 2, 1, 3)
    Q = s.q[(s.seq_offsets[:-1, None] + i).clamp(max=s.rows - 1).long()].float()  # [B, Lq, Nq, D]
    Q = Q.view(B, Lq, Nk, G, D).permute(0, 2, 3, 1, 4).reshape(B, Nk, G * Lq, D)
    x = torch.matmul(Q, K.transpose(2, 3)).mul_(s.alpha).view(B, Nk, G, Lq, Lk)
    seen = real[:, None, :] & ((j <= length[:, None] - n[:, None] + i[:, None]) | (not s.case["causal"]))  # [B, Lq, Lk]
    seen &= i[:, None] < n[:, None]
    return x.masked_fill_(~seen[:, None, None], -math.inf), page, row, real


def _new_rows(s):
    """Sequence and place in it of every new row."""
    t = torch.arange(s.rows, device="cuda", dtype=s.seq_offsets.dtype)
    b = torch.searchsorted(s.seq_offsets, t, right=True) - 1
    return b, t - s.seq_offsets[b]


def _lse(s):
    """Logarithms of the sums of the queries' weights [T, Nq], in 32 bits."""
    if not s.rows:
        return torch.empty(0, s.case["Nq"], device="cuda")
    x = _scores(s)[0]
    top = x.amax(-1, keepdim=True).clamp(min=torch.finfo(x.dtype).min)
    lse = x.sub_(top).exp_().sum(-1).log_() + top[..., 0]  # [B, Nk, G, Lq]
    b, i = _new_rows(s)
    return lse.permute(0, 3, 1, 2)[b, i].reshape(s.rows, s.case["Nq"])


def _attn(s):
    if not s.rows:
        return {"out": torch.empty_like(s.q)}
    x, page, row, real = _scores(s)
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top.masked_fill_(top == -math.inf, 0)).exp_()
    total = p.sum(-1, keepdim=True)
    V = _gather(s, page, 1, row).masked_fill_(~real[..., None, None], 0).permute(0, 2, 1, 3)
    o = torch.matmul(p.flatten(2, 3), V).view(*p.shape[:-1], -1) / total.masked_fill_(total == 0, 1)
    b, i = _new_rows(s)
    return {"out": o.permute(0, 3, 1, 2, 4)[b, i].reshape(s.q.shape).to(s.q.dtype)}


def _weights(s):
    page, row, real = _all_places(s)
    b, j = real.nonzero(as_tuple=True)
    page, row = page[b, j], row[b, j]
    if not s.rows:
        added = torch.zeros(page.numel(), s.case["Nk"], device="cuda")
    else:
        x = _scores(s)[0]
        lse = torch.zeros(s.case["B"], s.max_seqlen, *x.shape[1:3], device="cuda")
        at = _new_rows(s)
        lse[at] = s.lse.view(-1, *x.shape[1:3]).masked_fill(s.lse.view(-1, *x.shape[1:3]) == -math.inf, 0)
        added = x.sub_(lse.permute(0, 2, 3, 1)[..., None]).exp_().sum((2, 3)).permute(0, 2, 1)[b, j]
    s.weights[page, :, row] = s.weights[page, :, row] + added if s.case["accumulate"] else added
    return {"weights": s.weights}


def _evict(s):
    case, ps = s.case, s.case["page"]
    B, Nk, budget = case["B"], case["Nk"], case["budget"]
    length = _sequence_lengths(s)[:, None, None]
    count = length.clamp(max=budget)
    page, row, real = _all_places(s)
    j = torch.arange(s.max_seqlen_k, device="cuda")
    w = s.weights[page, :, row].permute(0, 2, 1)  # [B, Nk, Lk]
    w = w.masked_fill(j >= length - count.clamp(max=case["recent"]), math.inf).masked_fill(~real[:, None], -math.inf)
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order, (0, budget - order.shape[-1]), value=1 << 30)
    r = torch.arange(budget, device="cuda")
    kept = torch.where(r < count, order, 1 << 30).sort(-1).values
    kept = torch.where(r < count, kept, -1).int()  # [B, Nk, budget]
    # the rows themselves, copied before any is written
    b, hk, to = (kept >= 0).nonzero(as_tuple=True)
    source = kept[b, hk, to].long()
    page_of = lambda p: s.page_ids[s.page_offsets[b] + p // ps].long()  # noqa: E731
    old, new = (page_of(source), source % ps), (page_of(to), to % ps)
    tensors = [s.kv_cache] if case["cache"] == "same" else [s.kv_cache.view(torch.uint8)]
    tensors += [t.view(torch.uint8) for t in (s.kv_scale, s.kv_group_scale) if t is not None]
    for t in tensors:
        by_head = t.transpose(2, 3) if t is tensors[0] and case["cache"] != "fp4" else t  # [pages, 2, Nk, ps, ..]
        by_head[new[0], :, hk, new[1]] = by_head[old[0], :, hk, old[1]]
    # the shorter sequences' table: their first pages, -1 behind the last
    pages = (count[:, 0, 0] + ps - 1) // ps
    index = s.page_ids.dtype
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), pages.cumsum(0)])
    ids = torch.full_like(s.page_ids, -1)
    t = torch.arange(s.page_ids.numel(), device="cuda")
    owner = (torch.searchsorted(offsets, t, right=True) - 1).clamp(max=B - 1)
    at = (s.page_offsets[owner] + t - offsets[owner]).clamp(0, max(0, s.page_ids.numel() - 1)).long()
    ids = torch.where(t < offsets[-1], s.page_ids[at], ids)
    out = {"kept": kept, "page_offsets": offsets.to(index), "page_ids": ids,
           "last_page_len": torch.where(pages > 0, count[:, 0, 0] - (pages - 1) * ps, 1).to(index)}
    if case["cache"] == "fp4":
        short = _State()
        short.__dict__ |= s.__dict__ | {k: out[k] for k in ("page_offsets", "page_ids", "last_page_len")}
        short.seq_offsets, short.rows = s.kept_offsets, s.kept_rows
        return out | _read(short)
    return out | {"kv_cache": s.kv_cache, "kv_scale": s.kv_scale}


def _round_to(x, bits, least, largest):
    """x rounded to a binary format of `bits` bits behind the leading one, whose numbers below 2^least share its step."""
    step = _power(torch.frexp(x.abs().clamp(min=2.0 ** least)).exponent - 1 - bits, torch.float64)
    return (torch.round(x / step) * step).clamp(-largest, largest)


def _rows64(s, b):
    """Keys and values [Lk, Nk, D] of sequence b in 64 bits, and the pages that hold them."""
    ps, first, last = s.case["page"], int(s.page_offsets[b]), int(s.page_offsets[b + 1])
    length = (last - first - 1) * ps + int(s.last_page_len[b]) if last > first else 0
    ids = s.page_ids[first:last].long()
    planes = []
    for plane in (0, 1):
        if s.case["cache"] == "same":
            x = s.kv_cache[ids, plane].to(torch.float64)
        elif s.case["cache"] == "e4m3":
            x = s.kv_cache.view(torch.uint8)[ids, plane].view(FP8).to(torch.float64)
            x = x * _power(s.kv_scale[ids, plane].to(torch.int64) - 127, torch.float64).transpose(1, 2)[..., None]
        else:
            byte = s.kv_cache[ids, plane].to(torch.int64)
            x = torch.empty(*byte.shape[:-1], s.case["D"], dtype=torch.float64, device="cuda")
            for half in (0, 1):
                c = byte >> (4 * half) & 15
                m = torch.where(c & 6 == 0, 0.5 * (c & 1), (1 + 0.5 * (c & 1)) * _power((c >> 1 & 3) - 1, torch.float64))
                x[..., half::2] = torch.where(c >= 8, -m, m)
            factor = s.kv_group_scale.view(torch.uint8)[ids, plane].view(FP8).to(torch.float64)
            x = x * factor.repeat_interleave(16, -1) * _power(s.kv_scale[ids, plane].to(torch.int64) - 127, torch.float64)[..., None]
            x = x.transpose(1, 2)
        planes.append(x.flatten(0, 1)[:length])
    return planes, ids, length


def _quantised64(x):
    """The values that a 4-bit cache holds for rows x [.., D], in 64 bits."""
    largest = x.abs().amax(-1, keepdim=True).clamp(min=2688 * 2.0 ** EXP_MIN)
    e = torch.ceil(torch.log2(largest / 2688))
    e = torch.where(largest > 2688 * _power(e, torch.float64), e + 1, e)  # log2 rounds too
    e = torch.where(largest <= 2688 * _power(e - 1, torch.float64), e - 1, e).clamp(min=EXP_MIN)
    y = (x / _power(e, torch.float64)).unflatten(-1, (-1, 16))
    factor = _round_to(y.abs().amax(-1, keepdim=True) / 6, 3, -6, 448)
    code = torch.where(factor > 0, _round_to(y / factor.clamp(min=2.0 ** -9), 1, 0, 6), 0)
    return (code * factor).flatten(-2) * _power(e, torch.float64)


def exact(case, seed):
    s = prepare(case, seed)
    ends, Nk = [int(x) for x in s.seq_offsets], case["Nk"]
    if case["op"] == "append":
        return {"k": _quantised64(s.k.to(torch.float64)), "v": _quantised64(s.v.to(torch.float64))}
    if case["op"] == "read":
        k, v = (torch.zeros(s.rows, Nk, case["D"], dtype=torch.float64, device="cuda") for _ in range(2))
        for b in range(case["B"]):
            (k[ends[b]:ends[b + 1]], v[ends[b]:ends[b + 1]]), _, _ = _rows64(s, b)
        return {"k": k, "v": v}
    if case["op"] == "evict":
        return None  # every value is moved as it is, and the rest are whole numbers
    out = torch.zeros(s.q.shape, dtype=torch.float64, device="cuda")
    weights = s.weights.to(torch.float64) if case["op"] == "weights" else None
    G = case["Nq"] // Nk
    for b in range(case["B"]):
        (K, V), ids, length = _rows64(s, b)
        n = ends[b + 1] - ends[b]
        j = torch.arange(length, device="cuda")
        total = torch.zeros(length, Nk, dtype=torch.float64, device="cuda")
        for h in range(case["Nq"]):
            for i0 in range(0, n, 2048):
                i = torch.arange(i0, min(n, i0 + 2048), device="cuda")
                x = s.alpha * (s.q[ends[b] + i, h].to(torch.float64) @ K[:, h // G].T)
                if case["causal"]:
                    x = torch.where(j[None, :] <= (length - n + i)[:, None], x, -math.inf)
                if weights is None:
                    out[ends[b] + i, h] = torch.softmax(x, -1) @ V[:, h // G]
                else:
                    total[:, h // G] += torch.exp(x - s.lse[ends[b] + i, h].to(torch.float64)[:, None]).sum(0)
        if weights is not None:
            at = (ids[j // case["page"]], slice(None), j % case["page"])
            weights[at] = weights[at] + total if case["accumulate"] else total
    return {"out": out} if weights is None else {"weights": weights}
