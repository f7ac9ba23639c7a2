"""Cases of the 8-bit key / value cache operators and of the per-row sampler.

One decoding step appends the new tokens' keys and values to the cache, attends
over it, adds up the attention weights that eviction goes by, evicts where the
cache is over its budget, and draws the next tokens.  Each case is one of these
operators at one set of sizes.  ``run`` computes it in plain torch operations,
or, where ``own`` is true, by the library's calls.

The cache: blocks of ``block`` tokens, e4m3 codes [n_blocks, kv_heads, block,
head_dim], one fp32 power-of-two scale per block and head, a table of block ids
per sequence, and the number of tokens that each sequence holds.
"""

import math

import numpy as np
import torch

own = False

E4M3 = torch.float8_e4m3fn
E_MIN, E_MAX = -110, 120  # range of a block's exponent


# ----------------------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of the GPT-2 124M configuration (12 heads of 64, batch 12): one token per sequence
        {"name": "append_step", "op": "append", "dtype": "bf16", "seqs": 12, "kv_heads": 12, "dim": 64, "block": 16,
         "len_min": 1, "len_max": 1000, "new_min": 1, "new_max": 1},
        # the prompts of a GPT-2 XL batch (25 heads of 64, batch 8), of different lengths
        {"name": "append_prompt", "op": "append", "dtype": "bf16", "seqs": 8, "kv_heads": 25, "dim": 64, "block": 64,
         "len_min": 0, "len_max": 37, "new_min": 700, "new_max": 1001},
        # one user, early in the answer: latency counts
        {"name": "attention_one", "op": "attention", "dtype": "fp32", "seqs": 1, "heads": 12, "kv_heads": 12, "dim": 64,
         "block": 16, "len_min": 130, "len_max": 130, "new_min": 1, "new_max": 1},
        # a batch of users at GPT-2 124M's heads, lengths up to its block_size
        {"name": "attention_batch", "op": "attention", "dtype": "bf16", "seqs": 64, "heads": 12, "kv_heads": 12,
         "dim": 64, "block": 16, "len_min": 100, "len_max": 1023, "new_min": 1, "new_max": 1},
        # long contexts with shared heads
        {"name": "attention_long", "op": "attention", "dtype": "bf16", "seqs": 6, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 64, "len_min": 20000, "len_max": 40000, "new_min": 1, "new_max": 1},
        # the next part of a prompt, at GPT-2 XL's heads: many new tokens over what the cache holds
        {"name": "attention_chunk", "op": "attention", "dtype": "bf16", "seqs": 4, "heads": 25, "kv_heads": 25,
         "dim": 64, "block": 32, "len_min": 0, "len_max": 1501, "new_min": 63, "new_max": 200},
        # the weights of a decoding step, batch and long context
        {"name": "accumulate_batch", "op": "accumulate", "dtype": "bf16", "seqs": 64, "heads": 12, "kv_heads": 12,
         "dim": 64, "block": 16, "len_min": 100, "len_max": 1023, "new_min": 1, "new_max": 1},
        {"name": "accumulate_long", "op": "accumulate", "dtype": "bf16", "seqs": 6, "heads": 32, "kv_heads": 8,
         "dim": 128, "block": 64, "len_min": 20000, "len_max": 40000, "new_min": 1, "new_max": 1},
        # a batch whose caches are brought back to half their size
        {"name": "evict_batch", "op": "evict", "seqs": 64, "kv_heads": 12, "dim": 64, "block": 16, "len_min": 400,
         "len_max": 1023, "budget": 512, "recent": 64},
        # long contexts brought down to a fixed budget
        {"name": "evict_long", "op": "evict", "seqs": 6, "kv_heads": 8, "dim": 128, "block": 64, "len_min": 20000,
         "len_max": 40000, "budget": 8200, "recent": 500},
        # one row of the 50,257-way logits, fp32: nucleus sampling
        {"name": "sample_one", "op": "sample", "dtype": "fp32", "rows": 1, "vocab": 50257, "mode": "nucleus"},
        # a batch whose rows ask for different things (greedy, top-k, top-p, min-p, none)
        {"name": "sample_batch", "op": "sample", "dtype": "bf16", "rows": 256, "vocab": 50257, "mode": "mixed"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "accumulate", "evict", "sample"])
    dtype = rng.choice(["bf16", "fp32"])
    if op == "sample":
        rows = _log(rng, 1, 256)
        vocab = _log(rng, 65, 150000)
        while rows * vocab > 12_000_000:
            rows = max(1, rows // 2)
        return {"op": op, "dtype": dtype, "rows": rows, "vocab": vocab,
                "mode": rng.choice(["nucleus", "mixed", "top_k", "min_p", "all"])}
    dim = rng.choice([32, 64, 64, 128])
    kv = rng.choice([1, 2, 5, 8, 12, 25])
    block = rng.choice([16, 32, 64, 128])
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 20, 40000)
    while seqs * hi * kv * dim > 150_000_000:
        hi = max(20, hi // 2)
        seqs = max(1, seqs - seqs // 4)
    lo = int(hi * rng.choice([0.0, 0.3, 0.9]))
    c = {"op": op, "dtype": dtype, "seqs": seqs, "kv_heads": kv, "dim": dim, "block": block, "len_min": lo, "len_max": hi}
    if op == "evict":
        del c["dtype"]
        budget = max(2, int(hi * rng.uniform(0.2, 1.1)))
        c.update(budget=budget, recent=int(budget * rng.uniform(0.0, 1.0)))
        return c
    new = 1
    if op == "append":
        new = _log(rng, 1, 1200)
        while seqs * new * kv * dim > 15_000_000:
            new = max(1, new // 2)
    else:
        c["heads"] = kv * rng.choice([1, 1, 2, 4, 7])
        if rng.random() < 0.4:
            new = _log(rng, 2, 200)
            while seqs * new * c["heads"] * (hi + new) > 25_000_000 and new > 1:
                new = max(1, new // 2)
    c.update(new_min=max(1, new - rng.choice([0, new // 2])), new_max=new)
    return c


def _spread(lo, hi, n):
    """n whole numbers spread evenly from lo to hi."""
    return [lo + (hi - lo) * i // (n - 1) if n > 1 else (lo + hi) // 2 for i in range(n)]


def _lengths(case):
    """The sequences' lengths and new tokens: the same numbers for every seed (prepare shuffles them)."""
    return _spread(case["len_min"], case["len_max"], case["seqs"]), _spread(case.get("new_min", 0), case.get("new_max", 0),
                                                                           case["seqs"])


def work(case):
    op = case["op"]
    esize = 2 if case.get("dtype") == "bf16" else 4
    if op == "sample":
        return {"bytes": case["rows"] * (case["vocab"] * esize + 28), "flops": 2 * case["rows"] * case["vocab"]}
    lens, news = _lengths(case)
    news = sorted(news)
    kv, dim, P, S = case["kv_heads"], case["dim"], case["block"], case["seqs"]
    if op == "append":
        n = sum(news)
        return {"bytes": n * kv * dim * 2 * (esize + 1) + 2 * 4 * kv * (n // P + S), "flops": 4 * n * kv * dim}
    if op == "evict":
        kept = sum(min(n, case["budget"]) for n in lens)
        read = sum(n for n in lens if n > case["budget"])
        return {"bytes": kv * (4 * read + kept * (4 * dim + 12)) + 16 * kv * (kept // P + S), "flops": 4 * kept * kv * dim}
    slots = sum(lens) + sum(news)
    rows = sum(news) * case["heads"]
    # the mean pairing of lengths and new tokens: which sequence has which is shuffled by the seed
    pairs = sum(n * (sum(lens) / S) + n * (n + 1) / 2 for n in news) * case["heads"]
    scales = 4 * kv * (slots // P + S)
    if op == "attention":
        return {"bytes": slots * kv * dim * 2 + 2 * scales + rows * (2 * dim * esize + 4), "flops": 4 * dim * pairs}
    return {"bytes": slots * kv * (dim + 8) + scales + rows * (dim * esize + 4), "flops": 2 * dim * pairs}


# ----------------------------------------------------------------------------- inputs

def _exponent(amax):
    """The smallest e with amax <= 448 * 2^e (448 = 0.875 * 2^9 is e4m3's largest value), within its range."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _pow2(e):
    return torch.ldexp(torch.ones((), device=e.device), e)


def _fill(shape, gen, outliers):
    """A pool of cached keys or values: codes and scales.  Keys have a few channels that are larger than the rest."""
    n_blocks, kv, P, dim = shape
    codes = torch.empty(shape, dtype=E4M3, device="cuda")
    scale = torch.empty(n_blocks, kv, device="cuda")
    part = max(1, (1 << 26) // (kv * P * dim))
    gain = torch.ones(kv, 1, dim, device="cuda")
    if outliers:
        gain += 3.0 * (torch.rand(kv, 1, dim, device="cuda", generator=gen) < 0.06)
    for i in range(0, n_blocks, part):
        x = torch.randn(min(part, n_blocks - i), kv, P, dim, device="cuda", generator=gen) * gain
        e = _exponent(x.abs().amax((2, 3)))
        scale[i:i + part] = _pow2(e)
        codes[i:i + part] = (x * _pow2(-e)[:, :, None, None]).to(E4M3)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    if case["op"] == "sample":
        return _prepare_sample(case, gen, host)
    S, kv, dim, P = case["seqs"], case["kv_heads"], case["dim"], case["block"]
    lens, news = _lengths(case)
    lens, news = host.permutation(lens), host.permutation(news)
    cap = -(-(case["len_max"] + case.get("new_max", 0)) // P)  # blocks that a sequence can have
    out_cap = -(-case["budget"] // P) if case["op"] == "evict" else 0
    n_blocks = S * (cap + out_cap) + 3
    ids = torch.from_numpy(host.permutation(n_blocks).astype(np.int32)).cuda()
    st = {"op": case["op"], "case": case,
          "table": ids[:S * cap].reshape(S, cap).contiguous(),
          "length": torch.from_numpy(lens.astype(np.int32)).cuda()}
    st["k"], st["k_scale"] = _fill((n_blocks, kv, P, dim), gen, True)
    st["v"], st["v_scale"] = _fill((n_blocks, kv, P, dim), gen, False)
    st["weight"] = None
    if case["op"] in ("accumulate", "evict"):
        # accumulated weights: a few heavy tokens, many light ones
        st["weight"] = torch.rand(n_blocks, kv, P, device="cuda", generator=gen).pow_(8.0) * 20.0
    if case["op"] == "evict":
        st["table_out"] = ids[S * cap:S * (cap + out_cap)].reshape(S, out_cap).contiguous()
        st["kept"] = torch.full((S, kv, case["budget"]), -1, dtype=torch.int32, device="cuda")
        return st
    T = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    start = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
    n = int(start[-1])
    # one token for each sequence needs no offsets
    st["start"] = None if case["new_max"] == 1 else torch.from_numpy(start).cuda()
    st["max_new"] = int(case["new_max"])
    # the new tokens' q, k and v as a projection leaves them, beside each other in one row
    H = case.get("heads", kv)
    x = torch.randn(n, (H + 2 * kv) * dim, device="cuda", generator=gen)
    x = x.to(T)
    st["q"] = x[:, :H * dim].unflatten(1, (H, dim))
    st["new_k"] = x[:, H * dim:(H + kv) * dim].unflatten(1, (kv, dim))
    st["new_v"] = x[:, (H + kv) * dim:].unflatten(1, (kv, dim))
    if case["op"] == "attention":
        st["out"] = torch.zeros(n, H, dim, dtype=T, device="cuda")
        st["lse"] = torch.zeros(n, H, device="cuda")
    if case["op"] == "accumulate":
        st["lse"] = _lse(st)  # an attention over the same cache came before
    return st


def _prepare_sample(case, gen, host):
    rows, V = case["rows"], case["vocab"]
    ld = -(-V // 64) * 64  # the head's padded width
    T = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    z = torch.randn(rows, ld, device="cuda", generator=gen) * 2.0
    # some tokens stand out, as in a trained model's logits
    hot = torch.randint(0, V, (rows, 24), device="cuda", generator=gen)
    z.scatter_add_(1, hot, 4.0 + 5.0 * torch.rand(rows, 24, device="cuda", generator=gen))
    mode = case["mode"]
    kind = {"nucleus": 2, "top_k": 1, "min_p": 3, "all": 4}.get(mode)
    kind = host.integers(0, 6, rows) if kind is None else np.full(rows, kind)
    temp = np.where(kind == 0, 0.0, host.choice([0.7, 0.8, 1.0, 1.2], rows))
    top_k = np.where((kind == 1) | (kind == 5), host.choice([5, 40, 50, 200], rows), 0)
    top_p = np.where((kind == 2) | (kind == 5), host.choice([0.5, 0.9, 0.95], rows), 1.0)
    min_p = np.where((kind == 3) | (kind == 5), host.choice([0.02, 0.05, 0.1], rows), 0.0)
    f = lambda a, t: torch.from_numpy(np.ascontiguousarray(a.astype(t))).cuda()  # noqa: E731
    return {"op": "sample", "case": case, "V": V, "logits": z.to(T),
            "temperature": f(temp, np.float32), "top_k": f(top_k, np.int32), "top_p": f(top_p, np.float32),
            "min_p": f(min_p, np.float32), "uniform": f(host.random(rows), np.float32),
            "token": torch.zeros(rows, dtype=torch.int32, device="cuda"),
            "logp": torch.zeros(rows, device="cuda")}


# ----------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"append": _append, "attention": _attention, "accumulate": _accumulate, "evict": _evict,
            "sample": _sample}[state["op"]](state)


def _cache_out(st):
    return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _run_own(st):
    from gpt_decoder_lm_b200 import binding as gb
    op = st["op"]
    if op == "sample":
        gb.sample_rows(st["logits"], st["uniform"], st["token"], temperature=st["temperature"], top_k=st["top_k"],
                       top_p=st["top_p"], min_p=st["min_p"], logp=st["logp"], V=st["V"])
        return {"token": st["token"], "logp": st["logp"]}
    cache = st.get("cache")
    if cache is None:  # the handle that a program makes with its cache
        cache = st["cache"] = gb.KV8Cache(st["k"], st["v"], st["k_scale"], st["v_scale"], st["table"], st["length"],
                                          weight=st["weight"])
    if op == "append":
        cache.append(st["new_k"], st["new_v"], start=st["start"], max_new=st["max_new"])
        return _cache_out(st)
    if op == "attention":
        cache.attention(st["q"], st["out"], start=st["start"], max_new=st["max_new"], lse=st["lse"])
        return {"out": st["out"], "lse": st["lse"]}
    if op == "accumulate":
        cache.accumulate(st["q"], st["lse"], start=st["start"], max_new=st["max_new"])
        return {"weight": st["weight"]}
    cache.evict(st["table_out"], st["case"]["budget"], st["case"]["recent"], st["kept"])
    return dict(_cache_out(st), weight=st["weight"], kept=st["kept"])


def _rows(st):
    """For each new token: its sequence, its number within the sequence's new tokens, and how many each sequence has."""
    S = st["length"].numel()
    n = st["q"].shape[0]
    if st["start"] is None:
        seq = torch.arange(n, device="cuda")
        return seq, torch.zeros_like(seq), torch.ones(S, dtype=torch.long, device="cuda")
    start = st["start"].long()
    row = torch.arange(n, device="cuda")
    seq = torch.searchsorted(start[1:], row, right=True)
    return seq, row - start[seq], start[1:] - start[:-1]


def _append(st):
    P, kv = st["case"]["block"], st["case"]["kv_heads"]
    seq, i, n_new = _rows(st)
    length, table = st["length"].long(), st["table"].long()
    slot = length[seq] + i
    blk, off = table[seq, slot // P], slot % P
    # the part-filled blocks that new tokens come into: their earlier tokens stay
    open_seq = ((length % P > 0) & (n_new > 0)).nonzero()[:, 0]
    open_blk = table[open_seq, length[open_seq] // P]
    old = torch.arange(P, device="cuda")[None, :] < (length[open_seq] % P)[:, None]  # [open, P]
    for x, codes, scale in ((st["new_k"], st["k"], st["k_scale"]), (st["new_v"], st["v"], st["v_scale"])):
        x = x.float()
        mag = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax(-1)  # [n, kv]
        amax = torch.zeros_like(scale).index_reduce_(0, blk, mag, "amax")
        e = _exponent(amax)
        e_old = torch.frexp(scale[open_blk])[1] - 1
        e[open_blk] = torch.maximum(e[open_blk], e_old)
        was = codes.view(torch.uint8)[open_blk].view(E4M3)  # [open, kv, P, dim]
        moved = (was.float() * _pow2(e_old - e[open_blk])[:, :, None, None]).to(E4M3)
        keep = old[:, None, :, None]
        codes.view(torch.uint8)[open_blk] = torch.where(keep, moved.view(torch.uint8), was.view(torch.uint8))
        codes.view(torch.uint8)[blk, :, off] = (x * _pow2(-e[blk])[:, :, None]).to(E4M3).view(torch.uint8)
        scale[blk] = _pow2(e[blk])
    if st["weight"] is not None:
        st["weight"][blk, :, off] = 0.0
    return _cache_out(st)


def _gather(st, codes, scale):
    """The sequences' cached keys or values, [S, kv, L, dim] in fp32."""
    table = st["table"].long()
    x = codes.view(torch.uint8)[table].view(E4M3).float() * scale[table][..., None, None]  # [S, cap, kv, P, dim]
    return x.transpose(1, 2).flatten(2, 3)


def _scores(st):
    """Scaled scores [S, kv, G, N, L] of the new tokens (padded to N a sequence), -inf where a slot is not seen; the
    new tokens' places."""
    c = st["case"]
    kv, dim = c["kv_heads"], c["dim"]
    S, N, G = st["length"].numel(), st["max_new"], c["heads"] // c["kv_heads"]
    seq, i, n_new = _rows(st)
    q = torch.zeros(S, N, kv * G, dim, device="cuda")
    q[seq, i] = st["q"].float()
    q = q.reshape(S, N, kv, G, dim).permute(0, 2, 3, 1, 4)
    k = _gather(st, st["k"], st["k_scale"])
    L = k.shape[2]
    s = torch.matmul(q.reshape(S, kv, G * N, dim), k.transpose(2, 3)).reshape(S, kv, G, N, L) / math.sqrt(dim)
    seen = torch.arange(L, device="cuda") <= (st["length"].long()[:, None] + torch.arange(N, device="cuda"))[..., None]
    seen &= (torch.arange(N, device="cuda") < n_new[:, None])[..., None]
    return s.masked_fill(~seen[:, None, None], -math.inf), seq, i


def _lse(st):
    s, seq, i = _scores(st)
    return torch.logsumexp(s, -1).permute(0, 3, 1, 2).flatten(2)[seq, i].contiguous()


def _attention(st):
    s, seq, i = _scores(st)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    S, kv, G, N, L = s.shape
    v = _gather(st, st["v"], st["v_scale"])
    o = torch.matmul(p.reshape(S, kv, G * N, L), v).reshape(S, kv, G, N, -1) / l
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)
    lse = (m + torch.log(l))[..., 0].permute(0, 3, 1, 2).flatten(2)
    st["out"].copy_(o[seq, i])
    st["lse"].copy_(lse[seq, i])
    return {"out": st["out"], "lse": st["lse"]}


def _accumulate(st):
    s, seq, i = _scores(st)
    S, kv, G, N, L = s.shape
    lse = torch.full((S, N, kv * G), math.inf, device="cuda")
    lse[seq, i] = st["lse"]
    p = torch.exp(s - lse.reshape(S, N, kv, G).permute(0, 2, 3, 1)[..., None])  # exp(-inf) = 0 where not seen
    w = p.sum((2, 3))  # [S, kv, L]
    P = st["case"]["block"]
    table = st["table"].long()
    st["weight"].index_add_(0, table.flatten(), w.unflatten(2, (-1, P)).transpose(1, 2).flatten(0, 1))
    return {"weight": st["weight"]}


def _evict(st):
    c = st["case"]
    P, budget, recent, kv, dim = c["block"], c["budget"], c["recent"], c["kv_heads"], c["dim"]
    table, out = st["table"].long(), st["table_out"].long()
    S, L = table.shape[0], table.shape[1] * P
    length = st["length"].long()
    w = st["weight"][table].transpose(1, 2).flatten(2)  # [S, kv, L]
    j = torch.arange(L, device="cuda")
    # the last `recent` slots come first in the order, the slots behind the sequence last
    rank = torch.where(j >= (length - recent)[:, None], 1e30, 0.0)[:, None, :]
    w_order = torch.maximum(w, rank).masked_fill((j >= length[:, None])[:, None, :], -math.inf)
    order = torch.sort(w_order, dim=-1, descending=True, stable=True).indices[..., :budget]  # ties: the lowest slot
    n = length.clamp_max(budget)[:, None, None]
    places = torch.arange(budget, device="cuda")
    order = torch.nn.functional.pad(order, (0, max(0, budget - L)), value=L)
    kept = torch.sort(torch.where(places < n, order, L), -1).values  # in the slots' order; L: none
    st["kept"].copy_(torch.where(kept < L, kept, st["kept"]))
    valid = kept < L
    src = kept.clamp_max(L - 1)
    sblk = table[torch.arange(S, device="cuda")[:, None, None], src // P]  # [S, kv, budget]
    h = torch.arange(kv, device="cuda")[None, :, None]
    full = out.shape[1] * P
    grow = lambda x, v: torch.nn.functional.pad(x, (0,) * (2 * (x.dim() - 3)) + (0, full - budget), value=v)  # noqa: E731
    valid_f = grow(valid, False).unflatten(2, (-1, P)).transpose(1, 2)  # [S, blocks, kv, P]
    for codes, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])):
        x = codes.view(torch.uint8)[sblk, h, src % P].view(E4M3).float() * scale[sblk, h][..., None]
        x = grow(x, 0.0).unflatten(2, (-1, P)).transpose(1, 2)  # [S, blocks, kv, P, dim]
        x = x * valid_f[..., None]
        e = _exponent(x.abs().amax((-1, -2)))
        new = (x * _pow2(-e)[..., None, None]).to(E4M3).view(torch.uint8)
        codes.view(torch.uint8)[out] = torch.where(valid_f[..., None], new, codes.view(torch.uint8)[out])
        any_f = valid_f.any(-1)
        scale[out] = torch.where(any_f, _pow2(e), scale[out])
    wk = grow(st["weight"][sblk, h, src % P], 0.0).unflatten(2, (-1, P)).transpose(1, 2)
    st["weight"][out] = torch.where(valid_f, wk, st["weight"][out])
    return dict(_cache_out(st), weight=st["weight"], kept=st["kept"])


def _sample(st):
    V = st["V"]
    z = st["logits"][:, :V].double()
    rows = z.shape[0]
    greedy = ~(st["temperature"] > 0)
    t = torch.where(greedy, torch.ones_like(st["temperature"]), st["temperature"]).double()
    zmax = z.amax(1, keepdim=True)
    zs = torch.sort(z, 1, descending=True).values
    k = torch.where((st["top_k"] > 0) & (st["top_k"] < V), st["top_k"], V).long()
    keep = z >= zs.gather(1, k[:, None] - 1)
    p = torch.exp((z - zmax) / t[:, None]) * keep
    ps = torch.sort(p, 1, descending=True).values
    cum = torch.cumsum(ps, 1)
    nucleus = st["top_p"] < 1
    target = st["top_p"].double().clamp_min(0)[:, None] * cum[:, -1:]
    tau = ps.gather(1, (cum < target).sum(1, keepdim=True).clamp_max(V - 1))
    p = p * torch.where(nucleus[:, None], p >= tau, True) * (p >= st["min_p"].double().clamp(0, 1)[:, None])
    c = torch.cumsum(p, 1)
    pos = torch.arange(V, device="cuda")
    last = torch.where(p > 0, pos, -1).amax(1)
    drawn = torch.minimum((c <= st["uniform"].double()[:, None] * c[:, -1:]).sum(1), last)
    best = torch.where(z == zmax, pos, V).amin(1)
    token = torch.where(greedy, best, drawn)
    logp = torch.log(p.gather(1, token[:, None])[:, 0] / c[:, -1])
    st["token"].copy_(token)
    st["logp"].copy_(torch.where(greedy, torch.zeros_like(logp), logp))
    return {"token": st["token"], "logp": st["logp"]}


# ----------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "accumulate": _exact_accumulate,
            "evict": _exact_evict, "sample": _exact_sample}[case["op"]](st)


def _e4m3(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even; x within the format's range."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp_min(2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, x)


def _best_exponent(amax):
    if amax <= 0:
        return E_MIN
    e = math.ceil(math.log2(amax / 448.0))
    while amax > math.ldexp(448.0, e):
        e += 1
    while amax <= math.ldexp(448.0, e - 1):
        e -= 1
    return min(max(e, E_MIN), E_MAX)


def _sequences(st):
    """(sequence, its length, its rows of the packed tokens)"""
    start = st["start"].tolist() if st["start"] is not None else list(range(len(st["table"]) + 1))
    return [(s, n, range(start[s], start[s + 1])) for s, n in enumerate(st["length"].tolist())]


def _exact_append(st):
    P, kv = st["case"]["block"], st["case"]["kv_heads"]
    table = st["table"].tolist()
    got = {}
    for name in ("k", "v"):
        codes, scale = st[name].float(), st[name + "_scale"].clone()
        x = st["new_" + name].double()
        # one pass over the blocks that new tokens come into, all heads of one at a time
        amax = x.abs().amax(-1)
        jobs = []
        for s, n, rows in _sequences(st):
            at = n
            while at < n + len(rows):
                end = min((at // P + 1) * P, n + len(rows))
                jobs.append((table[s][at // P], at % P, rows[at - n], rows[at - n] + end - at))
                at = end
        tops = torch.stack([amax[r0:r1].amax(0) for _, _, r0, r1 in jobs]).cpu().tolist()
        olds = scale[torch.tensor([j[0] for j in jobs], device="cuda")].cpu().tolist()
        for (b, off, r0, r1), top, old in zip(jobs, tops, olds):
            e_old = [round(math.log2(v)) for v in old]
            e = [_best_exponent(v) for v in top]
            if off:
                e = [max(a, c) for a, c in zip(e, e_old)]
                back = torch.tensor([2.0 ** (c - a) for a, c in zip(e, e_old)], dtype=torch.float64, device="cuda")
                codes[b, :, :off] = _e4m3(codes[b, :, :off].double() * back[:, None, None]).float()
            f = torch.tensor([2.0 ** -a for a in e], dtype=torch.float64, device="cuda")
            codes[b, :, off:off + r1 - r0] = _e4m3(x[r0:r1].transpose(0, 1) * f[:, None, None]).float()
            scale[b] = (1.0 / f).float()
        got[name], got[name + "_scale"] = codes.to(E4M3), scale.double()
    return got


def _exact_kv(st, s, n, which):
    """The first n cached keys or values of sequence s, [kv, n, dim] in 64 bits."""
    P = st["case"]["block"]
    ids = st["table"][s, :-(-n // P)].long()
    x = st[which].view(torch.uint8)[ids].view(E4M3).double() * st[which + "_scale"][ids].double()[:, :, None, None]
    return x.transpose(0, 1).reshape(x.shape[1], -1, x.shape[3])[:, :n], ids


def _exact_softmax(st, s, n, rows):
    """Scores of the sequence's new tokens: [n_new, kv, G, n + n_new] with -inf at the slots that are not seen."""
    c = st["case"]
    total = n + len(rows)
    k, ids = _exact_kv(st, s, total, "k")
    q = st["q"][rows.start:rows.stop].double().unflatten(1, (c["kv_heads"], -1))
    score = torch.einsum("ikgd,kjd->ikgj", q, k) * c["dim"] ** -0.5
    late = torch.arange(total, device="cuda")[None, :] > n + torch.arange(len(rows), device="cuda")[:, None]
    score[late[:, None, None, :].expand_as(score)] = -math.inf
    return score, ids


def _exact_attention(st):
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["lse"].shape, dtype=torch.float64, device="cuda")
    for s, n, rows in _sequences(st):
        if len(rows):
            score, _ = _exact_softmax(st, s, n, rows)
            v, _ = _exact_kv(st, s, n + len(rows), "v")
            a = torch.softmax(score, -1)
            out[rows.start:rows.stop] = torch.einsum("ikgj,kjd->ikgd", a, v).flatten(1, 2)
            lse[rows.start:rows.stop] = torch.logsumexp(score, -1).flatten(1, 2)
    return {"out": out, "lse": lse}


def _exact_accumulate(st):
    c = st["case"]
    w = st["weight"].double()
    P = c["block"]
    for s, n, rows in _sequences(st):
        if len(rows):
            score, ids = _exact_softmax(st, s, n, rows)
            given = st["lse"][rows.start:rows.stop].double().unflatten(1, (c["kv_heads"], -1))
            a = torch.exp(score - given[..., None]).sum((0, 2))  # [kv, total]
            a = torch.nn.functional.pad(a, (0, len(ids) * P - a.shape[1]))
            w[ids] += a.unflatten(1, (-1, P)).transpose(0, 1)
    return {"weight": w}


def _exact_evict(st):
    c = st["case"]
    P, budget, recent, kv, dim = c["block"], c["budget"], c["recent"], c["kv_heads"], c["dim"]
    kept = st["kept"].cpu().numpy().astype(np.int64)
    res = {"weight": st["weight"].double()}
    lengths = st["length"].tolist()
    weight = st["weight"].cpu().numpy()
    table = st["table"].cpu().numpy()
    for s, n in enumerate(lengths):
        for h in range(kv):
            if n <= budget:
                kept[s, h, :n] = np.arange(n)
                continue
            w = weight[table[s], h].reshape(-1)[:n - recent]
            heavy = np.lexsort((np.arange(n - recent), -w.astype(np.float64)))[:budget - recent]
            kept[s, h] = np.concatenate([np.sort(heavy), np.arange(n - recent, n)])
    dev = torch.from_numpy(kept).cuda()
    for name in ("k", "v"):
        res[name], res[name + "_scale"] = st[name].clone(), st[name + "_scale"].double()
    heads = torch.arange(kv, device="cuda")[:, None]
    for s, n in enumerate(lengths):
        m = min(n, budget)
        at = dev[s, :, :m]
        ids = st["table"][s].long()[at // P]
        blocks = -(-m // P)
        to = st["table_out"][s, :blocks].long()
        place = torch.arange(m, device="cuda")
        for name in ("k", "v"):
            x = st[name].view(torch.uint8)[ids, heads, at % P].view(E4M3).double() * \
                st[name + "_scale"][ids, heads].double()[..., None]  # [kv, m, dim]
            x = torch.nn.functional.pad(x, (0, 0, 0, blocks * P - m)).unflatten(1, (blocks, P))
            top = x.abs().amax((2, 3))  # [kv, blocks]
            e = torch.ceil(torch.log2((top / 448.0).clamp_min(2.0 ** E_MIN)) - 1e-6)  # one too small next to a border
            e = (e + (top > 448.0 * torch.exp2(e))).clamp(E_MIN, E_MAX)
            code = _e4m3(x * torch.exp2(-e)[..., None, None]).flatten(1, 2)[:, :m].float().to(E4M3)
            res[name].view(torch.uint8)[to[place // P][None, :], heads, (place % P)[None, :]] = code.view(torch.uint8)
            res[name + "_scale"][to] = torch.exp2(e).transpose(0, 1)
        res["weight"][to[place // P][None, :], heads, (place % P)[None, :]] = \
            st["weight"][ids, heads, at % P].double()
    res["kept"] = dev.to(torch.int32)
    return res


def _exact_sample(st):
    V = st["V"]
    Z = st["logits"][:, :V].double().cpu().numpy()
    par = {n: st[n].double().cpu().numpy() for n in ("temperature", "top_k", "top_p", "min_p", "uniform")}
    token, logp = [], []
    for r in range(Z.shape[0]):
        z, t, k = Z[r], par["temperature"][r], int(par["top_k"][r])
        if not t > 0:
            token.append(int(np.argmax(z)))
            logp.append(0.0)
            continue
        order = np.argsort(-z, kind="stable")
        zs = z[order]
        n = V if not 0 < k < V else int(np.searchsorted(-zs, -zs[k - 1], side="right"))  # ties are kept
        p = np.exp((zs[:n] - zs[0]) / t)
        m = n
        if par["top_p"][r] < 1:
            cum = np.cumsum(p)
            m = min(n, 1 + int(np.searchsorted(cum, par["top_p"][r] * cum[-1], side="left")))
            m = int(np.searchsorted(-zs[:n], -zs[m - 1], side="right"))
        m = min(m, int(np.sum(p >= par["min_p"][r])))
        idx = np.sort(order[:m])
        q = np.exp((z[idx] - zs[0]) / t)
        c = np.cumsum(q)
        at = min(int(np.searchsorted(c, par["uniform"][r] * c[-1], side="right")), len(idx) - 1)
        token.append(int(idx[at]))
        logp.append(math.log(q[at] / c[-1]))
    return {"token": torch.tensor(token, dtype=torch.int32), "logp": torch.tensor(logp, dtype=torch.float64)}
