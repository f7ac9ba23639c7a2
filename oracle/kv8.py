"""Float64 oracle of the 8-bit key / value cache (gpt_kv8_*).

TEST INFRASTRUCTURE ONLY: it shares no code with the library and imports
nothing from the product package.  Plain loops over sequences, heads and
blocks; numpy only.

The format: a block of P tokens of one head has one scale 2^e, e the smallest
exponent in [-110, 120] at which its largest finite magnitude is at most
448 * 2^e; a stored value is an e4m3 value (4 exponent bits with bias 7, 3
mantissa bits, subnormals, no infinity, one NaN pattern) times the scale.
"""

from __future__ import annotations

import math

import numpy as np

from . import gpt_oracle as go

E_MIN, E_MAX = -110, 120

__all__ = ["decode", "encode", "exponent", "Cache", "Decoder"]


def _table() -> np.ndarray:
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = math.nan if (c & 127) == 127 else math.ldexp(m / 8, -6) if e == 0 else math.ldexp(1 + m / 8, e - 7)
        out[c] = -v if c & 128 else v
    return out


TABLE = _table()
_POS = TABLE[:127]  # ascending values of the non-negative codes


def decode(codes: np.ndarray) -> np.ndarray:
    return TABLE[np.asarray(codes, dtype=np.uint8)]


def encode(x: np.ndarray) -> np.ndarray:
    """The code nearest to each value (ties to the even code), NaN for what is not finite; |x| <= 448."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(np.where(np.isfinite(x), x, 0.0))
    assert (a <= 448).all()
    hi = np.clip(np.searchsorted(_POS, a, side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    c = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    c = np.where(np.isfinite(x), c, 127)
    return (c + 128 * np.signbit(x)).astype(np.uint8)


def exponent(amax: float) -> int:
    if amax <= 0:
        return E_MIN
    e = E_MIN
    while e < E_MAX and amax > math.ldexp(448.0, e):
        e += 1
    return e


class Cache:
    """Codes, scales and weights as numpy arrays laid out as the library's."""

    def __init__(self, k, v, k_scale, v_scale, table, length, weight=None):
        self.k, self.v = np.array(k, np.uint8), np.array(v, np.uint8)
        self.ks, self.vs = np.array(k_scale, np.float64), np.array(v_scale, np.float64)
        self.table, self.length = np.array(table), np.array(length)
        self.weight = None if weight is None else np.array(weight, np.float64)
        self.P = self.k.shape[2]

    def ok(self, b) -> bool:
        return 0 <= b < self.k.shape[0]

    def append(self, new_k, new_v, start):
        P = self.P
        for s, n0 in enumerate(self.length):
            rows = range(start[s], start[s + 1])
            at = int(n0)
            while at < n0 + len(rows):
                end = min((at // P + 1) * P, int(n0) + len(rows))
                if at // P >= self.table.shape[1]:
                    break
                b, off = int(self.table[s, at // P]), at % P
                if self.ok(b):
                    r = slice(rows.start + at - int(n0), rows.start + end - int(n0))
                    for x, codes, scale in ((new_k[r], self.k, self.ks), (new_v[r], self.v, self.vs)):
                        for h in range(x.shape[1]):
                            y = np.asarray(x[:, h], np.float64)
                            fin = np.abs(y[np.isfinite(y)])
                            e = exponent(fin.max() if fin.size else 0.0)
                            if off:
                                old = int(round(math.log2(scale[b, h])))
                                e = max(e, old)
                                c = codes[b, h, :off]
                                codes[b, h, :off] = encode(decode(c) * math.ldexp(1.0, old - e))
                            scale[b, h] = math.ldexp(1.0, e)
                            codes[b, h, off:off + end - at] = encode(y * math.ldexp(1.0, -e))
                    if self.weight is not None:
                        self.weight[b, :, off:off + end - at] = 0.0
                at = end

    def _slots(self, s, n):
        """(block, offset) of the first n slots of sequence s, None where the block is not in the pool."""
        out = []
        for j in range(min(n, self.table.shape[1] * self.P)):
            b = int(self.table[s, j // self.P])
            out.append((b, j % self.P) if self.ok(b) else None)
        return out

    def values(self, s, n, which):
        """[n_slots, heads, dim] values of the first n slots (zeros where the block is missing) and which are there."""
        codes, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        slots = self._slots(s, n)
        there = np.array([x is not None for x in slots], bool)
        vals = np.zeros((len(slots), codes.shape[1], codes.shape[3]))
        for j, x in enumerate(slots):
            if x is not None:
                vals[j] = decode(codes[x[0], :, x[1]]) * scale[x[0]][:, None]
        return vals, there

    def attention(self, q, start, scale):
        """(out, lse, probabilities per sequence [rows, heads, slots])."""
        q = np.asarray(q, np.float64)
        G = q.shape[1] // self.k.shape[1]
        out, lse, probs = np.zeros_like(q), np.full(q.shape[:2], np.nan), []
        for s, n0 in enumerate(self.length):
            n = start[s + 1] - start[s]
            kk, there = self.values(s, int(n0) + n, "k")
            vv, _ = self.values(s, int(n0) + n, "v")
            p_s = np.zeros((n, q.shape[1], len(there)))
            for i in range(n):
                see = there & (np.arange(len(there)) <= n0 + i)
                for h in range(q.shape[1]):
                    r = start[s] + i
                    if not see.any():
                        lse[r, h] = -np.inf
                        continue
                    z = scale * (kk[see, h // G] @ q[r, h])
                    m = z.max()
                    e = np.exp(z - m)
                    lse[r, h] = m + np.log(e.sum())
                    p_s[i, h, see] = e / e.sum()
                    out[r, h] = (e / e.sum()) @ vv[see, h // G]
            probs.append(p_s)
        return out, lse, probs

    def accumulate(self, probs):
        G = probs[0].shape[1] // self.k.shape[1]
        for s, p in enumerate(probs):
            for j, x in enumerate(self._slots(s, p.shape[2])):
                if x is not None:
                    for h in range(self.k.shape[1]):
                        self.weight[x[0], h, x[1]] += p[:, h * G:(h + 1) * G, j].sum()

    def evict(self, table_out, budget, recent):
        """Moves the kept slots into table_out's blocks; the kept slots [S, heads, budget]."""
        S, H = self.table.shape[0], self.k.shape[1]
        kept = np.full((S, H, budget), -1, np.int64)
        src = (self.k.copy(), self.v.copy(), self.ks.copy(), self.vs.copy(), self.weight.copy())
        for s in range(S):
            n = min(int(self.length[s]), self.table.shape[1] * self.P)
            slots = self._slots(s, n)
            for h in range(H):
                if n <= budget:
                    keep = list(range(n))
                else:
                    w = [-math.inf if x is None or np.isnan(src[4][x[0], h, x[1]]) else src[4][x[0], h, x[1]]
                         for x in slots[:n - recent]]
                    heavy = sorted(range(n - recent), key=lambda j: (-w[j], j))[:budget - recent]
                    keep = sorted(heavy) + list(range(n - recent, n))
                kept[s, h, :len(keep)] = keep
                for b0 in range(0, len(keep), self.P):
                    part = keep[b0:b0 + self.P]
                    bo = int(table_out[s, b0 // self.P])
                    for codes, scale, oc, osc in ((src[0], src[2], self.k, self.ks), (src[1], src[3], self.v, self.vs)):
                        x = np.stack([decode(codes[slots[j][0], h, slots[j][1]]) * scale[slots[j][0], h]
                                      if slots[j] is not None else np.zeros(codes.shape[3]) for j in part])
                        fin = np.abs(x[np.isfinite(x)])
                        e = exponent(fin.max() if fin.size else 0.0)
                        oc[bo, h, :len(part)] = encode(x * math.ldexp(1.0, -e))
                        osc[bo, h] = math.ldexp(1.0, e)
                    self.weight[bo, h, :len(part)] = [0.0 if slots[j] is None else src[4][slots[j][0], h, slots[j][1]]
                                                      for j in part]
        return kept


class Decoder:
    """A model decoding over 8-bit caches, one per layer, from prompts of different lengths: the definition that
    gpt_generate_kv8 follows, with the tokens given by the caller.  ``noise(x)``, where given, is applied to every
    layer's q, k, v (to see what rounding errors before the quantisation do)."""

    def __init__(self, cfg, P, prompts, block_tokens, max_blocks, budget=0, recent=0, noise=None):
        self.cfg, self.params, self.budget, self.recent = cfg, P, budget, recent
        self.noise = noise if noise is not None else (lambda x: x)
        B, H, hd = len(prompts), cfg.n_head, cfg.n_embd // cfg.n_head
        self.H, self.hd, self.B = H, hd, B
        self.capacity = max_blocks * block_tokens
        n = 2 * B * max_blocks
        shape = (n, H, block_tokens, hd)
        self.tables = [np.arange(B * max_blocks).reshape(B, max_blocks), np.arange(B * max_blocks, n).reshape(B, max_blocks)]
        self.layers = [Cache(np.zeros(shape), np.zeros(shape), np.ones((n, H)), np.ones((n, H)), self.tables[0],
                             np.zeros(B, np.int64), np.zeros(shape[:3])) for _ in range(cfg.n_layer)]
        self.pos = np.array([len(p) for p in prompts])
        self.bound, self.evictions, self.kept, self.margins = int(self.pos.max()), 0, None, []
        start = np.concatenate([[0], np.cumsum(self.pos)])
        self.z = np.zeros((B, cfg.vocab_size))
        qkv = [[] for _ in self.layers]
        for b, p in enumerate(prompts):
            _, c = go.forward(cfg, P, np.asarray(p)[None], None)
            self.z[b] = c["z"][0, -1]
            for l, lc in enumerate(c["layers"]):
                qkv[l].append([self.noise(lc[x][0].transpose(1, 0, 2)) for x in "qkv"])
        for cache, parts in zip(self.layers, qkv):
            q, k, v = (np.concatenate([x[i] for x in parts]) for i in range(3))
            cache.append(k, v, start)
            if budget:
                cache.accumulate(cache.attention(q, start, hd ** -0.5)[2])
            cache.length = cache.length + self.pos

    def step(self, tokens):
        """Logits after one more token for each sequence."""
        cfg, P, B = self.cfg, self.params, self.B
        if self.budget and self.bound == self.capacity:
            self.tables = self.tables[::-1]
            self.kept = []
            for cache in self.layers:
                self.margins.append([_margin(cache, s, h, self.budget, self.recent) for s in range(B) for h in range(self.H)])
                self.kept.append(cache.evict(self.tables[0], self.budget, self.recent))
                cache.table, cache.length = self.tables[0], np.minimum(cache.length, self.budget)
            self.bound = self.budget
            self.evictions += 1
        self.bound += 1
        x = P["wte"][tokens] + P["wpe"][self.pos]
        self.pos = self.pos + 1
        start = np.arange(B + 1)
        gpt2 = cfg.variant == "gpt2"
        for l, cache in enumerate(self.layers):
            pre = f"h.{l}."
            a, _ = go._norm_fwd(cfg, x, P.get(pre + "ln_1.weight"), P.get(pre + "ln_1.bias"))
            y = a @ P[pre + "attn.c_attn.weight"].T + (P[pre + "attn.c_attn.bias"] if gpt2 else 0.0)
            q, k, v = (self.noise(t.reshape(B, self.H, self.hd)) for t in np.split(y, 3, axis=-1))
            cache.append(k, v, start)
            o, _, probs = cache.attention(q, start, self.hd ** -0.5)
            if self.budget:
                cache.accumulate(probs)
            cache.length = cache.length + 1
            x = x + o.reshape(B, -1) @ P[pre + "attn.c_proj.weight"].T + (P[pre + "attn.c_proj.bias"] if gpt2 else 0.0)
            a, _ = go._norm_fwd(cfg, x, P.get(pre + "ln_2.weight"), P.get(pre + "ln_2.bias"))
            h = a @ P[pre + "mlp.c_fc.weight"].T + (P[pre + "mlp.c_fc.bias"] if gpt2 else 0.0)
            x = x + go._act_fwd(cfg, h) @ P[pre + "mlp.c_proj.weight"].T + (P[pre + "mlp.c_proj.bias"] if gpt2 else 0.0)
        a, _ = go._norm_fwd(cfg, x, P.get("ln_f.weight"), P.get("ln_f.bias"))
        self.z = a @ (P["wte"] if gpt2 else P["lm_head.weight"]).T
        return self.z


def _margin(cache, s, h, budget, recent):
    """How far apart, relative to the larger, the lightest kept and the heaviest dropped weight are (inf: none dropped)."""
    n = int(cache.length[s])
    if n <= budget or recent == budget:
        return math.inf
    w = sorted((cache.weight[b, h, o] for b, o in cache._slots(s, n)[:n - recent]), reverse=True)
    return (w[budget - recent - 1] - w[budget - recent]) / w[budget - recent - 1]
