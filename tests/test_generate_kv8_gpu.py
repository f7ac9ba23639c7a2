"""gpt_generate_kv8: a model decoding over the 8-bit cache, from prompts of
different lengths, with eviction, against the float64 oracle (oracle/kv8.py's
Decoder) fed with the tokens that the GPU drew.

Tolerances.  A rounding before the quantisation can move a code by one step:
with q, k, v off by 1e-6 (fp32) the oracle's own logits move by up to 3.3e-4 at
these sizes, with 2^-8 (bf16: q, k, v rounded once, and activations before
them) by up to 0.036.  fp32: 2e-3 (six such codes).  bf16: 0.09 (0.036 and the
0.05 that bf16 generation without quantisation is tested with).  Kept slots are
compared where the weights on both sides of the budget's border differ by more
than 1e-3 of themselves (a moved code changes a weight by less)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

import oracle  # noqa: E402
from gpt_decoder_lm_b200 import binding as gb  # noqa: E402
from gpt_decoder_lm_b200 import workloads as W  # noqa: E402
from oracle import kv8 as O  # noqa: E402
from tests.helpers import oracle_config  # noqa: E402

TOL = {"fp32": 2e-3, "bf16": 0.09}
CASES = {"char": (W.CHAR, dict(n_layer=2, batch_size=4, block_size=128)),
         "micro": (W.MICRO, dict(n_layer=2, n_embd=64, n_head=2, block_size=64, batch_size=3))}


def setup(name, precision):
    w, over = CASES[name]
    w = w.with_(precision=precision)
    oc = oracle_config(w).with_(**over)
    return gb.Model(gb.make_config(w, **over), seed=w.weight_seed), oracle.init_params(oc, w.weight_seed), oc


def dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype))).cuda()


def make_cache(oc, P, max_blocks):
    n = oc.n_layer * oc.batch_size
    c = gb.KV8Cache.allocate(n, oc.n_head, oc.n_embd // oc.n_head, P, max_blocks, n_blocks=2 * n * max_blocks, weight=True)
    for t in (c.k, c.v):
        t.fill_(0x7f)  # NaN: nothing may depend on what the cache held
    return c, (c.table + n * max_blocks).contiguous()


def check(oc, params, out, logp, U, prompts, temps, greedy, n_new, P, max_blocks, budget, recent, tol):
    """Feeds the GPU's tokens to the oracle and checks every draw; the oracle's decoder."""
    d = O.Decoder(oc, params, prompts, P, max_blocks, budget, recent)
    sure = 0
    for i in range(n_new):
        for b, z in enumerate(d.z):
            tok = out[b, i]
            if greedy[b]:
                top = np.sort(z)[-2:]
                if top[1] - top[0] > 2 * tol:
                    assert tok == np.argmax(z), (i, b)
                    sure += 1
                assert z[tok] >= z.max() - 2 * tol, (i, b)
                assert logp[b, i] == 0.0 or temps[b] > 0
            else:  # temperature alone: u lies in the token's share, whose borders move by at most 2 tol / temperature
                p = np.exp((z - z.max()) / temps[b])
                c = np.cumsum(p) / p.sum()
                e = 2 * tol / temps[b]
                assert (c[tok - 1] if tok else 0.0) - e <= U[i, b] <= c[tok] + e, (i, b)
                assert abs(logp[b, i] - np.log(p[tok] / p.sum())) <= 2 * tol / temps[b]
        if i + 1 < n_new:
            d.step(out[:, i])
    assert sure >= n_new // 4
    return d


@pytest.mark.parametrize("name,precision,budget", [("char", "fp32", 0), ("char", "bf16", 0), ("micro", "fp32", 0),
                                                    ("char", "fp32", 24), ("char", "bf16", 24), ("micro", "fp32", 24),
                                                    ("micro", "bf16", 31)])
def test_generation_follows_the_oracle(name, precision, budget):
    m, params, oc = setup(name, precision)
    B, P = oc.batch_size, 16
    recent, max_blocks = min(6, budget), 2 if budget else oc.block_size // 16
    T0, n_new = 20, 40
    lens = [20, 9, 14, 1][:B]
    rng = np.random.default_rng(1)
    prompts = [rng.integers(0, oc.vocab_size, n) for n in lens]
    padded = np.full((B, T0), -5)  # what lies behind a prompt is not read
    for b, p in enumerate(prompts):
        padded[b, :len(p)] = p
    U = rng.random((n_new, B)).astype(np.float32)
    # greedy, plain sampling, and two filters that leave the largest alone
    temps = np.array([0.0, 0.9, 1.0, 0.7], np.float32)[:B]
    top_k, top_p = np.array([0, 0, 1, 0])[:B], np.array([1.0, 1.0, 1.0, 1e-6])[:B]
    cache, other = make_cache(oc, P, max_blocks)
    kept = torch.full((cache.n_seq, oc.n_head, max(budget, 1)), -1, dtype=torch.int32, device="cuda")
    out = torch.full((B, n_new), -1, dtype=torch.int32, device="cuda")
    logp = torch.full((B, n_new), 9.0, device="cuda")
    args = dict(prompt_len=dev(lens, np.int32), budget=budget, recent=recent, table_out=other if budget else None,
                kept=kept if budget else None, temperature=dev(temps, np.float32), top_k=dev(top_k, np.int32),
                top_p=dev(top_p, np.float32), min_p=dev(np.zeros(B), np.float32), logp=logp)
    first = cache.table
    n = m.generate_kv8(cache, dev(padded, np.int32), n_new, dev(U, np.float32), out, **args)
    got = out.cpu().numpy()
    assert ((got >= 0) & (got < oc.vocab_size)).all()
    greedy = [True, False, True, True][:B]
    d = check(oc, params, got, logp.cpu().numpy(), U, prompts, temps, greedy, n_new, P, max_blocks, budget, recent,
              TOL[precision])
    assert n == d.evictions and (n >= 4) == (budget > 0)
    assert cache.table is (other if n % 2 else first)
    want = np.concatenate([c.length for c in d.layers])
    assert cache.length.cpu().numpy().tolist() == want.tolist() and int(cache.flags) == 0
    if budget and precision == "fp32":
        sure = (np.array(d.margins).reshape(n, oc.n_layer, B, oc.n_head) > 1e-3).all(0)
        ref = np.stack(d.kept)
        same = (kept.cpu().numpy().reshape(ref.shape) == ref).all(-1)
        assert same[sure].all() and sure.mean() > 0.9
    m.close()


def test_repeated_calls_replay_and_take_new_contents():
    """Eager, captured and replayed calls give the same tokens; a replay reads the buffers' new contents."""
    m, _, oc = setup("char", "bf16")
    B, n_new, T0 = oc.batch_size, 30, 12
    cache, other = make_cache(oc, 16, 2)
    first = cache.table
    rng = np.random.default_rng(2)
    prompt = dev(rng.integers(0, oc.vocab_size, (B, T0)), np.int32)
    plen, U = dev([12, 3, 7, 1], np.int32), dev(rng.random((n_new, B)), np.float32)
    out, logp = torch.zeros(B, n_new, dtype=torch.int32, device="cuda"), torch.zeros(B, n_new, device="cuda")
    kept = torch.zeros(cache.n_seq, oc.n_head, 28, dtype=torch.int32, device="cuda")

    def call():
        cache.table = first
        m.generate_kv8(cache, prompt, n_new, U, out, prompt_len=plen, budget=28, recent=10, table_out=other, kept=kept,
                       logp=logp)
        return out.clone(), logp.clone()
    m.set_graphs(True)
    runs = [call() for _ in range(4)]
    for r in runs[1:]:
        assert torch.equal(r[0], runs[0][0]) and torch.equal(r[1], runs[0][1])
    prompt.copy_(torch.flip(prompt, (0,)))
    plen.copy_(dev([2, 12, 5, 9], np.int32))
    replayed = call()
    assert not torch.equal(replayed[0], runs[0][0])
    m.set_graphs(False)
    eager = call()
    assert torch.equal(replayed[0], eager[0]) and torch.equal(replayed[1], eager[1])
    # one plain generating call between does not disturb the next
    m.set_graphs(True)
    seq = torch.zeros(B, T0 + 4, dtype=torch.int32, device="cuda")
    m.generate(prompt, 4, 0.0, 0, 1.0, U[:4].contiguous(), seq)
    again = call()
    assert torch.equal(again[0], eager[0])
    m.close()


def test_prompt_lengths_and_tokens_are_checked():
    m, _, oc = setup("char", "bf16")
    B = oc.batch_size
    cache, _ = make_cache(oc, 16, 2)
    U, out = torch.zeros(3, B, device="cuda"), torch.zeros(B, 3, dtype=torch.int32, device="cuda")
    good = torch.zeros(B, 8, dtype=torch.int32, device="cuda")
    for lens in ([8, 0, 1, 1], [9, 1, 1, 1], [-3, 1, 1, 1]):
        with pytest.raises(gb.GptError) as e:
            m.generate_kv8(cache, good, 3, U, out, prompt_len=dev(lens, np.int32))
        assert e.value.name == "GPT_ERR_INVALID_ARG"
        m.clear_flags()
    bad = good.clone()
    bad[1, 2] = oc.vocab_size
    m.generate_kv8(cache, bad, 3, U, out, prompt_len=dev([8, 2, 8, 8], np.int32))  # behind the prompt's end
    with pytest.raises(gb.GptError) as e:
        m.generate_kv8(cache, bad, 3, U, out)
    assert e.value.name == "GPT_ERR_TOKEN_RANGE"
    m.close()


def test_refusals():
    m, _, oc = setup("char", "bf16")
    B = oc.batch_size
    cache, other = make_cache(oc, 16, 2)
    prompt = torch.zeros(B, 20, dtype=torch.int32, device="cuda")
    kept = torch.zeros(cache.n_seq, oc.n_head, 24, dtype=torch.int32, device="cuda")

    def call(n_new=10, p=prompt, c=cache, **kw):
        U, out = torch.zeros(max(n_new, 0), B, device="cuda"), torch.zeros(B, max(n_new, 0), dtype=torch.int32, device="cuda")
        return m.generate_kv8(c, p, n_new, U, out, **kw)
    assert call(n_new=13) == 0  # 20 + 13 - 1 = 32 slots
    for kw in (dict(n_new=0), dict(n_new=109), dict(n_new=14), dict(budget=24, recent=25, table_out=other, kept=kept),
               dict(budget=24, kept=kept), dict(budget=24, table_out=other), dict(budget=24, table_out=cache.table, kept=kept),
               dict(budget=32, table_out=other, kept=torch.zeros(cache.n_seq, oc.n_head, 32, dtype=torch.int32, device="cuda")),
               dict(budget=-1), dict(p=torch.zeros(B, 33, dtype=torch.int32, device="cuda")),
               dict(p=prompt.long()), dict(prompt_len=torch.zeros(B, device="cuda")),
               dict(c=make_cache(oc.with_(n_layer=1), 16, 2)[0]), dict(c=make_cache(oc.with_(n_head=3), 16, 2)[0])):
        with pytest.raises(gb.GptError):
            call(**kw)
    assert call(n_new=40, budget=24, recent=24, table_out=other, kept=kept) > 0
    m.close()


def test_recompute_is_refused():
    w, over = CASES["char"]
    m = gb.Model(gb.make_config(w.with_(precision="bf16"), recompute=1, **over), seed=1)
    cache, _ = make_cache(oracle_config(w).with_(**over), 16, 2)
    with pytest.raises(gb.GptError) as e:
        m.generate_kv8(cache, torch.zeros(4, 5, dtype=torch.int32, device="cuda"), 2, torch.zeros(2, 4, device="cuda"),
                       torch.zeros(4, 2, dtype=torch.int32, device="cuda"))
    assert e.value.name == "GPT_ERR_UNSUPPORTED"
    m.close()


@pytest.mark.parametrize("flags", [True, False])
def test_tables_outside_the_pool_are_reported(flags):
    """A block id outside the pool, in either table: the call returns an error, each time, whether or not the cache has a
    flag word of its own; a good call after it is good."""
    m, _, oc = setup("char", "bf16")
    B = oc.batch_size
    cache, other = make_cache(oc, 16, 2)
    if not flags:
        cache = gb.KV8Cache(cache.k, cache.v, cache.k_scale, cache.v_scale, cache.table, cache.length, cache.weight)
    n_new = 40
    prompt, U = torch.zeros(B, 8, dtype=torch.int32, device="cuda"), torch.full((n_new, B), 0.5, device="cuda")
    out = torch.zeros(B, n_new, dtype=torch.int32, device="cuda")
    kept = torch.zeros(cache.n_seq, oc.n_head, 24, dtype=torch.int32, device="cuda")
    first = cache.table.clone()

    def call(table, table_out):
        cache.table = table
        return m.generate_kv8(cache, prompt, n_new, U, out, budget=24, recent=10, table_out=table_out, kept=kept)
    call(first, other)
    good = out.clone()
    bad, bad_other = first.clone(), other.clone()
    bad[3, 1], bad_other[-1, 0] = cache.k.shape[0], -1
    for t, o in ((bad, other), (bad, other), (first, bad_other), (first, bad_other)):
        with pytest.raises(gb.GptError) as e:
            call(t, o)
        assert e.value.name == "GPT_ERR_INVALID_ARG"
        if flags:
            assert int(cache.flags) == gb.FLAG_BLOCK_RANGE
            cache.flags.zero_()
    call(first, other)
    assert torch.equal(out, good) and (not flags or int(cache.flags) == 0)
    # a prompt's length is checked at every call too
    for _ in range(2):
        cache.table = first
        with pytest.raises(gb.GptError) as e:
            m.generate_kv8(cache, prompt, 3, U[:3].contiguous(), torch.zeros(B, 3, dtype=torch.int32, device="cuda"),
                           prompt_len=dev([9, 1, 1, 1], np.int32))
        assert e.value.name == "GPT_ERR_INVALID_ARG"
    m.close()


@pytest.mark.parametrize("lens,T0,budget", [([9, 5, 3, 1], 20, 24), ([12, 12, 2, 7], 32, 20)])
def test_eviction_counts_from_the_longest_prompt(lens, T0, budget):
    """A buffer wider than its longest prompt: eviction comes when that one's next token does not fit, as the oracle has
    it, and the number of evictions, the lengths and the kept slots agree."""
    m, params, oc = setup("char", "fp32")
    B, P, max_blocks, recent, n_new = oc.batch_size, 16, 2, 6, 40
    rng = np.random.default_rng(7)
    prompts = [rng.integers(0, oc.vocab_size, n) for n in lens]
    padded = np.full((B, T0), -5)
    for b, p in enumerate(prompts):
        padded[b, :len(p)] = p
    U = rng.random((n_new, B)).astype(np.float32)
    cache, other = make_cache(oc, P, max_blocks)
    first = cache.table
    kept = torch.full((cache.n_seq, oc.n_head, budget), -1, dtype=torch.int32, device="cuda")
    out = torch.full((B, n_new), -1, dtype=torch.int32, device="cuda")
    plen, prompt, uniform = dev(lens, np.int32), dev(padded, np.int32), dev(U, np.float32)

    def call():
        cache.table = first
        return m.generate_kv8(cache, prompt, n_new, uniform, out, prompt_len=plen, budget=budget, recent=recent,
                              table_out=other, kept=kept)
    n = call()
    d = O.Decoder(oc, params, prompts, P, max_blocks, budget, recent)
    got = out.cpu().numpy()
    for i in range(n_new - 1):
        d.step(got[:, i])
    assert n == d.evictions and n > 0
    assert cache.length.cpu().numpy().tolist() == np.concatenate([c.length for c in d.layers]).tolist()
    sure = (np.array(d.margins).reshape(n, oc.n_layer, B, oc.n_head) > 1e-3).all(0)
    ref = np.stack(d.kept)
    assert (kept.cpu().numpy().reshape(ref.shape) == ref).all(-1)[sure].all() and sure.mean() > 0.9
    # other lengths in the same buffers are another call, not a replay of this one
    for _ in range(2):
        assert call() == n
    plen.copy_(dev([T0, 1, 2, 3], np.int32))
    prompt.copy_(dev(rng.integers(0, oc.vocab_size, (B, T0)), np.int32))
    longer, bound = 0, T0
    for _ in range(n_new - 1):
        if bound == max_blocks * P:
            longer, bound = longer + 1, budget
        bound += 1
    assert call() == longer != n
    m.close()
