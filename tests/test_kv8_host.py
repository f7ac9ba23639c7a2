"""Host side of the 8-bit cache: refusals of the C entry points (before any
device work) and the oracle's own format."""

import ctypes as C
import math

import numpy as np
import pytest

from gpt_decoder_lm_b200 import binding as gb
from oracle import kv8 as O

A = 4096  # a non-null, aligned address; nothing reads it


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return gb.lib()


def cache(**over):
    d = dict(n_seq=2, n_head_kv=2, head_dim=64, block_tokens=16, n_blocks=8, max_blocks=4, d_k=A, d_v=A, d_k_scale=A,
             d_v_scale=A, d_weight=A, d_table=A, d_len=A, d_flags=A)
    d.update(over)
    return gb.Kv8CacheStruct(*[d[n] for n, _ in gb.Kv8CacheStruct._fields_])


def append(lib, c, start=None, n_rows=2, max_new=1, k=A, k_ld=128, v=A, v_ld=128, bf16=1):
    return gb.STATUS[lib.gpt_kv8_append(C.byref(c), start, n_rows, max_new, bf16, k, k_ld, v, v_ld, None)]


@pytest.mark.parametrize("over,want", [
    ({"head_dim": 48}, "GPT_ERR_UNSUPPORTED"), ({"head_dim": 256}, "GPT_ERR_UNSUPPORTED"),
    ({"block_tokens": 8}, "GPT_ERR_UNSUPPORTED"), ({"block_tokens": 48}, "GPT_ERR_UNSUPPORTED"),
    ({"n_seq": 0}, "GPT_ERR_INVALID_ARG"), ({"n_seq": 70000}, "GPT_ERR_UNSUPPORTED"),
    ({"n_head_kv": 0}, "GPT_ERR_INVALID_ARG"), ({"n_head_kv": 40000}, "GPT_ERR_UNSUPPORTED"),
    ({"n_blocks": 0}, "GPT_ERR_INVALID_ARG"), ({"max_blocks": 0}, "GPT_ERR_INVALID_ARG"),
    ({"max_blocks": 1 << 28}, "GPT_ERR_UNSUPPORTED"),
    ({"d_k": None}, "GPT_ERR_INVALID_ARG"), ({"d_v": None}, "GPT_ERR_INVALID_ARG"),
    ({"d_k": A + 8}, "GPT_ERR_INVALID_ARG"), ({"d_v": A + 1}, "GPT_ERR_INVALID_ARG"),
    ({"d_k_scale": None}, "GPT_ERR_INVALID_ARG"), ({"d_v_scale": None}, "GPT_ERR_INVALID_ARG"),
    ({"d_table": None}, "GPT_ERR_INVALID_ARG"), ({"d_len": None}, "GPT_ERR_INVALID_ARG"),
])
def test_bad_caches_are_refused_by_every_call(lib, over, want):
    c = cache(**over)
    assert append(lib, c) == want
    assert gb.STATUS[lib.gpt_kv8_attention(C.byref(c), None, 2, 1, 4, 1, A, 256, 0.125, 0, A, 256, None, None)] == want
    assert gb.STATUS[lib.gpt_kv8_accumulate(C.byref(c), None, 2, 1, 4, 1, A, 256, 0.125, 0, A, None)] == want
    assert gb.STATUS[lib.gpt_kv8_evict(C.byref(c), 2 * A, 4, 8, 2, A, None)] == want
    assert gb.STATUS[lib.gpt_kv8_advance(C.byref(c), None, 2, 1, 0, None)] == want
    assert gb.STATUS[lib.gpt_kv8_append(None, None, 2, 1, 1, A, 128, A, 128, None)] == "GPT_ERR_INVALID_ARG"


@pytest.mark.parametrize("kw", [
    dict(n_rows=0), dict(n_rows=3), dict(max_new=0), dict(max_new=2), dict(start=A, n_rows=4, max_new=0),
    dict(k=None), dict(v=None), dict(k_ld=127), dict(v_ld=64), dict(k=A + 1), dict(v=A + 2, bf16=0)])
def test_bad_rows_are_refused(lib, kw):
    assert append(lib, cache(), **kw) == "GPT_ERR_INVALID_ARG"


def test_bad_attention_accumulate_evict_and_advance_arguments(lib):
    c = cache()

    def att(n_head=4, q=A, q_ld=256, scale=0.125, max_len=0, o=A, o_ld=256):
        return gb.STATUS[lib.gpt_kv8_attention(C.byref(c), None, 2, 1, n_head, 1, q, q_ld, scale, max_len, o, o_ld, None,
                                               None)]
    for kw in (dict(n_head=0), dict(n_head=3), dict(q=None), dict(o=None), dict(q_ld=255), dict(o_ld=1),
               dict(scale=math.nan), dict(max_len=-1)):
        assert att(**kw) == "GPT_ERR_INVALID_ARG", kw
    none = cache(d_weight=None)
    assert gb.STATUS[lib.gpt_kv8_accumulate(C.byref(none), None, 2, 1, 4, 1, A, 256, 0.125, 0, A, None)] == \
        "GPT_ERR_INVALID_ARG"
    assert gb.STATUS[lib.gpt_kv8_accumulate(C.byref(c), None, 2, 1, 4, 1, A, 256, 0.125, 0, None, None)] == \
        "GPT_ERR_INVALID_ARG"

    def evict(cc=c, table=2 * A, blocks=4, budget=8, recent=2, kept=A):
        return gb.STATUS[lib.gpt_kv8_evict(C.byref(cc), table, blocks, budget, recent, kept, None)]
    for kw in (dict(cc=none), dict(table=None), dict(table=A), dict(blocks=0), dict(budget=0), dict(budget=65),
               dict(recent=-1), dict(recent=9), dict(kept=None)):
        assert evict(**kw) == "GPT_ERR_INVALID_ARG", kw
    for n_rows, max_new, max_len in ((2, 1, -1), (2, -1, 0), (0, 1, 0)):
        assert gb.STATUS[lib.gpt_kv8_advance(C.byref(c), None, n_rows, max_new, max_len, None)] == "GPT_ERR_INVALID_ARG"


def test_oracle_codes_are_e4m3():
    """Known values of the format, and torch's own conversion on a grid."""
    torch = pytest.importorskip("torch")
    assert O.decode([0x00, 0x01, 0x08, 0x38, 0x7E, 0xFE]).tolist() == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 448.0, -448.0]
    x = np.concatenate([np.linspace(-448, 448, 20011), np.exp2(np.linspace(-12, 8, 4001))]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(O.encode(x), want)
    for a, e in ((448.0, 0), (448.1, 1), (1.75, -8), (1.76, -7), (0.0, O.E_MIN), (1e-38, O.E_MIN), (3e38, 120)):
        assert O.exponent(a) == e


def test_sample_rows_refusals(lib):
    def call(z=A, bf16=1, rows=2, V=10, ld=10, u=A, out=A):
        return gb.STATUS[lib.gpt_sample_rows(z, bf16, rows, V, ld, None, None, None, None, u, out, None, None)]
    for kw in (dict(z=None), dict(z=A + 1), dict(z=A + 2, bf16=0), dict(rows=0), dict(V=0), dict(ld=9), dict(u=None),
               dict(out=None)):
        assert call(**kw) == "GPT_ERR_INVALID_ARG", kw
    assert call(V=524289, ld=524289) == "GPT_ERR_UNSUPPORTED" and call(rows=65536) == "GPT_ERR_UNSUPPORTED"


def test_eviction_grid_limits(lib):
    """A budget or a number of destination blocks beyond what one launch covers is refused, not run in part."""
    import ctypes as C
    ptr = 1 << 20

    def call(n_seq, heads, budget, blocks):
        c = gb.Kv8CacheStruct(n_seq, heads, 64, 16, 8, 4, ptr, ptr, ptr, ptr, ptr, ptr, ptr, None)
        return gb.STATUS[lib.gpt_kv8_evict(C.byref(c), 2 * ptr, blocks, budget, 0, ptr, None)]
    assert call(65535, 32767, 17, 2) == "GPT_ERR_UNSUPPORTED"
    assert call(1, 1, (1 << 30) + 16, 1 << 30) == "GPT_ERR_UNSUPPORTED"
    assert call(1, 1, 33, 2) == "GPT_ERR_INVALID_ARG"
