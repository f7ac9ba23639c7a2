"""The 8-bit key / value cache (gpt_kv8_*) against the float64 oracle
(oracle/kv8.py).

Codes, scales and kept slots are exact: the library divides by powers of two
and rounds once, as the oracle does.  Attention: both sides read the same codes.

Tolerances, for values v with |v| <= V and rows of weights that sum to 1:
* bf16 rows.  The weights are rounded to fp16, at most 2^-11 each, and the
  fp32 sum adds less than 2^-14: |o - o64| <= 2^-10 V before the output's own
  rounding, 2^-8 |o64|.
* fp32 rows.  Queries and weights are held to 2^-22 as two fp16 terms.  A
  score's error is at most 2^-21 of sum |q k| (the terms and the fp32 sum of
  the MMA, which truncates), and moves a weight by as much relative to it; the
  base-2 exponential adds 2^-21.  With sum |q k| scale <= B:
  |o - o64| <= (2 B + 4) 2^-21 V.
* lse: B 2^-21 + 2^-20 absolute, and its own rounding 2^-23 |lse|; for bf16 rows
  the same (bf16 queries are exact in fp16, the sum is fp32).
* accumulated weights: rows * exp() with relative error (2 B + 4) 2^-20 in
  each term, all of one sign.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpt_decoder_lm_b200 import binding as gb  # noqa: E402
from oracle import kv8 as O  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def make(seed, lens, H, hd, P, extra=0, weight=True, spread=True, garbage=True):
    """A cache that holds quantised random tokens, its blocks in random order; what lies behind the sequences'
    tokens is garbage (NaN codes among it)."""
    rng = np.random.default_rng(seed)
    S, cap = len(lens), max(1, -(-(max(lens) + extra) // P))
    n_blocks = S * cap + 2
    table = rng.permutation(n_blocks)[:S * cap].reshape(S, cap).astype(np.int32)
    k = rng.integers(0, 256, (n_blocks, H, P, hd)).astype(np.uint8)
    v = rng.integers(0, 256, (n_blocks, H, P, hd)).astype(np.uint8)
    ks = np.exp2(rng.integers(-9, -5, (n_blocks, H)) if spread else np.full((n_blocks, H), -7)).astype(np.float32)
    vs = np.exp2(rng.integers(-10, -5, (n_blocks, H)) if spread else np.full((n_blocks, H), -7)).astype(np.float32)
    for s, n in enumerate(lens):  # the tokens' own codes are numbers
        for j in range(n):
            b, o = table[s, j // P], j % P
            for c in (k, v):
                x = c[b, :, o]
                x[(x & 127) == 127] ^= 64
    w = (rng.random((n_blocks, H, P)) ** 4 * 8).astype(np.float32)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    length = np.array(lens, np.int32)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpu = gb.KV8Cache(t(k), t(v), t(ks), t(vs), t(table), t(length), t(w) if weight else None, flags)
    return gpu, O.Cache(k, v, ks, vs, table, length, w if weight else None), rng


def starts(news):
    return np.concatenate([[0], np.cumsum(news)]).astype(np.int32)


def rows_of(rng, n, heads, hd, dtype, wide=True, gain=1.0):
    """[n, heads, hd] rows, part of wider ones, and the same values in float64."""
    x = torch.from_numpy(rng.standard_normal((n, heads + (2 if wide else 0), hd)).astype(np.float32) * gain).to(DT[dtype])
    view = x.cuda()[:, (1 if wide else 0):(1 if wide else 0) + heads]
    return view, x[:, (1 if wide else 0):(1 if wide else 0) + heads].double().numpy()


def same_cache(gpu, ref):
    assert np.array_equal(gpu.k.cpu().numpy(), ref.k)
    assert np.array_equal(gpu.v.cpu().numpy(), ref.v)
    assert np.array_equal(gpu.k_scale.cpu().numpy().astype(np.float64), ref.ks)
    assert np.array_equal(gpu.v_scale.cpu().numpy().astype(np.float64), ref.vs)


def dev(a):
    return None if a is None else torch.from_numpy(a).cuda()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,news,H,hd,P", [
    ([0, 5, 15, 16, 40], [1, 1, 1, 1, 1], 2, 64, 16),
    ([0, 5, 31, 32, 33], [70, 0, 1, 3, 64], 3, 32, 32),
    ([7], [300], 1, 128, 128),
    ([0, 63], [64, 2], 5, 128, 64),
])
def test_append_codes(lens, news, H, hd, P, dtype):
    gpu, ref, rng = make(1, lens, H, hd, P, extra=max(news))
    st = starts(news)
    k, k64 = rows_of(rng, int(st[-1]), H, hd, dtype, gain=0.3)
    v, v64 = rows_of(rng, int(st[-1]), H, hd, dtype)
    gpu.append(k, v, start=dev(st), max_new=max(news))
    ref.append(k64, v64, st)
    same_cache(gpu, ref)
    assert np.array_equal(gpu.weight.cpu().numpy().astype(np.float64), ref.weight)
    assert int(gpu.flags) == 0
    assert gpu.length.tolist() == lens


def test_append_one_row_a_sequence_and_unaligned_rows():
    gpu, ref, rng = make(2, [3, 16, 0, 9], 2, 64, 16, extra=1)
    base = torch.randn(4 * 2 * 2 * 64 + 3, device="cuda").bfloat16()
    k = base[1:1 + 4 * 128].reshape(4, 2, 64)          # 2-byte aligned
    v = base[3:3 + 4 * 129].as_strided((4, 2, 64), (129, 64, 1), 3)  # odd pitch
    gpu.append(k, v)
    ref.append(k.double().cpu().numpy(), v.double().cpu().numpy(), starts([1] * 4))
    same_cache(gpu, ref)


def test_append_scale_grows_and_subnormals():
    """Token by token into one block, each larger than the last: the earlier codes are rounded to the larger scale,
    down to zero."""
    gpu, ref, _ = make(3, [0], 1, 32, 16, extra=16)
    rng = np.random.default_rng(4)
    for i in range(16):
        x = (rng.standard_normal((1, 1, 32)) * 2.0 ** (i * 1.5 - 8)).astype(np.float32)
        gpu.append(torch.from_numpy(x).cuda(), torch.from_numpy(-x).cuda())
        ref.append(x.astype(np.float64), -x.astype(np.float64), starts([1]))
        same_cache(gpu, ref)
        gpu.advance()
        ref.length += 1
    assert int(gpu.length) == 16


@pytest.mark.parametrize("value", [0.0, 448.0, 449.0, 1e-38, 1e-45, 3e38, 2.0 ** -119, 7.0 * 2.0 ** -120])
def test_append_extremes(value):
    gpu, ref, _ = make(5, [0], 1, 32, 16, extra=2)
    x = np.zeros((2, 1, 32), np.float32)
    x[0, 0, 3] = value
    x[1, 0, 4] = -value / 3
    gpu.append(torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), start=dev(starts([2])), max_new=2)
    ref.append(x.astype(np.float64), x.astype(np.float64), starts([2]))
    same_cache(gpu, ref)


def test_append_not_finite():
    gpu, _, _ = make(6, [0], 1, 32, 16, extra=4)
    x = np.ones((4, 1, 32), np.float32)
    x[1, 0, 5], x[2, 0, 6], x[3, 0, 7] = np.nan, np.inf, -np.inf
    gpu.append(torch.from_numpy(x).cuda(), torch.from_numpy(x).cuda(), start=dev(starts([4])), max_new=4)
    b = int(gpu.table[0, 0])
    got = O.decode(gpu.k.cpu().numpy()[b, 0, :4]) * float(gpu.k_scale[b, 0])
    bad = ~np.isfinite(x[:, 0])
    assert np.isnan(got[bad]).all() and (got[~bad] == 1.0).all()


def check_attention(gpu, ref, q, q64, st, news, dtype, scale=None, max_len=0, v_max=None, out=None):
    n, H, hd = q.shape
    out = torch.full((n, H, hd), 7.0, dtype=DT[dtype], device="cuda") if out is None else out
    lse = torch.full((n, H), 7.0, device="cuda")
    gpu.attention(q, out, start=dev(st), max_new=max(max(news), 1), lse=lse, scale=scale, max_len=max_len)
    sc = hd ** -0.5 if scale is None else scale
    o64, l64, probs = ref.attention(q64, st, sc)
    G = H // ref.k.shape[1]
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for s, n_new in enumerate(news):
        if n_new == 0:
            continue
        r = slice(st[s], st[s + 1])
        kk, there = ref.values(s, int(ref.length[s]) + n_new, "k")
        vv, _ = ref.values(s, int(ref.length[s]) + n_new, "v")
        B = max(float(np.max(np.abs(sc) * np.abs(kk[:, h // G]) @ np.abs(q64[r, h]).T)) for h in range(H)) if len(kk) else 0.0
        V = float(np.abs(vv).max()) if len(vv) else 0.0
        tol = (2 * B + 4) * 2.0 ** -21 * V
        tol_o = tol + (2.0 ** -10 * V + 2.0 ** -8 * np.abs(o64[r]) if dtype == "bf16" else 2.0 ** -24 * np.abs(o64[r]))
        assert (np.abs(got[r] - o64[r]) <= tol_o + 1e-30).all(), (s, np.abs(got[r] - o64[r]).max(), np.min(tol_o))
        inf = np.isneginf(l64[r])
        assert np.array_equal(np.isneginf(gl[r]), inf)
        d = np.abs(gl[r][~inf] - l64[r][~inf])
        assert (d <= B * 2.0 ** -21 + 2.0 ** -20 + 2.0 ** -23 * np.abs(l64[r])[~inf]).all(), (s, d.max())
    return out, lse, probs


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,P,H,G", [(64, 16, 3, 1), (128, 64, 2, 4), (32, 128, 1, 8), (64, 32, 2, 12), (128, 16, 1, 16),
                                      (32, 16, 2, 3)])
def test_attention_one_token(hd, P, H, G, dtype):
    lens = [0, 1, 15, 16, 31, 47, 130, 700]
    gpu, ref, rng = make(10, [n + 1 for n in lens], H, hd, P)
    ref.length -= 1
    gpu.length -= 1
    q, q64 = rows_of(rng, len(lens), H * G, hd, dtype)
    check_attention(gpu, ref, q, q64, starts([1] * len(lens)), [1] * len(lens), dtype)
    assert int(gpu.flags) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,P,H,G,lens,news", [
    (64, 16, 2, 1, [0, 3, 40], [1, 17, 33]),
    (64, 32, 1, 3, [0, 100, 0, 7], [40, 0, 5, 2]),
    (128, 64, 1, 2, [61, 0], [5, 64]),
    (32, 128, 2, 5, [0, 300], [3, 2]),
])
def test_attention_many_tokens(hd, P, H, G, lens, news, dtype):
    gpu, ref, rng = make(11, [a + b for a, b in zip(lens, news)], H, hd, P)
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), H * G, hd, dtype)
    check_attention(gpu, ref, q, q64, st, news, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,P,H,G,lens,news", [
    (64, 16, 1, 1, [900, 0, 31], [70, 130, 17]), (128, 32, 1, 2, [300, 5], [40, 9]), (32, 64, 2, 1, [513, 64], [65, 16]),
    (64, 128, 1, 7, [50], [19]), (128, 16, 1, 1, [1000], [129]), (32, 16, 1, 3, [7], [64])])
def test_attention_blocks_of_rows(hd, P, H, G, lens, news, dtype):
    """More rows than one block of the kernel takes, and fewer; with and without a split over the slots (which goes by
    the bound on the lengths)."""
    gpu, ref, rng = make(17, [a + b for a, b in zip(lens, news)], H, hd, P)
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), H * G, hd, dtype)
    for max_len in (0, 1):
        check_attention(gpu, ref, q, q64, st, news, dtype, max_len=max_len)
    assert int(gpu.flags) == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,news", [(64, 1, [1, 1]), (64, 2, [6, 3]), (64, 1, [30, 20]), (64, 1, [100, 60]), (128, 1, [60, 1]),
                                       (32, 3, [40, 40])])
def test_attention_scales_and_offsets(hd, G, news, dtype):
    """A negative scale and a scale of 0 (every visible slot counts alike), rows of zeros, and q and out at an odd offset,
    for every form of the kernel."""
    lens = [70, 200]
    gpu, ref, rng = make(19, [a + b for a, b in zip(lens, news)], 1, hd, 16)
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), G, hd, dtype)
    q[-1] = 0
    q64[-1] = 0
    for scale in (-0.2, 0.0, 0.125):
        out, lse, _ = check_attention(gpu, ref, q, q64, st, news, dtype, scale=scale)
        wide = torch.full((2, q.shape[0], G * hd + 1), 5.0, dtype=q.dtype, device="cuda")
        wide[0, :, 1:] = q.flatten(1)
        at = wide[:, :, 1:].unflatten(2, (G, hd))
        got_lse = torch.zeros_like(lse)
        gpu.attention(at[0], at[1], start=dev(st), max_new=max(news), lse=got_lse, scale=scale)
        assert torch.equal(at[1], out) and torch.equal(got_lse, lse) and (wide[1, :, 0] == 5.0).all()


@pytest.mark.parametrize("max_len", [0, 1])
def test_attention_blocks_of_rows_with_holes_and_nan(max_len):
    """Block ids outside the pool, and NaN in V, among many rows; a sequence none of whose blocks is in the pool."""
    gpu, ref, rng = make(18, [300, 90], 1, 64, 16)
    table = ref.table.copy()
    table[0, [0, 3, 17]] = [-1, ref.k.shape[0], 2 ** 31 - 1]
    table[1] = -1
    ref.table = table
    gpu.table = torch.from_numpy(table).cuda()
    news = [100, 90]
    ref.length[:] = [200, 0]
    gpu.length.copy_(torch.tensor([200, 0], dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, 190, 2, 64, "bf16")
    out, lse, _ = check_attention(gpu, ref, q, q64, st, news, "bf16", max_len=max_len)
    assert (out[100:] == 0).all() and torch.isneginf(lse[100:]).all() and int(gpu.flags) == gb.FLAG_BLOCK_RANGE
    want = torch.isnan(out)
    assert not want.any()
    for slot, dim in ((250, 3), (170, 60)):  # the first is seen by the rows from 50 on, the second by all
        gpu.v[int(table[0, slot // 16]), 0, slot % 16, dim] = 0xFF
    gpu.attention(q, out, start=dev(st), max_new=100, max_len=max_len)
    want[50:100, :, 3] = True
    want[:100, :, 60] = True
    assert torch.equal(torch.isnan(out), want)


@pytest.mark.parametrize("max_len", [0, 1])
@pytest.mark.parametrize("hd,G,n", [(128, 1, 20), (128, 2, 70), (64, 1, 100), (32, 5, 30)])
def test_attention_sums_of_tiles_in_fp32(hd, G, n, max_len):
    """Lengths around multiples of the slots between which fp32 sums are set aside, with running maxima that grow from
    tile to tile, so that what was set aside is scaled too; one sequence sees holes and one NaN."""
    lens = [64 * tiles + d for tiles in (3, 4, 5, 8, 9, 13) for d in (-1, 0, 1)]
    gpu, ref, rng = make(29, [m + n for m in lens], 1, hd, 16)
    for s in range(len(lens)):
        for b in range(ref.table.shape[1]):
            ref.ks[ref.table[s, b], 0] = 2.0 ** (b // 8 - 11)
    gpu.k_scale.copy_(torch.from_numpy(ref.ks.astype(np.float32)))
    table = ref.table.copy()
    table[4, [0, 5, 17]] = [-1, ref.k.shape[0], 2 ** 31 - 1]
    ref.table = table
    gpu.table = torch.from_numpy(table).cuda()
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    news = [n] * len(lens)
    st = starts(news)
    q, q64 = rows_of(rng, n * len(lens), G, hd, "fp32")
    out, lse, _ = check_attention(gpu, ref, q, q64, st, news, "fp32", max_len=max_len)
    assert torch.isfinite(out).all() and int(gpu.flags) == gb.FLAG_BLOCK_RANGE
    gpu.v[int(table[-1, 3]), 0, 7, 9] = 0x7F  # slot 55 of the last sequence, which all its rows see
    again = torch.zeros_like(out)
    gpu.attention(q, again, start=dev(st), max_new=n, max_len=max_len)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[-n:, :, 9] = True
    assert torch.equal(torch.isnan(again), want) and torch.equal(again[~want], out[~want])


def test_attention_splits_agree_with_the_oracle():
    """One sequence, long enough to be split over a cluster's blocks; the bound on the length decides how."""
    gpu, ref, rng = make(12, [5001], 1, 64, 16)
    gpu.length -= 1
    ref.length -= 1
    q, q64 = rows_of(rng, 1, 2, 64, "fp32")
    for max_len in (0, 1, 300, 2500, 10 ** 6):
        check_attention(gpu, ref, q, q64, starts([1]), [1], "fp32", max_len=max_len)


@pytest.mark.parametrize("n,hd,P", [(1, 64, 16), (9, 128, 64), (40, 32, 16)])
def test_long_contexts_in_fp32(n, hd, P):
    """Over 20,000 slots fp32 outputs stay at fp32's accuracy.  Per weight: the score's error, 2^-23 of sum |q k| (q as
    two fp16 terms) and 2^-24 for each of the sums' steps, the exponential's 2^-22 and the weight's 2^-22; these are
    independent from slot to slot, as are the values, so that they stand to the output as to a weight: with sum |q k|
    about 8 and 8 steps below 2e-6 (a sum that is cut off, not rounded, at each of its steps leaves 7e-6)."""
    gen = torch.Generator(device="cuda").manual_seed(n)
    len_ = 20000
    blocks = -(-(len_ + n) // P)
    c = gb.KV8Cache.allocate(1, 1, hd, P, blocks)
    k = torch.randn(len_ + n, 1, hd, device="cuda", generator=gen)
    v = torch.randn(len_ + n, 1, hd, device="cuda", generator=gen)
    at = dev(starts([len_ + n]))
    c.append(k, v, start=at, max_new=len_ + n)
    c.length.fill_(len_)
    q = torch.randn(n, 2, hd, device="cuda", generator=gen)
    out, lse = torch.zeros_like(q), torch.zeros(n, 2, device="cuda")
    c.attention(q, out, start=dev(starts([n])), max_new=n, lse=lse)

    def values(codes, scale):
        x = codes.view(torch.float8_e4m3fn).double() * scale.double()[:, :, None, None]
        return x.transpose(0, 1).reshape(-1, hd)[:len_ + n]
    z = torch.einsum("ihd,jd->ihj", q.double(), values(c.k, c.k_scale)) * hd ** -0.5
    z.masked_fill_((torch.arange(len_ + n, device="cuda") > len_ + torch.arange(n, device="cuda")[:, None])[:, None], -np.inf)
    want = torch.softmax(z, -1) @ values(c.v, c.v_scale)
    assert float((out.double() - want).norm() / want.norm()) <= 2e-6
    assert float((lse.double() - torch.logsumexp(z, -1)).abs().max()) <= 4e-6


def test_attention_scale_ranges():
    """Blocks whose value scales are far apart, and where the large weight sits on the small values."""
    gpu, ref, rng = make(13, [64], 1, 64, 16, spread=False)
    for i, e in enumerate([-60, 20, -7, -30]):
        b = int(ref.table[0, i])
        ref.vs[b] = 2.0 ** e
        gpu.v_scale[b] = 2.0 ** e
    ref.length -= 1
    gpu.length -= 1
    q, q64 = rows_of(rng, 1, 1, 64, "fp32", gain=0.2)
    check_attention(gpu, ref, q, q64, starts([1]), [1], "fp32")
    # all weight on the block with scale 2^-60: its values come out to fp32 accuracy of themselves
    k = ref.k.copy()
    k[:] = O.encode(np.zeros(k.shape))
    k[int(ref.table[0, 0]), 0, :, 0] = O.encode(np.array(448.0))
    ref.k = k
    gpu.k.copy_(torch.from_numpy(k))
    q64 = np.zeros((1, 1, 64))
    q64[0, 0, 0] = 1000.0
    q = torch.from_numpy(q64.astype(np.float32)).cuda()
    out = torch.zeros(1, 1, 64, device="cuda")
    gpu.attention(q, out)
    o64, _, _ = ref.attention(q64, starts([1]), 0.125)
    assert np.abs(out.double().cpu().numpy() - o64).max() <= 2.0 ** -19 * 448 * 2.0 ** -60


def test_attention_nan_reaches_only_rows_that_see_it():
    """A NaN in a token's V (and in another's K) makes the rows that see it NaN, in that dimension (or all), and no
    earlier row."""
    gpu, ref, rng = make(14, [40], 1, 64, 16)
    gpu.length.fill_(20)
    b = int(ref.table[0, 30 // 16])
    gpu.v[b, 0, 30 % 16, 11] = 0x7F
    q, _ = rows_of(rng, 20, 1, 64, "bf16")
    out = torch.zeros(20, 1, 64, dtype=torch.bfloat16, device="cuda")
    gpu.attention(q, out, start=dev(starts([20])), max_new=20)
    nan = torch.isnan(out[:, 0]).cpu().numpy()
    want = np.zeros((20, 64), bool)
    want[10:, 11] = True
    assert np.array_equal(nan, want)
    gpu.k[b, 0, 30 % 16, 5] = 0xFF
    gpu.attention(q, out, start=dev(starts([20])), max_new=20)
    nan = torch.isnan(out[:, 0]).cpu().numpy()
    assert nan[10:].all() and not nan[:10].any()


def test_bad_tables_and_offsets_are_left_out():
    """Block ids outside the pool, offsets out of order and tokens past the capacity: nothing is read or written there,
    the rest is as ever, and the flag word says so."""
    gpu, ref, rng = make(15, [33, 20, 16], 2, 64, 16)
    table = ref.table.copy()
    table[0, 1], table[1, 0], table[1, 1] = -1, ref.k.shape[0], 2 ** 31 - 1
    ref.table = table
    gpu.table = torch.from_numpy(table).cuda()
    ref.length -= 1
    gpu.length -= 1
    q, q64 = rows_of(rng, 3, 2, 64, "fp32")
    out, lse, probs = check_attention(gpu, ref, q, q64, starts([1] * 3), [1] * 3, "fp32")
    assert (out[1] == 0).all() and torch.isneginf(lse[1]).all()  # sequence 1 has no block at all
    assert int(gpu.flags) == gb.FLAG_BLOCK_RANGE
    gpu.accumulate(q, lse)
    ref.accumulate(probs)
    np.testing.assert_allclose(gpu.weight.cpu().numpy(), ref.weight, rtol=1e-4)
    gpu.append(q, q)
    ref.append(q64, q64, starts([1] * 3))
    same_cache(gpu, ref)
    gpu.flags.zero_()
    # sequence 1's offsets descend: it has no rows; sequence 0 takes more than max_new
    before = gpu.k.clone()
    gpu.append(q, q, start=torch.tensor([0, 3, 2, 3], dtype=torch.int32, device="cuda"), max_new=2)
    assert int(gpu.flags) == gb.FLAG_ROW_RANGE
    changed = (gpu.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert set(changed) <= {int(table[2, 15 // 16])}
    gpu.flags.zero_()
    gpu.length.fill_(48)  # the capacity
    before = gpu.k.clone()
    gpu.append(q, q)
    assert int(gpu.flags) == gb.FLAG_CACHE_FULL and torch.equal(gpu.k, before)


@pytest.mark.parametrize("n", [1, 5, 70])
def test_bound_on_new_rows_above_the_rows(n):
    """max_new is a bound: a caller's own, larger than all the rows of this step, changes nothing."""
    results = []
    for max_new in (n, 1000, 2 ** 31 - 1):
        gpu, ref, rng = make(22, [40 + n], 2, 64, 16)
        gpu.length.fill_(40)
        q, _ = rows_of(rng, n, 4, 64, "bf16")
        k, _ = rows_of(rng, n, 2, 64, "bf16")
        out, lse, st = torch.zeros_like(q), torch.zeros(n, 4, device="cuda"), dev(starts([n]))
        gpu.append(k, k, start=st, max_new=max_new)
        gpu.attention(q, out, start=st, max_new=max_new, lse=lse)
        gpu.accumulate(q, lse, start=st, max_new=max_new)
        gpu.advance(start=st, n_rows=n, max_new=max_new)
        results.append((gpu.k, gpu.v, gpu.k_scale, out, lse, gpu.weight, gpu.length))
        assert int(gpu.flags) == 0 and int(gpu.length[0]) == 40 + n
    for other in results[1:]:
        for x, y in zip(results[0], other):
            assert torch.equal(x.nan_to_num(), y.nan_to_num()) if x.is_floating_point() else torch.equal(x, y)


def test_rows_behind_the_last_sequence_stay():
    gpu, ref, rng = make(16, [5, 9], 1, 64, 16)
    gpu.length.fill_(3)
    ref.length[:] = 3
    st = np.array([0, 2, 3], np.int32)
    q, q64 = rows_of(rng, 6, 1, 64, "bf16")
    out, lse, _ = check_attention(gpu, ref, q, q64, st, [2, 1], "bf16")
    assert (out[3:] == 7).all() and (lse[3:] == 7).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,P,H,G,lens,news", [
    (64, 16, 3, 1, [0, 1, 33, 600], [1, 1, 1, 1]),
    (128, 64, 1, 4, [5, 300], [20, 3]),
    (32, 32, 2, 7, [0, 63, 64], [65, 0, 2]),
    (64, 128, 1, 20, [129], [1]),
])
def test_accumulate(hd, P, H, G, lens, news, dtype):
    gpu, ref, rng = make(20, [a + b for a, b in zip(lens, news)], H, hd, P)
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), H * G, hd, dtype, gain=0.5)
    out, lse, probs = check_attention(gpu, ref, q, q64, st, news, dtype)
    before = gpu.weight.clone().cpu().numpy()
    gpu.accumulate(q, lse, start=dev(st), max_new=max(news))
    w0 = ref.weight.copy()
    ref.accumulate(probs)
    got = gpu.weight.cpu().numpy().astype(np.float64)
    B = max(float(np.max(hd ** -0.5 * np.abs(ref.values(s, lens[s] + news[s], "k")[0][:, h // G])
                         @ np.abs(q64[st[s]:st[s + 1], h]).T, initial=0.0))
            for s in range(len(lens)) for h in range(H * G))
    gain = ref.weight - w0
    assert (np.abs(got - ref.weight) <= (2 * B + 4) * 2.0 ** -20 * gain + 2.0 ** -23 * ref.weight + 1e-30).all()
    assert np.array_equal(got[gain == 0], before[gain == 0])  # slots that no row sees
    # each row's weights sum to 1
    total = sum(n * H * G for n in news)
    assert abs((got - before).sum() - total) <= 1e-3 * total
    # again: the same sums, bit for bit
    gpu2, _, rng2 = make(20, [a + b for a, b in zip(lens, news)], H, hd, P)
    gpu2.length.copy_(torch.tensor(lens, dtype=torch.int32))
    gpu2.accumulate(q, lse, start=dev(st), max_new=max(news))
    assert torch.equal(gpu2.weight, gpu.weight)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,P,H,G,lens,news,max_len", [
    (64, 16, 1, 1, [150, 0, 31], [130, 70, 17], 0), (128, 32, 1, 2, [300, 5], [40, 9], 1), (32, 64, 2, 1, [200, 64], [65, 16], 0),
    (64, 128, 1, 7, [50], [19], 1), (32, 16, 1, 3, [7], [64], 100)])
def test_accumulate_many_rows(hd, P, H, G, lens, news, max_len, dtype):
    """More rows than a decoding step has, over several tiles of rows and blocks of slots, the grid smaller than the
    sequence (the bound on the lengths is a hint), a sequence with blocks outside the pool, and rows at an odd offset."""
    gpu, ref, rng = make(21, [a + b for a, b in zip(lens, news)], H, hd, P)
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    table = ref.table.copy()
    if len(lens) == 3:
        table[1] = -7
    ref.table = table
    gpu.table = torch.from_numpy(table).cuda()
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), H * G, hd, dtype, gain=0.5)
    out, lse, probs = check_attention(gpu, ref, q, q64, st, news, dtype, max_len=max_len)
    before = gpu.weight.clone()
    gpu.accumulate(q, lse, start=dev(st), max_new=max(news), max_len=max_len)
    w0 = ref.weight.copy()
    ref.accumulate(probs)
    got = gpu.weight.cpu().numpy().astype(np.float64)
    B = max(float(np.max(hd ** -0.5 * np.abs(ref.values(s, lens[s] + news[s], "k")[0][:, h // G])
                         @ np.abs(q64[st[s]:st[s + 1], h]).T, initial=0.0))
            for s in range(len(lens)) for h in range(H * G))
    gain = ref.weight - w0
    assert (np.abs(got - ref.weight) <= (2 * B + 4) * 2.0 ** -20 * gain + 2.0 ** -23 * ref.weight + 1e-30).all()
    assert np.array_equal(got[gain == 0], before.double().cpu().numpy()[gain == 0])  # slots that no row sees
    odd = torch.zeros(q.shape[0], q.shape[1] * hd + 1, dtype=q.dtype, device="cuda")
    odd[:, 1:] = q.flatten(1)
    first = gpu.weight.clone()
    gpu.weight.copy_(before)
    gpu.accumulate(odd[:, 1:].unflatten(1, q.shape[1:]), lse, start=dev(st), max_new=max(news), max_len=max_len)
    assert torch.equal(gpu.weight, first)


@pytest.mark.parametrize("H,hd,P,lens,budget,recent", [
    (2, 64, 16, [100, 30, 31, 64, 0, 1], 31, 7),
    (1, 128, 64, [1000], 257, 257),
    (3, 32, 32, [129, 400], 64, 0),
    (1, 64, 128, [300, 5], 1, 0),
    (2, 64, 16, [50], 1, 1),
])
def test_evict(H, hd, P, lens, budget, recent):
    gpu, ref, rng = make(30, lens, H, hd, P)
    S, out_cap = len(lens), -(-budget // P)
    # a pool with more blocks: those of the table to move into
    n0 = ref.k.shape[0]
    grow = lambda a: np.concatenate([a, rng.integers(0, 256, (S * out_cap,) + a.shape[1:]).astype(a.dtype)])  # noqa: E731
    ref = O.Cache(grow(ref.k), grow(ref.v), np.concatenate([ref.ks, np.ones((S * out_cap, H))]),
                  np.concatenate([ref.vs, np.ones((S * out_cap, H))]), ref.table, ref.length, grow(ref.weight))
    ref.weight[:n0][ref.weight[:n0] < 1e-3] = 0.0  # ties
    ref.weight[int(ref.table[0, 0]), 0, 0] = np.nan
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a.astype(d))).cuda()  # noqa: E731
    gpu = gb.KV8Cache(t(ref.k, np.uint8), t(ref.v, np.uint8), t(ref.ks, np.float32), t(ref.vs, np.float32),
                      t(ref.table, np.int32), t(ref.length, np.int32), t(ref.weight, np.float32), gpu.flags)
    ref.weight = gpu.weight.double().cpu().numpy()
    table_out = (n0 + rng.permutation(S * out_cap)).reshape(S, out_cap).astype(np.int32)
    kept = torch.full((S, H, budget), 99, dtype=torch.int32, device="cuda")
    gpu.evict(dev(table_out), budget, recent, kept)
    want = ref.evict(table_out, budget, recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    same_cache(gpu, ref)
    assert np.array_equal(gpu.weight.cpu().numpy().astype(np.float64), ref.weight, equal_nan=True)
    gpu.table = dev(table_out)
    gpu.advance(max_new=0, max_len=budget)
    assert gpu.length.tolist() == [min(n, budget) for n in lens]
    assert int(gpu.flags) == 0


def test_evict_ties_keep_the_lowest_slots_and_long_sequences():
    """Equal weights, and a sequence too long for the selection's shared memory."""
    for n, budget, recent in ((700, 300, 20), (45000, 900, 100)):
        H, hd, P = 1, 32, 128
        cap, out_cap = -(-n // P), -(-budget // P)
        c = gb.KV8Cache.allocate(1, H, hd, P, cap, n_blocks=cap + out_cap, weight=True)
        c.length.fill_(n)
        c.k_scale.fill_(1.0), c.v_scale.fill_(1.0)
        c.weight.fill_(0.25)
        heavy = torch.arange(0, n - recent, 50, device="cuda")[:200]
        c.weight.view(cap + out_cap, P)[heavy // P, heavy % P] = torch.rand(heavy.numel(), device="cuda") + 1.0
        kept = torch.zeros(1, 1, budget, dtype=torch.int32, device="cuda")
        c.evict(torch.arange(cap, cap + out_cap, dtype=torch.int32, device="cuda")[None].contiguous(), budget, recent, kept)
        h = set(heavy.tolist()[:budget - recent])
        rest = [j for j in range(n - recent) if j not in h][:budget - recent - len(h)]
        assert kept[0, 0].tolist() == sorted(h | set(rest)) + list(range(n - recent, n))


@pytest.mark.parametrize("P,most", [(16, 700), (128, 1024), (32, 1025), (64, 2048), (16, 2064)])
@pytest.mark.parametrize("kind", ["spread", "few values", "one value", "two values far apart", "negative and infinite"])
def test_evict_selection(P, most, kind):
    """The kept slots at the capacities where the selection changes its form, for weights that separate early, late or
    not at all, and budgets at both ends."""
    lens = [most, most - 1, most // 2, 3]
    gpu, ref, rng = make(60, lens, 2, 32, P)
    out_cap = -(-most // P)
    n = ref.k.shape[0]
    shape = ref.weight.shape
    w = {"spread": rng.random(shape) ** 4 * 8, "few values": rng.integers(0, 4, shape) * 0.25, "one value": np.full(shape, 0.5),
         "two values far apart": np.where(rng.random(shape) < 0.5, 1e-30, 1e30),
         "negative and infinite": np.where(rng.random(shape) < 0.1, np.inf, rng.standard_normal(shape))}[kind].astype(np.float32)
    grown = torch.zeros(n + 4 * out_cap, *gpu.k.shape[1:], dtype=torch.uint8, device="cuda")
    grown[:n] = gpu.k
    weight = torch.zeros(n + 4 * out_cap, *shape[1:], device="cuda")
    weight[:n] = torch.from_numpy(w).cuda()
    scale = torch.ones(n + 4 * out_cap, 2, device="cuda")
    c = gb.KV8Cache(grown, grown.clone(), scale, scale.clone(), gpu.table, gpu.length, weight, gpu.flags)
    to = torch.arange(n, n + 4 * out_cap, dtype=torch.int32, device="cuda").reshape(4, out_cap)
    for budget, recent in ((1, 0), (most // 3, 5), (most - 1, 1), (most // 2, most // 2), (most, 0)):
        kept = torch.full((4, 2, budget), -9, dtype=torch.int32, device="cuda")
        c.evict(to, budget, recent, kept)
        got = kept.cpu().numpy()
        for s, length in enumerate(lens):
            for h in range(2):
                ws = np.concatenate([w[b, h] for b in ref.table[s]])[:length].astype(np.float64)
                if length <= budget:
                    want = np.concatenate([np.arange(length), np.full(budget - length, -1)])
                else:
                    m = length - recent
                    heavy = np.lexsort((np.arange(m), -ws[:m]))[:budget - recent]
                    want = np.concatenate([np.sort(heavy), np.arange(m, length)])
                assert np.array_equal(got[s, h], want), (budget, recent, s, h)
    assert int(c.flags) == 0


def test_a_run_of_steps_with_eviction():
    """Append, attention, accumulation, eviction and advance over many steps, as decoding uses them."""
    rng = np.random.default_rng(40)
    S, H, G, hd, P, budget, recent, most = 3, 2, 2, 64, 16, 40, 8, 56
    cap, out_cap = -(-most // P), -(-budget // P)
    c = gb.KV8Cache.allocate(S, H, hd, P, cap, n_blocks=2 * S * cap, weight=True)
    tables = [c.table, c.table + S * cap]
    ref = O.Cache(c.k.cpu().numpy(), c.v.cpu().numpy(), c.k_scale.cpu().numpy(), c.v_scale.cpu().numpy(),
                  c.table.cpu().numpy(), c.length.cpu().numpy(), c.weight.cpu().numpy())
    st = starts([21, 3, 1])  # prompts
    news = [21, 3, 1]
    kept = torch.zeros(S, H, budget, dtype=torch.int32, device="cuda")
    for step in range(60):
        n = int(st[-1])
        q, q64 = rows_of(rng, n, H * G, hd, "bf16")
        k, k64 = rows_of(rng, n, H, hd, "bf16")
        v, v64 = rows_of(rng, n, H, hd, "bf16")
        c.append(k, v, start=dev(st), max_new=max(news))
        ref.append(k64, v64, st)
        same_cache(c, ref)
        out, lse, probs = check_attention(c, ref, q, q64, st, news, "bf16")
        c.accumulate(q, lse, start=dev(st), max_new=max(news))
        ref.accumulate(probs)
        np.testing.assert_allclose(c.weight.cpu().numpy(), ref.weight, rtol=1e-4, atol=1e-6)
        ref.weight = c.weight.double().cpu().numpy()  # so that near ties fall alike
        c.advance(start=dev(st), n_rows=n, max_new=max(news))
        ref.length = ref.length + np.array(news)
        if ref.length.max() >= most - 1:
            tables = tables[::-1]
            c.evict(tables[0], budget, recent, kept)
            assert np.array_equal(kept.cpu().numpy(), ref.evict(tables[0].cpu().numpy(), budget, recent))
            c.table = tables[0]
            c.advance(max_new=0, max_len=budget)
            ref.table, ref.length = tables[0].cpu().numpy(), np.minimum(ref.length, budget)
            same_cache(c, ref)
        assert c.length.tolist() == ref.length.tolist()
        st, news = starts([1] * S), [1] * S
    assert int(c.flags) == 0


def test_captured_and_on_another_stream():
    """A captured step replays on new contents; a step on another stream gives the same bits."""
    gpu, ref, rng = make(50, [30, 100], 2, 64, 16, extra=4)
    q, _ = rows_of(rng, 2, 4, 64, "bf16", wide=False)
    k, _ = rows_of(rng, 2, 2, 64, "bf16", wide=False)
    out, lse = torch.zeros_like(q), torch.zeros(2, 4, device="cuda")

    def step():
        gpu.append(k, k)
        gpu.attention(q, out, lse=lse)
        gpu.accumulate(q, lse)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        k.copy_(torch.randn_like(k))
        q.copy_(torch.randn_like(q))
        w = gpu.weight.clone()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone(), gpu.weight.clone(), gpu.k.clone()
        gpu.weight.copy_(w)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        s.synchronize()
        for a, b in zip(got, (out, lse, gpu.weight, gpu.k)):
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes of codes: the last blocks hold the sequence."""
    hd, P, H = 128, 128, 64
    per = H * P * hd  # bytes of a block: 1 MiB
    n_blocks = (1 << 32) // per + 4
    k = torch.zeros(n_blocks, H, P, hd, dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    ks = torch.full((n_blocks, H), 2.0 ** -7, device="cuda")
    table = torch.tensor([[n_blocks - 1, n_blocks - 2]], dtype=torch.int32, device="cuda")
    length = torch.tensor([130], dtype=torch.int32, device="cuda")
    c = gb.KV8Cache(k, v, ks, ks.clone(), table, length)
    x = torch.randn(1, H, hd, device="cuda")
    c.append(x, x)
    assert int((k[n_blocks - 2, :, 2] != 0).sum()) > H * hd // 2 and int(k[:4].max()) == 0
    out = torch.zeros(1, H, hd, device="cuda")
    c.attention(torch.zeros_like(x), out)  # the mean of the values
    got = (out * 131 - x).abs().max()
    assert float(got) <= 2.0 ** -3 * float(x.abs().max())  # the codes' rounding, 2^-4 of the value


def zeros_cache(H, hd, P, lens, budget, k, v, ks, vs, w, table):
    """A cache with the given numpy contents, and the blocks behind them for the kept slots; the oracle's copy."""
    S, n0, out_cap = len(lens), k.shape[0], -(-budget // P)
    grow = lambda a, x: np.concatenate([a, np.full((S * out_cap,) + a.shape[1:], x, a.dtype)])  # noqa: E731
    ref = O.Cache(grow(k, 0x7F), grow(v, 0x7F), grow(ks, 1.0), grow(vs, 1.0), table, np.array(lens), grow(w, 0.0))
    t = lambda a, d: torch.from_numpy(np.ascontiguousarray(a.astype(d))).cuda()  # noqa: E731
    gpu = gb.KV8Cache(t(ref.k, np.uint8), t(ref.v, np.uint8), t(ref.ks, np.float32), t(ref.vs, np.float32),
                      t(table, np.int32), t(ref.length, np.int32), t(ref.weight, np.float32),
                      torch.zeros(1, dtype=torch.int32, device="cuda"))
    return gpu, ref, np.arange(n0, n0 + S * out_cap, dtype=np.int32).reshape(S, out_cap)


@pytest.mark.parametrize("kind", ["zero tokens of blocks with others", "zeros beside far smaller values", "NaN tokens and zeros",
                                  "blocks outside the pool"])
@pytest.mark.parametrize("H,hd,P", [(2, 64, 16), (1, 128, 64), (3, 32, 32), (1, 128, 128)])
def test_evict_keeps_zeros(H, hd, P, kind):
    """Kept codes that are zero stay zero (of either sign), however far apart their block's scale and the new block's are:
    a block none of whose kept tokens is anything but zero has the smallest exponent."""
    rng = np.random.default_rng(hd + P)
    n = 2 * P
    table = np.array([[1, 0]], np.int32)
    k = rng.choice(np.array([0, 128], np.uint8), (2, H, P, hd))  # zeros of both signs
    v = rng.choice(np.array([0, 128], np.uint8), (2, H, P, hd))
    ks, vs = np.full((2, H), 2.0 ** -8), np.full((2, H), 2.0 ** 3)
    heavy = rng.permutation(n - 1)[:P]  # the kept ones, beside the last
    w = np.zeros((2, H, P))
    for j in heavy:
        w[table[0, j // P], :, j % P] = 1.0 + rng.random(H)
    dropped = np.setdiff1d(np.arange(n - 1), heavy)
    for j in dropped:  # what is not kept has values
        for c in (k, v):
            c[table[0, j // P], :, j % P] = rng.integers(0, 127, (H, hd))
    if kind == "zeros beside far smaller values":
        ks[1], vs[1] = 2.0 ** 20, 2.0 ** 40
        ks[0], vs[0] = 2.0 ** -30, 2.0 ** -100
        for j in range(P, n):
            for c in (k, v):
                c[0, :, j % P, ::3] = rng.integers(0, 127, c[0, :, j % P, ::3].shape)
    if kind == "NaN tokens and zeros":
        for j in heavy[::2]:
            k[table[0, j // P], :, j % P] = 0x7F
            v[table[0, j // P], :, j % P, 5] = 0xFF
    if kind == "blocks outside the pool":
        table = np.array([[-1, 2 + 5 * P]], np.int32)
    gpu, ref, to = zeros_cache(H, hd, P, [n], P + 1, k, v, ks, vs, w, table)
    kept = torch.zeros(1, H, P + 1, dtype=torch.int32, device="cuda")
    gpu.evict(dev(to), P + 1, 1, kept)
    assert np.array_equal(kept.cpu().numpy(), ref.evict(to, P + 1, 1))
    assert np.array_equal(gpu.k_scale.cpu().numpy().astype(np.float64), ref.ks)
    assert np.array_equal(gpu.v_scale.cpu().numpy().astype(np.float64), ref.vs)
    for got, want in ((gpu.k, ref.k), (gpu.v, ref.v)):
        got = got.cpu().numpy()
        nan = (want & 127) == 127
        assert np.array_equal((got & 127) == 127, nan) and np.array_equal(got[~nan], want[~nan])
    assert int(gpu.flags) == (gb.FLAG_BLOCK_RANGE if kind == "blocks outside the pool" else 0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,news", [(64, 1, [1, 1, 1]), (64, 2, [6, 3, 1]), (64, 1, [30, 20, 3]), (64, 1, [100, 60, 2]),
                                       (128, 1, [60, 1, 20]), (32, 3, [40, 40, 1])])
@pytest.mark.parametrize("scale,gain", [(0.125, 2.0 ** -70), (0.125, 2.0 ** -30), (0.0, 1.0), (1e-38, 1.0)])
def test_attention_factors_of_scores_that_underflow(hd, G, news, dtype, scale, gain):
    """All-zero key blocks (the smallest scale) and tiny queries or scales: the scores are zero, and what a row does not
    see stays unseen, in every form of the kernel."""
    lens = [70, 9, 37]
    gpu, ref, rng = make(23, [a + b for a, b in zip(lens, news)], 1, hd, 16)
    for s in range(3):
        for b in ref.table[s][s % 2::2]:
            ref.k[b], ref.ks[b] = rng.choice(np.array([0, 128], np.uint8), ref.k[b].shape), 2.0 ** O.E_MIN
    gpu.k.copy_(torch.from_numpy(ref.k))
    gpu.k_scale.copy_(torch.from_numpy(ref.ks.astype(np.float32)))
    ref.length[:] = lens
    gpu.length.copy_(torch.tensor(lens, dtype=torch.int32))
    st = starts(news)
    q, q64 = rows_of(rng, int(st[-1]), G, hd, dtype, gain=gain)
    out, lse, probs = check_attention(gpu, ref, q, q64, st, news, dtype, scale=scale)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    before = gpu.weight.clone()
    gpu.accumulate(q, lse, start=dev(st), max_new=max(news), scale=scale)
    assert abs(float((gpu.weight - before).double().sum()) - G * sum(news)) <= 1e-3 * G * sum(news)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,n", [(64, 1, 1), (64, 2, 6), (64, 1, 30), (64, 1, 100), (128, 1, 60), (32, 3, 40)])
def test_attention_value_scales_at_both_ends(hd, G, n, dtype):
    """The whole weight on a block of zero values (the smallest scale), beside values of 2^27 and more: zeros, not
    0 times infinity."""
    gpu, ref, rng = make(24, [100 + n], 1, hd, 16)
    gpu.length.fill_(100)
    b0, st = int(ref.table[0, 0]), dev(starts([n]))
    gpu.v[b0], gpu.v_scale[b0] = 0, 2.0 ** O.E_MIN
    others = torch.from_numpy(ref.table[0, 1:].astype(np.int64)).cuda()
    gpu.v_scale[others] = 2.0 ** 27
    gpu.k.zero_()
    gpu.k[b0, :, 3, 0] = 0x38  # 1.0 at slot 3
    gpu.k_scale.fill_(1.0)
    q = torch.zeros(n, G, hd, device="cuda", dtype=DT[dtype])
    out, lse = torch.ones_like(q), torch.zeros(n, G, device="cuda")
    q[:, :, 0] = 200.0
    gpu.attention(q, out, start=st, max_new=n, lse=lse, scale=1.0)
    assert (out == 0).all() and float((lse - 200.0).abs().max()) <= 200.0 * 2.0 ** -20


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hd,G,n", [(64, 1, 1), (64, 2, 6), (64, 1, 30), (64, 1, 100), (128, 1, 60), (32, 3, 40)])
def test_queries_at_the_end_of_the_range(hd, G, n, dtype):
    """Queries as large as their type has: the slot with the largest score takes the whole weight."""
    gpu, ref, rng = make(26, [100 + n], 1, hd, 16)
    gpu.length.fill_(100)
    b0, st = int(ref.table[0, 0]), dev(starts([n]))
    gpu.k.zero_()
    gpu.k[b0, :, 3, 0] = 0x38  # 1.0 at slot 3
    gpu.k_scale.fill_(1.0)
    want = torch.from_numpy(ref.values(0, 4, "v")[0][3, 0]).cuda().to(DT[dtype])
    q = torch.zeros(n, G, hd, device="cuda", dtype=DT[dtype])
    out, lse = torch.ones_like(q), torch.zeros(n, G, device="cuda")
    for first in (2.0 ** 112, 2.0 ** 118, 2.0 ** 127):
        q[:, :, 0] = first
        q[:, :, 1] = -first / 2
        gpu.attention(q, out, start=st, max_new=n, lse=lse, scale=0.25)
        assert torch.equal(out, want.expand_as(out)), first
        assert ((lse.double() - first / 4).abs() <= 2.0 ** -20 * first / 4).all()


@pytest.mark.parametrize("max_len", [0, 1])
@pytest.mark.parametrize("z", [6.0, 12.0, 18.0])
@pytest.mark.parametrize("hd,P,G,n", [(64, 16, 1, 1), (64, 128, 3, 5), (128, 64, 4, 1), (128, 16, 4, 3), (32, 16, 2, 1),
                                      (64, 16, 1, 40), (64, 64, 3, 21), (32, 32, 2, 20), (64, 16, 1, 100), (32, 16, 1, 70),
                                      (128, 32, 1, 30), (128, 16, 5, 27)])
def test_a_heavy_slot_over_a_long_flat_tail_in_fp32(hd, P, G, n, z, max_len):
    """One slot z nats above 40,000 equal ones, whose weights, though small each, are together a part of the output: a
    rounding that depends on the largest weight would show with its full sum, since it is the same for all of them.

    |o - o64| <= (2 B + 4) 2^-21 V as in the other fp32 cases, with B = z sum |q k| = z: of a weight relative to itself,
    beside the sums: 32 steps in the tensor core, cut off at 2^-23 of their sum or less, and one addition, 2^-24, for every
    256 slots that one block (here all: max_len 1) has, of up to V each."""
    tail = 40000
    blocks = -(-(tail + 1 + n) // P)
    c = gb.KV8Cache.allocate(1, 1, hd, P, blocks)
    c.length.fill_(tail)
    vt = torch.from_numpy(O.encode(np.linspace(-1.0, 1.0, hd))).cuda()  # the tail's values and the heavy slot's: fixed codes
    vh = torch.flip(vt, (0,))
    c.v.copy_(vt.expand_as(c.v))
    c.v[0, :, 0] = vh
    c.k[0, 0, 0, 0] = 0x38  # 1.0 where the others have 0
    c.k_scale.fill_(1.0), c.v_scale.fill_(1.0)
    q = torch.zeros(n, G, hd, device="cuda")
    q[:, :, 0] = z + torch.linspace(0, 0.3, n * G, device="cuda").reshape(n, G)
    out, lse = torch.zeros_like(q), torch.zeros(n, G, device="cuda")
    c.attention(q, out, start=dev(starts([n])), max_new=n, lse=lse, scale=1.0, max_len=max_len)
    z64 = q[:, :, 0].double()
    e = torch.exp(-z64) * (tail + torch.arange(n, device="cuda", dtype=torch.float64))[:, None]  # the visible tail
    h64, t64 = (torch.from_numpy(O.decode(x.cpu().numpy())).cuda() for x in (vh, vt))
    want = (h64 + e[..., None] * t64) / (1 + e[..., None])
    B = z + 0.3
    tol = (2 * B + 4) * 2.0 ** -21 + 32 * 2.0 ** -23 + (tail // 256) * 2.0 ** -24
    err = float((out.double() - want).abs().max())
    assert err <= tol, (err, tol)
    assert float((lse.double() - (z64 + torch.log1p(e))).abs().max()) <= B * 2.0 ** -21 + 2.0 ** -20 + 2.0 ** -23 * (B + 11)


def test_advance_by_offsets_alone():
    """Rows of different numbers, without the number of all rows: the lengths grow by the offsets' differences, as the
    other calls take them."""
    gpu, _, _ = make(25, [40, 40, 40], 1, 32, 16, extra=64)
    gpu.length.copy_(torch.tensor([5, 0, 7], dtype=torch.int32))
    gpu.advance(start=dev(starts([30, 0, 12])), max_new=30)
    assert gpu.length.tolist() == [35, 0, 19] and int(gpu.flags) == 0
    gpu.advance(start=dev(starts([1, 1, 1])))
    assert gpu.length.tolist() == [36, 1, 20] and int(gpu.flags) == 0
    gpu.advance(start=dev(starts([2, 1, 1])))  # more than max_new
    assert gpu.length.tolist() == [36, 2, 21] and int(gpu.flags) == gb.FLAG_ROW_RANGE


@pytest.mark.parametrize("max_len", [0, 1])
@pytest.mark.parametrize("z", [6.0, 12.0])
@pytest.mark.parametrize("hd,P,G,n", [(64, 16, 1, 1), (128, 64, 4, 1), (32, 16, 2, 5), (64, 16, 1, 40), (32, 32, 2, 20),
                                      (64, 16, 1, 100), (128, 16, 5, 27)])
def test_the_sum_of_weights_over_a_long_flat_tail_in_bf16(hd, P, G, n, z, max_len):
    """The log-sum-exp of bf16 rows is an fp32 output, and the accumulated weights go by it: one slot z nats above 40,000
    equal ones, whose weights all round alike when they are added.  |lse - lse64| <= B 2^-21 + 2^-20 + 2^-23 |lse| with
    B = z, |o - o64| <= 2^-10 V + 2^-8 |o64|, as in the other cases."""
    tail = 40000
    blocks = -(-(tail + 1 + n) // P)
    c = gb.KV8Cache.allocate(1, 1, hd, P, blocks)
    c.length.fill_(tail)
    c.v.fill_(0x38)  # 1.0 everywhere but for the heavy slot's 0
    c.v[0, :, 0] = 0
    c.k[0, 0, 0, 0] = 0x38
    c.k_scale.fill_(1.0), c.v_scale.fill_(1.0)
    q = torch.zeros(n, G, hd, device="cuda", dtype=torch.bfloat16)
    q[:, :, 0] = z
    out, lse = torch.zeros_like(q), torch.zeros(n, G, device="cuda")
    c.attention(q, out, start=dev(starts([n])), max_new=n, lse=lse, scale=1.0, max_len=max_len)
    e = np.exp(-z) * (tail + torch.arange(n, device="cuda", dtype=torch.float64))[:, None]
    err = float((lse.double() - (z + torch.log1p(e))).abs().max())
    assert err <= z * 2.0 ** -21 + 2.0 ** -20 + 2.0 ** -23 * (z + 5), err
    want = (e / (1 + e))[..., None]
    assert ((out.double() - want).abs() <= 2.0 ** -10 + 2.0 ** -8 * want).all()
