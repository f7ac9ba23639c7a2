"""gpt_sample_rows (per-row temperature, top-k, top-p, min-p) against the float64 oracle (oracle/sampling.py).

The kernel holds probabilities to about 2^-34 relative, so a token differs from
the oracle's only where the uniform falls within about 2^-33 of a border; the
seeds below were not chosen, and at some ten thousand draws over up to 2^17
borders each a difference is not expected (10^4 * 2^-33 * the number of tokens
that carry the mass, below 10^3).  log-probabilities: fp32 rounding, 2^-24
relative, beside 2^-32 absolute."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

from gpt_decoder_lm_b200 import binding as gb  # noqa: E402
from oracle import sampling as S  # noqa: E402

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def draw(z, par, u, V=None, logp=True):
    dev = {n: torch.from_numpy(np.ascontiguousarray(a)).cuda() for n, a in par.items()}
    rows = z.shape[0]
    out = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((rows,), 7.0, device="cuda") if logp else None
    gb.sample_rows(z, torch.from_numpy(u).cuda(), out, logp=lp, V=V, **dev)
    return out.cpu().numpy(), None if lp is None else lp.cpu().numpy()


def check(z, par, u, V=None):
    got, lp = draw(z, par, u, V)
    z64 = z.double().cpu().numpy()[:, :V]
    for r in range(z.shape[0]):
        v = {n: float(a[r]) for n, a in par.items()}
        tok, ref = S.sample_row_minp(z64[r], v.get("temperature", 1.0), int(v.get("top_k", 0)), v.get("top_p", 1.0),
                                     v.get("min_p", 0.0), float(u[r]))
        assert got[r] == tok, (r, v, got[r], tok)
        assert lp[r] == ref or abs(lp[r] - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -32, (r, v, lp[r], ref)


def params(rng, rows):
    kind = rng.integers(0, 7, rows)
    return {"temperature": np.where(kind == 0, rng.choice([0.0, -1.0, np.nan], rows),
                                    rng.choice([0.3, 0.8, 1.0, 1.7], rows)).astype(np.float32),
            "top_k": np.where(kind % 2 == 1, rng.choice([1, 2, 5, 40, 200, 5000, 10 ** 9], rows), 0).astype(np.int32),
            "top_p": np.where(kind >= 3, rng.choice([0.0, 0.1, 0.5, 0.9, 0.999, -1.0], rows), 1.0).astype(np.float32),
            "min_p": np.where((kind == 2) | (kind == 5), rng.choice([0.001, 0.05, 0.5, 1.0, 3.0], rows), 0).astype(np.float32)}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,V,ld", [(1, 50257, 50304), (3, 1, 1), (40, 65, 65), (20, 1000, 1003), (19, 50257, 50257),
                                       (150, 4097, 4160), (300, 513, 520), (2, 130001, 130001), (80, 130001, 130001)])
def test_mixed_rows(rows, V, ld, dtype):
    rng = np.random.default_rng(V + rows)
    z = torch.from_numpy((rng.standard_normal((rows, ld)) * 2.5).astype(np.float32)).to(DT[dtype]).cuda()
    check(z, params(rng, rows), rng.random(rows).astype(np.float32), V)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["flat", "equal", "grid", "peaked", "wide", "tiny"])
def test_shapes_of_rows(kind, dtype):
    """Nearly uniform rows, rows of one value, few values with many ties, one token with all the mass, logits spread
    over thousands, and logits that differ by less than fp32's epsilon times their size."""
    rng = np.random.default_rng(len(kind))
    rows, V = 24, 20011
    z = {"flat": rng.standard_normal((rows, V)) * 1e-3, "equal": np.full((rows, V), 3.25),
         "grid": rng.integers(0, 5, (rows, V)).astype(float), "peaked": np.where(rng.random((rows, V)) < 1e-4, 60.0, 0.0),
         "wide": rng.standard_normal((rows, V)) * 3000, "tiny": rng.standard_normal((rows, V)) * 1e-30}[kind]
    check(torch.from_numpy(z.astype(np.float32)).to(DT[dtype]).cuda(), params(rng, rows), rng.random(rows).astype(np.float32))


@pytest.mark.parametrize("dtype,rows,V,ld,sigma", [
    ("fp32", 2, 50257, 50257, 0.02), ("fp32", 160, 30011, 30011, 0.02), ("bf16", 3, 90001, 90001, 0.05),
    ("fp32", 2, 400003, 400003, 2.0), ("fp32", 1, 524288, 524288, 0.01), ("bf16", 2, 524287, 524288, 3.0)])
def test_crowded_borders_and_long_rows(dtype, rows, V, ld, sigma):
    """Rows whose border lies among thousands of nearly equal tokens, over one block and over clusters, and rows that
    do not fit in the blocks' memory; the second row starts at an odd offset."""
    rng = np.random.default_rng(V + rows)
    z = torch.from_numpy((rng.standard_normal((rows, ld)) * sigma).astype(np.float32)).to(DT[dtype]).cuda()
    par = {"temperature": rng.choice([0.7, 1.0], rows).astype(np.float32),
           "top_k": np.where(np.arange(rows) % 3 == 1, V // 3, 0).astype(np.int32),
           "top_p": np.where(np.arange(rows) % 3 != 1, rng.choice([0.5, 0.9, 0.9999], rows), 1.0).astype(np.float32),
           "min_p": np.zeros(rows, np.float32)}
    check(z, par, rng.random(rows).astype(np.float32), V)


def test_infinities_nan_and_empty_rows():
    rng = np.random.default_rng(3)
    V = 700
    z = rng.standard_normal((10, V)).astype(np.float32)
    z[0] = -np.inf
    z[1] = np.nan
    z[2, ::2] = -np.inf
    z[3, 5:] = np.nan
    z[4, [7, 300]] = np.inf
    z[5] = -np.inf
    z[5, 600] = -3e38
    z[6] = np.float32(-3.4e38)
    z[7, 9] = np.inf
    z[8, 100:] = -np.inf
    z[9] = np.where(np.arange(V) % 2 == 0, 0.0, -0.0)
    for t, k, p, m in ((0.7, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0), (1.3, 50, 0.9, 0.01), (1.0, 699, 0.0, 0.0),
                       (np.inf, 0, 1.0, 0.0)):
        par = {"temperature": np.full(10, t, np.float32), "top_k": np.full(10, k, np.int32),
               "top_p": np.full(10, p, np.float32), "min_p": np.full(10, m, np.float32)}
        if t == np.inf:  # uniform over what can be drawn
            got, _ = draw(torch.from_numpy(z).cuda(), par, np.full(10, 0.5, np.float32))
            for r in range(2, 10):
                fin = np.flatnonzero(np.isposinf(z[r]) if np.isposinf(z[r]).any() else np.isfinite(z[r]))
                assert got[r] == fin[int(0.5 * len(fin))], r
            continue
        check(torch.from_numpy(z).cuda(), par, rng.random(10).astype(np.float32))


def test_uniforms_at_the_ends_and_defaults():
    rng = np.random.default_rng(4)
    z = torch.from_numpy(rng.standard_normal((6, 3001)).astype(np.float32)).cuda()
    u = np.array([0.0, np.float32(1 - 2.0 ** -24), 0.5, 1.0, -1.0, np.nan], np.float32)
    got, _ = draw(z, {}, u)
    assert got[0] == 0 and got[1] == 3000 and got[3] == 3000 and got[4] == 0 and got[5] == 0
    got2, _ = draw(z, {"temperature": np.ones(6, np.float32), "top_k": np.zeros(6, np.int32)}, u, logp=False)
    assert np.array_equal(got, got2)


def test_agrees_with_gpt_sample_where_both_apply():
    rng = np.random.default_rng(5)
    z = torch.from_numpy((rng.standard_normal((64, 5003)) * 3).astype(np.float32)).cuda()
    u = rng.random(64).astype(np.float32)
    out = torch.zeros(64, dtype=torch.int32, device="cuda")
    gb.sample(z, 0.8, 40, 0.9, torch.from_numpy(u).cuda(), out)
    got, _ = draw(z, {"temperature": np.full(64, 0.8, np.float32), "top_k": np.full(64, 40, np.int32),
                      "top_p": np.full(64, 0.9, np.float32)}, u)
    assert (got == out.cpu().numpy()).sum() >= 63  # gpt_sample's probabilities are fp32


def test_frequencies_follow_the_kept_probabilities():
    V, rows = 64, 8192
    rng = np.random.default_rng(6)
    z = (rng.standard_normal(V) * 2).astype(np.float32)
    u = ((np.arange(rows) + 0.5) / rows).astype(np.float32)
    f = lambda v, t=np.float32: np.full(rows, v, t)  # noqa: E731
    got, lp = draw(torch.from_numpy(np.tile(z, (rows, 1))).cuda(),
                   {"temperature": f(0.8), "top_k": f(20, np.int32), "top_p": f(0.95), "min_p": f(0.02)}, u)
    count = np.bincount(got, minlength=V) / rows
    for t in np.unique(got):
        assert abs(count[t] - np.exp(lp[got == t][0])) <= 1.0 / rows + 1e-6


def test_captured_and_on_another_stream():
    rng = np.random.default_rng(7)
    z = torch.from_numpy(rng.standard_normal((5, 9001)).astype(np.float32)).cuda()
    u = torch.from_numpy(rng.random(5).astype(np.float32)).cuda()
    out, lp = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.zeros(5, device="cuda")
    tp = torch.full((5,), 0.9, device="cuda")
    gb.sample_rows(z, u, out, top_p=tp, logp=lp)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb.sample_rows(z, u, out, top_p=tp, logp=lp)
    for _ in range(3):
        z.normal_()
        g.replay()
        torch.cuda.synchronize()
        want = out.clone(), lp.clone()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            gb.sample_rows(z, u, out, top_p=tp, logp=lp)
        s.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lp, want[1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("V", [700, 3001, 20011])
def test_temperatures_at_which_the_whole_range_of_logits_counts(V, dtype):
    """Logits as far apart as the type allows (their distance is beyond fp32), at temperatures, infinity among them,
    where all of them or most have weight, under each filter."""
    rng = np.random.default_rng(V)
    rows = 12
    z = (rng.uniform(-1, 1, (rows, V)) * 3.38e38).astype(np.float32)
    z[:, 0], z[:, V // 2] = 3.38e38, -3.38e38
    z[1, 5], z[2, 7:20], z[3, 9] = np.inf, -np.inf, np.nan
    z = torch.from_numpy(z).to(DT[dtype]).cuda()
    for t in (1e36, 1.1e37, 1e38, 3.4e38, np.inf):
        for k, p, m in ((0, 1.0, 0.0), (40, 1.0, 0.0), (V // 2, 0.9, 0.0), (0, 0.5, 0.0), (0, 0.97, 0.2), (0, 1.0, 0.4)):
            par = {"temperature": np.full(rows, t, np.float32), "top_k": np.full(rows, k, np.int32),
                   "top_p": np.full(rows, p, np.float32), "min_p": np.full(rows, m, np.float32)}
            check(z, par, rng.random(rows).astype(np.float32))


def test_the_smallest_temperatures():
    """Temperatures below 2^-122 count as 2^-122, for logits so close that it matters; for others the largest is drawn."""
    rng = np.random.default_rng(11)
    rows, V = 16, 3001
    z = (rng.uniform(-1, 1, (rows, V)) * 2.0 ** -121).astype(np.float32)
    z[8:] = rng.standard_normal((8, V))
    u, floor = rng.random(rows).astype(np.float32), np.float32(2.0 ** -122)
    for t in (2.0 ** -122, 1e-37, 1e-38, 1e-45):
        for k, p, m in ((0, 1.0, 0.0), (40, 1.0, 0.0), (0, 0.5, 0.0), (V // 2, 0.9, 0.1)):
            par = {"temperature": np.full(rows, t, np.float32), "top_k": np.full(rows, k, np.int32),
                   "top_p": np.full(rows, p, np.float32), "min_p": np.full(rows, m, np.float32)}
            got, lp = draw(torch.from_numpy(z).cuda(), par, u)
            for r in range(rows):
                tok, ref = S.sample_row_minp(z[r].astype(np.float64), float(floor), k, float(par["top_p"][r]),
                                             float(par["min_p"][r]), float(u[r]))
                assert got[r] == tok, (t, k, p, m, r)
                assert abs(lp[r] - ref) <= 2.0 ** -24 * abs(ref) + 2.0 ** -32
