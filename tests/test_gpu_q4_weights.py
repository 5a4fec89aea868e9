"""Precision of the decode steps over the 4-bit cache where positions differ in
size by many orders: a value, however large, counts by its weight alone, and
what it leaves of the other positions' precision is bound by its weight too.

Tolerance, from the arithmetic, for one query head and group of 32 values, with
P_j the normalised weights (sum 1), S_j = 15 step_j of V's group, n keys:
  - a score, in natural units, is off by at most delta_j: with A_j the sum of
    |q_i| (|lo| + 15 step) / sqrt(d) over a key's values, 24 fp32 roundings of
    partial sums within A_j; fp32 queries keep 22 bits of the head's largest
    (two integer terms), bf16 ones are exact but their products with the codes
    may be truncated at 2^-12 of the largest with one code unit, twice a group;
    the bias and the difference from the maximum, two roundings each; ex2 is
    within 2^-21.  A weight off by delta_j moves o by P_j delta_j |v_j - o|;
  - the weights' sum and the numerator are sums of at most 2 n / 16 + 24
    terms one after the other: 2^-23 each of sum P_j (|lo_j| + S_j);
  - P step is rounded to f16 (2^-11 of itself) or two terms of it (2^-22), but
    no finer than f16's 2^-25 where the largest of a column is kept at 2^8 or
    more (fp32: 2^11): 2^-33 (2^-36) of the largest P_j S_j, for each of n keys;
    (bf16: sums over a tile may be truncated, 2^-14 of the largest P step: well
    inside the first where it is counted once more;)
  - the output's rounding: 2^-24 or 2^-8 of |o|.
"""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def tight(q, K, V, log_w, dtype):
    """o [Hq, d] and the bound of |got - o|; q [Hq, d], K, V [H, n, d] fp64
    values of the cache, log_w [Hq, n]."""
    Hq, d = q.shape
    G, n = Hq // K.shape[0], K.shape[1]
    o, tol = np.zeros((Hq, d)), np.zeros((Hq, d))
    wide = lambda g: np.repeat(g, 32, -1)  # noqa: E731
    for h in range(Hq):
        see = log_w[h] > -np.inf
        if not see.any():
            continue
        k, v, lw = K[h // G][see], V[h // G][see], log_w[h][see]
        x = k @ q[h] / np.sqrt(d) + lw
        p = np.exp(x - x.max())
        P = (p / p.sum())[:, None]
        o[h] = (P * v).sum(0)
        g = lambda t: t.reshape(len(t), -1, 32)  # noqa: E731
        # a group's lo and 15 step are not known here, but its smallest value
        # and its span, which is 14 steps or more of its 15 (or none)
        klo, kspan = np.abs(g(k)).max(-1), (g(k).max(-1) - g(k).min(-1)) * 15 / 14
        vlo, S = wide(np.abs(g(v)).max(-1)), wide((g(v).max(-1) - g(v).min(-1)) * 15 / 14)
        size = np.abs(q[h])
        A = (size * (wide(klo) + wide(kspan))).sum(-1) / np.sqrt(d)
        delta = 24 * 2.0 ** -24 * A + 2 * 2.0 ** -23 * (np.abs(lw) + np.abs(x - x.max()) + np.abs(x).max()) \
            + 2.0 ** -21
        if dtype == "f32":
            delta = delta + 2.0 ** -22 * size.max() * wide(kspan).sum(-1) / np.sqrt(d)
        else:
            delta = delta + 2 * 2.0 ** -12 * size.max() * (kspan / 15).sum(-1) / np.sqrt(d)
        terms = 2 * n / 16 + 24
        tol[h] = (P * delta[:, None] * np.abs(v - o[h])).sum(0) \
            + 2 * terms * 2.0 ** -23 * (P * (vlo + S)).sum(0) \
            + (2.0 ** -10 if dtype == "bf16" else 2.0 ** -22) * (P * S).sum(0) \
            + n * 2.0 ** (-33 if dtype == "bf16" else -36) * (P * S).max(0) \
            + np.abs(o[h]) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)
    return o, tol


class Rows:
    """One sequence's rows k, v [H, n, d] (fp32, host) in a cache of their own."""

    def __init__(self, k, v, page):
        H, n, d = k.shape
        self.page, self.d, self.n = page, d, n
        per = -(-n // page)
        self.table = np.arange(per, dtype=np.int32)[None, ::-1].copy()
        self.cache = plsh.Q4Cache.empty(per, H, d, torch.from_numpy(self.table).cuda(), page)
        dev = lambda x: torch.from_numpy(np.ascontiguousarray(x[None], dtype=np.float32)).cuda()  # noqa: E731
        plsh.q4_cache_write(self.cache, dev(k), dev(v), i32([0]))
        data = self.cache.data.cpu().numpy().reshape(per, H, -1, 20 * d)
        self.K, self.V = q4.read_sequence(data, self.table[0], page, d, n)

    def check(self, got, q, log_w, dtype):
        got = got[0, :, 0].double().cpu().numpy()
        o, tol = tight(q[0, :, 0].double().cpu().numpy(), self.K, self.V, log_w, dtype)
        off = np.abs(got - o)
        assert (off <= tol).all(), f"off by {(off / np.maximum(tol, 1e-300)).max():.3g} tolerances"


def draw(seed, H, n, d):
    rng = np.random.default_rng(seed)
    return rng, rng.standard_normal((H, n, d)) + 0.3, rng.standard_normal((H, n, d)) + 0.3


@pytest.mark.parametrize("factor", [1e3, 1e6, 1e8, 1e20])
@pytest.mark.parametrize("heads,d,page", [(4, 128, 64), (8, 128, 32), (2, 64, 16), (12, 64, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_large_value_that_only_another_head_sees(dtype, heads, d, page, factor):
    """Head 0 sees a key whose V is larger by a factor; its group mates see the
    keys behind it in the same tile, or those and others, but not that one."""
    n, pos, big = 250, 239, 226
    rng, k, v = draw(heads, 1, n, d)
    v[:, big] *= factor
    rows = Rows(k, v, page)
    starts = [np.array([0, n])] + [np.array([0, s, n]) for s in (228, 227, 236, 239)]
    starts = [starts[0] if h == 0 else starts[1 + h % 4] for h in range(heads)]
    bins = plsh.bins_from_host(n, heads, 1, np.concatenate([[0], np.cumsum([len(x) for x in starts])]),
                               np.concatenate(starts))
    # (queries so small that the weights are nearly the counts: what is left is
    # P V's precision)
    q = torch.from_numpy(rng.standard_normal((1, heads, 1, d)) * 1e-3).cuda().to(DT[dtype])
    got = plsh.alibi_decode_q4(q, rows.cache, bins, i32([pos]))
    plsh.stream_status()
    j = np.arange(n)
    first = np.array([0 if h == 0 else starts[h][1] for h in range(heads)])
    log_w = np.where((j >= first[:, None]) & (j <= pos), 0.0, -np.inf)
    rows.check(got, q, log_w, dtype)
    bins.free()


def _away(q, score, d):
    """A key whose score with q is `score`."""
    return q * (score * np.sqrt(d) / (q @ q))


@pytest.mark.parametrize("factor", [1.0, 1e4, 1e8, 1e20])
@pytest.mark.parametrize("score", [-90.0, -60.0, -18.0, 0.0, 40.0])
@pytest.mark.parametrize("heads,d", [(4, 128), (8, 64), (1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("exact", [True, False])
def test_a_large_value_counts_by_its_weight(exact, dtype, heads, d, score, factor):
    """A recent key whose V is larger by a factor, with scores from far below
    to far above the others', whose own scores step up by 30 half way back: it
    may outweigh what comes before it and be outweighed by what comes after."""
    n, pos, big = 420, 411, 405
    rng, k, v = draw(heads + d, 1, n, d)
    one = rng.standard_normal(d)
    q = torch.from_numpy(np.stack([one * (1 + 0.01 * h) for h in range(heads)])[None, :, None]) \
        .cuda().to(DT[dtype])
    base = q[0, 0, 0].double().cpu().numpy()
    k *= 0.02
    k[:, :300] += _away(base, 30.0, d)
    k[:, big] = _away(base, score, d)
    v[:, big] *= factor
    rows = Rows(k, v, 64)
    j = np.arange(n)
    if exact:
        sigma = np.full(heads, 200.0)
        got = plsh.alibi_exact_decode_q4(q, rows.cache, sigma, i32([pos]))
        log_w = q4.log_weights_exact(sigma, pos, n)
    else:
        st = np.tile(np.array([0, 100, n, 0, 402, n, 0, 330, n]), heads)
        bins = plsh.bins_from_host(n, heads, 3, np.arange(0, 9 * heads + 1, 3), st)
        got = plsh.alibi_decode_q4(q, rows.cache, bins, i32([pos]))
        c = (j >= 100) * 1.0 + (j >= 402) + (j >= 330)
        with np.errstate(divide="ignore"):
            log_w = np.tile(np.log(np.where(j <= pos, c, 0.0)), (heads, 1))
        bins.free()
    plsh.stream_status()
    rows.check(got, q, log_w, dtype)


@pytest.mark.parametrize("factor", [1.0, 1e5, 1e9])
@pytest.mark.parametrize("heads,d", [(4, 128), (8, 128), (2, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_values_in_long_rows_of_one_block(dtype, heads, d, factor):
    """A thousand sequences of the same pages: each row is one block's, several
    tiles a warp, with a large V of no weight among the newest, one that fades
    as older keys score more, and one among the oldest."""
    B, n = 1000, 900
    rng, k, v = draw(heads * d, 1, n, d)
    one = rng.standard_normal(d)
    q = torch.from_numpy(np.stack([one * (1 + 0.01 * h) for h in range(heads)])[None, :, None]) \
        .cuda().to(DT[dtype])
    base = q[0, 0, 0].double().cpu().numpy()
    k *= 0.02
    for at, score in ((slice(0, 600), 25.0), (slice(895, 896), -60.0), (slice(890, 891), 12.0), (slice(3, 4), -30.0)):
        k[:, at] = 0.02 * rng.standard_normal(k[:, at].shape) + _away(base, score, d)
    v[:, [3, 890, 895]] *= factor
    rows = Rows(k, v, 64)
    cache = plsh.Q4Cache(rows.cache.data, rows.cache.table.expand(B, -1).contiguous(), 1, d, 64)
    sigma = np.full(heads, 400.0)
    got = plsh.alibi_exact_decode_q4(q.expand(B, -1, -1, -1).contiguous(), cache, sigma, i32([n - 1] * B))
    plsh.stream_status()
    for b in (0, 1, 499, 998, 999):
        rows.check(got[b:b + 1], q, q4.log_weights_exact(sigma, n - 1, n), dtype)


@pytest.mark.parametrize("d,heads", [(128, 4), (128, 8), (64, 3)])
@pytest.mark.parametrize("exact", [True, False])
def test_fp32_steps_keep_fp32(exact, d, heads):
    """Small queries: the scores' errors vanish and P V's precision shows (a
    single f16 term, or sums of subnormal products, would be off by many times the
    tolerance)."""
    n, pos = 130, 121
    rng, k, v = draw(7 * d + heads, 1, n, d)
    rows = Rows(k, v, 32)
    q = torch.from_numpy((rng.standard_normal((1, heads, 1, d)) * 1e-4).astype(np.float32)).cuda()
    if exact:
        sigma = np.linspace(20.0, 90.0, heads)
        got = plsh.alibi_exact_decode_q4(q, rows.cache, sigma, i32([pos]))
        log_w = q4.log_weights_exact(sigma, pos, n)
    else:
        bins = plsh.sample_bins(n, np.linspace(20.0, 90.0, heads), 9, seed=3)
        off, st = bins.to_host()
        got = plsh.alibi_decode_q4(q, rows.cache, bins, i32([pos]))
        log_w = q4.log_weights_approx(off, st, heads, 9, pos, n)
        bins.free()
    plsh.stream_status()
    rows.check(got, q, log_w, "f32")
