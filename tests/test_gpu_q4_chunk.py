"""Exact ALiBi attention of several new tokens a sequence over the 4-bit cache,
and of a batch behind a shared prefix, against the fp64 oracle on the values the
cache holds.

Tolerance: that of the decode step's tests (derived there), and for bf16, where
many rows of a KV head go to the tensor cores with values rounded to f16 (2^-11 of
themselves at most, half a step of 11 bits; the largest of 32 positions' lies in
[2^14, 2^15), so f16's smallest step, 2^-24, is 2^-38 of it):
  - K: every product of a score is off by 2^-11 of itself: the score by 2^-11 A at
    most, with A as there without the bias; o by twice that times R.  Where keys of
    32 positions differ by more than 2^29 the small ones lose more, 2^-38 of the
    largest: the bound leaves 2^-7 d of 2^-11 A for it;
  - P and V: 2^-11 each of a convex combination of values within R: 2^-10 R.
These are bounds of the worst signs.  Roundings of independent sign leave much
less, and the whole output is held to that: its relative 2-norm error is below
2.5e-3 in bf16 (the output's own rounding: at most 2^-8 / sqrt(3) = 2.26e-3 for
uniform errors of half a step, 1.7e-3 for mixed significands; K's, P's and V's,
2^-11 / sqrt(3) each at most, add 1e-4 to that in quadrature) and 2e-6 in fp32.
"""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4
from positional_lsh_approximation_gb300.inputs import alibi_sigmas
from test_gpu_q4_decode import DT, Setup, i32, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def bound(q, K, V, o, dtype, G):
    tol = tolerance(q, K, V, o, dtype, G)
    if dtype == "f32":
        return tol
    d = K.shape[2]
    A = np.abs(q).max(-1) * np.repeat(np.abs(K).sum(-1).max(-1), G) / np.sqrt(d)
    R = np.repeat(np.abs(V).max((1, 2)), G)
    return tol + (R * (2 * 2.0 ** -11 * (1 + d * 2.0 ** -7) * A + 2.0 ** -10))[:, None]


class Rows(Setup):
    def __init__(self, B, Hq, H, d, page, n, dtype, m, wide=True, **kw):
        super().__init__(B, Hq, H, d, page, n, dtype, **kw)
        g = torch.Generator("cuda").manual_seed(99)
        self.m = m
        self.q = torch.randn(B, Hq, m, d, device="cuda", generator=g).to(DT[dtype])
        G = Hq // H
        passes = m * -(-G // 8) if G > 4 else -(-m // (8 // G))
        if wide and dtype == "bf16" and passes >= 6:
            # a table long enough for the tensor cores to be taken (its pages again and again)
            per = self.table.shape[1]
            long = max(per, -(-2 ** 19 // (B * H * passes * page)))
            self.table = np.tile(self.table, (1, -(-long // per)))[:, :long].copy()
            self.cache = plsh.Q4Cache(self.cache.data, torch.from_numpy(self.table).cuda(), H, d, page)

    def want(self, b, p, i, sigma, drop=None):
        data = self.host()
        K, V = q4.read_sequence(data, self.table[b], self.page, self.d, p + 1)
        w = q4.log_weights_exact(sigma, p, p + 1)
        if drop is not None:
            w[:, drop] = -np.inf
        q = self.q[b, :, i].double().cpu().numpy()
        return q4.decode_row(q, K, V, w), K, V, q

    def check_rows(self, got, pos, lens, sigma, rows=None, norm=True):
        got = got.double().cpu().numpy()
        data = self.host()
        err = size = 0.0
        for b in range(self.B):
            count = self.m if lens is None else min(max(lens[b], 0), self.m)
            if pos[b] < 0:
                assert (got[b, :, :count] == 0).all()
                continue
            if count == 0:
                continue
            K, V = q4.read_sequence(data, self.table[b], self.page, self.d, pos[b] + count)
            for i in range(count) if rows is None else [x for x in rows if x < count]:
                p = pos[b] + i
                q = self.q[b, :, i].double().cpu().numpy()
                want = q4.decode_row(q, K[:, :p + 1], V[:, :p + 1], q4.log_weights_exact(sigma, p, p + 1))
                tol = bound(q, K[:, :p + 1], V[:, :p + 1], want, self.dtype, self.Hq // self.H)
                off = np.abs(got[b, :, i] - want)
                assert (off <= tol).all(), f"sequence {b}, row {i}: off by {(off / tol).max():.2f} tolerances"
                err += ((got[b, :, i] - want) ** 2).sum()
                size += (want ** 2).sum()
        if norm and size:
            assert np.sqrt(err / size) < (2.5e-3 if self.dtype == "bf16" else 2e-6), np.sqrt(err / size)


CASES = [
    # B, Hq, H, d, page, n, dtype, m, first positions, lens
    (1, 1, 1, 128, 16, 1, "bf16", 1, [0], None),
    (1, 4, 1, 128, 64, 64, "bf16", 64, [0], None),                     # a whole prompt
    (1, 8, 2, 128, 64, 300, "bf16", 37, [263], None),
    (2, 8, 2, 64, 32, 530, "bf16", 40, [490, 17], [40, 23]),
    (1, 1, 1, 128, 16, 400, "bf16", 333, [67], None),                  # more rows than a tile
    (3, 12, 1, 128, 64, 260, "bf16", 50, [210, -1, 0], [50, 20, 1]),   # an idle slot, twelve heads on one
    (2, 3, 1, 64, 16, 700, "bf16", 90, [610, 300], [0, 90]),           # nothing for the first
    (1, 20, 4, 128, 128, 1500, "bf16", 7, [1493], None),               # five heads on one: 35 rows
    (5, 17, 1, 64, 64, 333, "bf16", 20, [313, 5, 127, 128, 129], None),
    (1, 32, 8, 128, 256, 4100, "bf16", 100, [4000], None),             # rows of several CTAs
    (9, 4, 4, 128, 64, 200, "bf16", 40, [(37 * b) % 160 for b in range(9)], [5 * b for b in range(9)]),
    (1, 4, 2, 128, 16, 129, "bf16", 129, [0], None),
    (2, 2, 1, 64, 64, 5000, "bf16", 16, [4984, 2500], None),
    (2, 2, 1, 64, 64, 5000, "bf16", 32, [4968, 2500], [31, 32]),
    (9, 4, 4, 128, 64, 200, "bf16", 64, [(37 * b) % 130 for b in range(9)], [8 * b for b in range(9)]),
    (2, 2, 2, 64, 32, 90, "bf16", 5, [31, 80], [5, 4]),                # five rows a pass
    (2, 2, 2, 128, 32, 90, "f32", 9, [62, 1], None),                   # five and four
    (3, 6, 2, 128, 16, 130, "bf16", 7, [100, 0, 60], [6, 7, 1]),       # two rows of three heads, and one
    (4, 8, 2, 64, 64, 260, "f32", 3, [63, 254, -1, 7], [3, 3, 3, 0]),
    (3, 8, 2, 128, 64, 300, "bf16", 2, [298, -1, 30], [2, 2, 1]),      # few rows: not on the tensor cores
    (2, 3, 1, 64, 16, 150, "f32", 11, [139, 20], [11, 5]),
    (2, 8, 2, 128, 64, 700, "f32", 5, [600, 250], None),
    (1, 12, 1, 64, 16, 400, "f32", 40, [360], None),
]


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_chunk_matches_the_oracle(case, wide):
    *shape, pos, lens = case
    s = Rows(*shape, wide=wide, seed=shape[5])
    sigma = alibi_sigmas(s.Hq)
    out = torch.full_like(s.q, 7.0)
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos), None if lens is None else i32(lens), out=out)
    plsh.stream_status()
    assert got is out
    s.check_rows(got, pos, lens, sigma)
    for b in range(s.B):                             # rows behind the last: as they were
        assert (got[b, :, min(lens[b], s.m) if lens else s.m:] == 7).all()
    again = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos), None if lens is None else i32(lens))
    plsh.stream_status()
    for b in range(s.B):
        k = min(lens[b], s.m) if lens else s.m
        assert torch.equal(again[b, :, :k], got[b, :, :k]) and (again[b, :, k:] == 0).all()


@pytest.mark.parametrize("sigma", [0.05, 3.0, 1e6])
@pytest.mark.parametrize("d", [64, 128])
def test_steep_and_flat_slopes_and_scores_that_jump(sigma, d):
    s = Rows(2, 4, 2, d, 32, 900, "bf16", 28, seed=5)
    s.k[:, :, 100:140] *= 8                          # met late: the newest keys come first
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0, 0]))
    pos, sig = [872, 300], np.full(4, sigma)
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sig, i32(pos))
    plsh.stream_status()
    s.check_rows(got, pos, None, sig)


def test_a_chunk_is_what_its_tokens_are_one_by_one():
    s = Rows(3, 8, 2, 128, 64, 500, "bf16", 33, seed=6)
    sigma = alibi_sigmas(8)
    pos = [467, 100, 0]
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos)).double()
    err = size = 0.0
    for i in range(33):
        one = plsh.alibi_exact_decode_q4(s.q[:, :, i:i + 1].contiguous(), s.cache, sigma, i32(pos) + i).double()
        err += ((got[:, :, i:i + 1] - one) ** 2).sum().item()
        size += (one ** 2).sum().item()
    assert np.sqrt(err / size) < 2.5e-3 * np.sqrt(2)          # two roundings
    plsh.stream_status()


@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (5, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_was_never_written_has_no_effect(heads, d, dtype):
    Hq, H = heads
    s = Rows(2, Hq, H, d, 32, 200, dtype, 60, seed=21)
    pos, lens = [93, 129], [40, 33]
    sigma = alibi_sigmas(Hq)
    got = []
    for fill in (0, 255, 127):
        s.cache.data.fill_(fill)
        plsh.q4_cache_write(s.cache, s.k, s.v, i32([0, 0]), i32([133, 162]))
        got.append(plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos), i32(lens)))
        plsh.stream_status()
    assert torch.isfinite(got[0]).all()
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def poison(s, b, p, which, value=float("nan")):
    k, v = s.k[b:b + 1, :, p:p + 1].clone(), s.v[b:b + 1, :, p:p + 1].clone()
    (k if which == "k" else v)[..., 37] = value
    table = torch.from_numpy(s.table[b:b + 1].copy()).cuda()
    plsh.q4_cache_write(plsh.Q4Cache(s.cache.data, table, s.H, s.d, s.page), k, v, i32([p]))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("place", [50, 310, 330])
def test_nan_reaches_the_rows_that_see_it_and_no_other(which, dtype, place):
    s = Rows(2, 4, 1, 128, 64, 400, dtype, 40, seed=2)
    pos = [300, 360]
    sigma = np.full(4, 40.0)
    want = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos))
    poison(s, 0, place, which)
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos))
    plsh.stream_status()
    first = max(0, place - 300)                      # the first row that sees it
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, :, :first], want[0, :, :first])
    seen = torch.isnan(got[0, :, first:])
    if which == "k":
        assert seen.all()
    else:                                            # a value's group: 32 .. 63
        assert seen[..., 32:64].all() and not seen[..., :32].any() and not seen[..., 64:].any()
        keep = torch.cat([got[0, :, first:, :32], got[0, :, first:, 64:]], -1).double()
        ref = torch.cat([want[0, :, first:, :32], want[0, :, first:, 64:]], -1).double()
        assert ((keep - ref).norm() / ref.norm()).item() < 2.5e-3 * 2 ** 0.5


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_values(dtype):
    """Queries and keys far from unit scale, groups of V of very different sizes,
    positions of K that are much larger than others: each is held to its own."""
    s = Rows(2, 8, 2, 128, 64, 500, dtype, 20, seed=5)
    size = torch.tensor([1e4, 1.0, 1e-4, 1e-8], device="cuda").repeat_interleave(32)
    s.v = s.v * size
    s.k[:, :, 100:130] *= 3
    pos = [480, 60]
    for qs, ks in ((1e3, 1e-3), (1e-6, 1e6), (30.0, 1.0)):
        plsh.q4_cache_write(s.cache, s.k * ks, s.v, i32([0, 0]))
        s.q = torch.randn(2, 8, 20, 128, device="cuda").to(DT[dtype]) * qs
        sigma = alibi_sigmas(8)
        got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos)).double().cpu().numpy()
        plsh.stream_status()
        for b in range(2):
            for i in (0, 11, 19):
                want, K, V, q = s.want(b, pos[b] + i, i, sigma)
                for y in range(4):
                    sl = slice(32 * y, 32 * y + 32)
                    tol = bound(q, K, V[:, :, sl], want[:, sl], dtype, 4)
                    off = np.abs(got[b, :, i, sl] - want[:, sl])
                    assert (off <= tol).all(), f"group {y}: {(off / tol).max():.2f}"


@pytest.mark.parametrize("factor", [1.0, 1e4, 1e10])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_large_key_or_value_that_weighs_nothing(which, factor):
    """Of another step, or a key of the same one: the other keys lose nothing."""
    s = Rows(1, 4, 1, 128, 64, 600, "bf16", 32, seed=9)
    sigma, pos = np.full(4, 2.0), [560]
    x = s.k if which == "k" else s.v
    at = 300 if which == "v" else 520
    if which == "k":
        # away from every query: its score is far below the others'
        s.q = s.q.abs()
        x[:, :, at] = -x[:, :, at].abs()
    x[:, :, at] *= factor
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0]))
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos)).double().cpu().numpy()
    plsh.stream_status()
    err = size = 0.0
    for i in range(32):
        want, *_ = s.want(0, pos[0] + i, i, sigma)
        err += ((got[0, :, i] - want) ** 2).sum()
        size += (want ** 2).sum()
    assert np.sqrt(err / size) < 2.5e-3


def test_values_past_the_range_are_reported():
    """Of one piece (how many steps lie in one follows from the batch): reported, or
    the pieces' ranges hold them and the result is right."""
    s = Rows(1, 4, 1, 128, 64, 400, "bf16", 16, seed=9)
    s.v[:, :, 100] *= 1e25                           # against the newest step's
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0]))
    sigma = np.full(4, 50.0)
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([384]))
    try:
        plsh.stream_status()
        s.check_rows(got, [384], None, sigma)
    except plsh.PlshError as e:
        assert e.status == plsh.PLSH_ERR_RANGE
    s = Rows(300, 4, 1, 128, 64, 400, "bf16", 16, seed=9)      # a CTA has several steps of a sequence
    s.v[:, :, 100] *= 1e25
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * 300))
    plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([384] * 300))
    with pytest.raises(plsh.PlshError) as e:
        plsh.stream_status()
    assert e.value.status == plsh.PLSH_ERR_RANGE


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), 2.0 ** 111])
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(bad):
    s = Rows(1, 4, 1, 64, 16, 100, "bf16", 20, seed=2)
    sigma = alibi_sigmas(4)
    want = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([80]))
    s.q[0, 2, 9, 7] = bad
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([80]))
    assert torch.isnan(got[0, 2, 9]).all()
    rest = torch.ones(4, 20, dtype=torch.bool)
    rest[2, 9] = False
    assert torch.equal(got[0].cpu()[rest], want[0].cpu()[rest])


@pytest.mark.parametrize("dtype,m", [("bf16", 28), ("bf16", 3), ("bf16", 6), ("f32", 9)])
def test_places_out_of_range_are_reported(dtype, m):
    s = Rows(3, 4, 2, 128, 16, 64, dtype, m, seed=3)
    sigma = alibi_sigmas(4)

    def failed():
        with pytest.raises(plsh.PlshError) as err:
            plsh.stream_status()
        assert err.value.status == plsh.PLSH_ERR_INVALID
    cap = 16 * s.table.shape[1]
    good = [cap - m, 5, 0]
    want = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(good))
    plsh.stream_status()
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([cap - m + 2, 2 ** 31 - 1, 0]))
    failed()
    assert (got[0, :, m - 2:] == 0).all() and (got[0, :, :m - 2] != 0).any() and (got[1] == 0).all()
    assert torch.equal(got[2], want[2])
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([-1, -2 ** 31, 0]))
    plsh.stream_status()
    assert (got[:2] == 0).all() and torch.equal(got[2], want[2])
    # a bad page: its keys are absent (sequence 0's second page)
    for bad in (-1, s.cache.pages, -2 ** 31):
        s.cache.table[0, 1] = bad
        got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(good))
        failed()
        assert torch.equal(got[1:], want[1:])
        t = s.table.copy()
        s.table[0, 1] = 0
        o, K, V, q = s.want(0, good[0] + m - 1, m - 1, sigma, drop=slice(16, 32))
        s.table = t
        assert (np.abs(got[0, :, m - 1].double().cpu().numpy() - o) <= bound(q, K, V, o, dtype, 2)).all()
    s.cache.table[0] = -1
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(good))
    failed()
    assert (got[0] == 0).all() and torch.equal(got[1:], want[1:])
    # pages behind the last position are not read
    s.cache.table.copy_(torch.from_numpy(s.table))
    s.cache.table[1, (5 + m - 1) // 16 + 1:] = -5
    assert torch.equal(plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(good)), want)
    plsh.stream_status()


def test_streams_graphs_and_workspaces():
    a = Rows(2, 8, 2, 128, 64, 1000, "bf16", 30, seed=1)
    b = Rows(3, 8, 2, 64, 32, 700, "bf16", 50, seed=2)
    sig = alibi_sigmas(8)
    pa, pb, lb = i32([970, 400]), i32([650, 3, 200]), i32([50, 20, 0])
    wa = plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa)
    wb = plsh.alibi_exact_chunk_q4(b.q, b.cache, sig, pb, lb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        ga = plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa, stream=s1)
        gb = plsh.alibi_exact_chunk_q4(b.q, b.cache, sig, pb, lb, stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        ga = plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa)
    with torch.cuda.graph(g2):
        gb = plsh.alibi_exact_chunk_q4(b.q, b.cache, sig, pb, lb)
    for qa, qb, ql in (([970, 400], [650, 3, 200], [50, 20, 0]), ([17, -1], [100, 649, 0], [1, 50, 50])):
        pa.copy_(i32(qa))
        pb.copy_(i32(qb))
        lb.copy_(i32(ql))
        wa = plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa)
        wb = plsh.alibi_exact_chunk_q4(b.q, b.cache, sig, pb, lb)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s1):
                g1.replay()
            with torch.cuda.stream(s2):
                g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    # a workspace of the caller's, no smaller than it must be
    need = plsh.q4_chunk_work_bytes(a.q, a.cache)
    w = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa, work=w), wa)
    with pytest.raises(plsh.PlshError, match="work must be"):
        plsh.alibi_exact_chunk_q4(a.q, a.cache, sig, pa, work=w[:-16])
    plsh.stream_status()


PREFIXES = [
    # B, Hq, H, d, page, prefix pages, most own positions, dtype, positions
    (1, 4, 1, 128, 64, 1, 5, "bf16", [64]),
    (40, 4, 1, 128, 64, 3, 70, "bf16", [192 + (17 * b) % 70 for b in range(40)]),
    (33, 8, 2, 64, 32, 9, 40, "bf16", [-1 if b % 7 == 3 else (13 * b) % 328 for b in range(33)]),   # some within
    (70, 3, 1, 128, 16, 13, 33, "bf16", [207 + (5 * b) % 34 for b in range(70)]),     # a step that ends inside
    (17, 20, 4, 128, 128, 4, 200, "bf16", [511 + (31 * b) % 201 for b in range(17)]),
    (12, 17, 1, 64, 64, 2, 64, "bf16", [127 + (11 * b) % 65 for b in range(12)]),     # three chunks of heads
    (300, 2, 1, 64, 64, 6, 3, "bf16", [384 + b % 3 for b in range(300)]),
    # the tensor cores'
    (64, 4, 1, 128, 64, 390, 70, "bf16", [24960 + (17 * b) % 70 for b in range(64)]),
    (96, 8, 2, 64, 32, 260, 40, "bf16", [-1 if b % 7 == 3 else (131 * b) % 8360 for b in range(96)]),     # some within
    (128, 3, 1, 128, 16, 773, 33, "bf16", [12367 + (5 * b) % 34 for b in range(128)]),      # a step that ends inside
    (50, 20, 4, 128, 128, 62, 200, "bf16", [7935 + (31 * b) % 201 for b in range(50)]),
    (40, 17, 1, 64, 64, 205, 64, "bf16", [13119 + (11 * b) % 65 for b in range(40)]),       # three chunks of heads
    (16, 32, 8, 128, 256, 48, 600, "bf16", [12288 + (97 * b) % 600 for b in range(16)]),
    (300, 2, 1, 64, 64, 82, 3, "bf16", [5248 + b % 3 for b in range(300)]),                 # more rows than an item
    (16, 32, 8, 128, 256, 16, 600, "bf16", [4096 + (97 * b) % 600 for b in range(16)]),
    (1100, 40, 40, 64, 16, 8, 5, "bf16", [127 + b % 6 for b in range(1100)]),               # several items in a CTA
    (700, 64, 64, 128, 16, 7, 3, "bf16", [(7 * b) % 115 for b in range(700)]),
    (3, 8, 2, 128, 64, 3, 70, "bf16", [200, -1, 30]),
    (5, 3, 1, 64, 16, 9, 33, "f32", [144, 143, 176, -1, 0]),
    (34, 8, 1, 128, 64, 2, 10, "f32", [128 + b % 10 for b in range(34)]),
]


class Shared:
    """Sequences behind a prefix; the table's first entries are not valid."""

    def __init__(self, B, Hq, H, d, page, shared, own, dtype, seed=0):
        rng = np.random.default_rng(seed)
        per = -(-own // page)
        pages = shared + B * per + 2
        order = rng.permutation(pages).astype(np.int32)
        self.prefix, P = order[:shared], shared * page
        mine = order[shared:shared + B * per].reshape(B, per)
        self.table = np.concatenate([np.tile(self.prefix, (B, 1)), mine], 1)
        self.B, self.Hq, self.H, self.d, self.page, self.dtype, self.P = B, Hq, H, d, page, dtype, P
        g = torch.Generator("cuda").manual_seed(seed)
        data = torch.randint(0, 256, (pages, H, page // 16, 20 * d), dtype=torch.uint8, device="cuda", generator=g)
        rows = lambda b, n: [torch.randn(b, H, n, d, device="cuda", generator=g) + 0.3 for _ in range(2)]  # noqa: E731
        plsh.q4_cache_write(plsh.Q4Cache(data, i32(self.prefix[None]), H, d, page), *rows(1, P), i32([0]))
        self.full = plsh.Q4Cache(data, torch.from_numpy(self.table).cuda(), H, d, page)
        plsh.q4_cache_write(self.full, *rows(B, own), i32([P] * B))
        hidden = self.table.copy()
        hidden[:, :shared] = -9
        self.cache = plsh.Q4Cache(data, torch.from_numpy(hidden).cuda(), H, d, page)
        self.q = torch.randn(B, Hq, 1, d, device="cuda", generator=g).to(DT[dtype])
        self.d_prefix = i32(self.prefix)

    def host(self):
        return self.cache.data.cpu().numpy().reshape(self.cache.pages, self.H, -1, 20 * self.d)

    def check(self, got, pos, sigma, drop=None):
        data, got = self.host(), got.double().cpu().numpy()[:, :, 0]
        err = size = 0.0
        P = self.P
        shared = q4.read_sequence(data, self.prefix, self.page, self.d, P)
        for b in range(self.B):
            if pos[b] < 0:
                assert (got[b] == 0).all()
                continue
            if self.B * P > 10 ** 5 and b % 9 not in (0, 4) and b < self.B - 2:
                continue
            n = pos[b] + 1
            K, V = (x[:, :n] for x in shared)
            if n > P:
                mine = q4.read_sequence(data, self.table[b, P // self.page:], self.page, self.d, n - P)
                K, V = (np.concatenate([x, y], 1) for x, y in zip(shared, mine))
            w = q4.log_weights_exact(sigma, pos[b], n)
            if drop is not None:
                w[:, drop] = -np.inf
            q = self.q[b, :, 0].double().cpu().numpy()
            want = q4.decode_row(q, K, V, w)
            tol = bound(q, K, V, want, self.dtype, self.Hq // self.H)
            off = np.abs(got[b] - want)
            assert (off <= tol).all(), f"sequence {b}: off by {(off / tol).max():.2f} tolerances"
            err += ((got[b] - want) ** 2).sum()
            size += (want ** 2).sum()
        assert np.sqrt(err / size) < (2.5e-3 if self.dtype == "bf16" else 2e-6)


@pytest.mark.parametrize("case", PREFIXES, ids=[str(i) for i in range(len(PREFIXES))])
def test_prefix_decode_matches_the_oracle(case):
    *shape, pos = case
    s = Shared(*shape, seed=shape[0])
    sigma = alibi_sigmas(s.Hq)
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix)
    plsh.stream_status()
    s.check(got, pos, sigma)
    assert torch.equal(plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix), got)
    flat = np.full(s.Hq, 1e5)
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, flat, i32(pos), s.d_prefix)
    s.check(got, pos, flat)
    # every sequence within the prefix, or idle
    inside = [min(p, s.P - 1) for p in pos]
    s.check(plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(inside), s.d_prefix), inside, sigma)
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32([-1] * s.B), s.d_prefix)
    assert (got == 0).all()
    plsh.stream_status()


@pytest.mark.parametrize("dtype,B,shared", [("bf16", 96, 520), ("bf16", 40, 12), ("bf16", 3, 12), ("f32", 4, 12)])
def test_prefix_places_out_of_range_are_reported(dtype, B, shared):
    s = Shared(B, 4, 2, 128, 16, shared, 40, dtype, seed=B)
    sigma, pos = np.full(4, s.P / 2), [s.P + (7 * b) % 40 for b in range(B)]

    def failed():
        with pytest.raises(plsh.PlshError) as err:
            plsh.stream_status()
        assert err.value.status == plsh.PLSH_ERR_INVALID
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32([10 ** 6] + pos[1:]), s.d_prefix)
    failed()
    s.check(got, [-1] + pos[1:], sigma)              # (a row of 0; the others' sums may be cut elsewhere)
    bad = s.d_prefix.clone()
    bad[3] = s.cache.pages
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), bad)
    failed()
    s.check(got, pos, sigma, drop=slice(48, 64))


@pytest.mark.parametrize("B,shared", [(64, 390), (40, 3)])
def test_prefix_nan_and_queries_that_are_no_numbers(B, shared):
    s = Shared(B, 4, 1, 128, 64, shared, 64, "bf16", seed=4)
    sigma, pos = np.full(4, 60.0), [s.P + b for b in range(B)]
    pos[7] = 100                                     # does not see position 150
    want = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix)
    s.q[5, 1, 0, 3] = float("inf")
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix)
    assert torch.isnan(got[5, 1]).all() and torch.equal(got[:5], want[:5]) and torch.equal(got[6:], want[6:])
    k, v = torch.randn(2, 1, 1, 1, 128, device="cuda")
    v[..., 100] = float("nan")
    plsh.q4_cache_write(plsh.Q4Cache(s.cache.data, i32(s.prefix[None]), 1, 128, 64), k, v, i32([150]))
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix)
    assert torch.equal(got[7], want[7])
    others = [b for b in range(B) if b not in (5, 7)]
    assert torch.isnan(got[others][..., 96:]).all() and torch.isfinite(got[others][..., :96]).all()


@pytest.mark.parametrize("dtype,m,B", [("bf16", 40, 64), ("bf16", 3, 4), ("f32", 3, 4)])
def test_pages_past_four_gigabytes(dtype, m, B):
    """The same rows in a small cache and in the last pages of one of 4.6 GB."""
    H, Hq, d, page, shared, far = 8, 32, 128, 256, 16, 13900
    one = plsh.q4_cache_bytes(1, H, page, d)
    g = torch.Generator("cuda").manual_seed(3)
    prefix = torch.randperm(shared, device="cuda", generator=g).to(torch.int32)
    own = shared + torch.randperm(B, device="cuda", generator=g).to(torch.int32)
    table = torch.cat([prefix.expand(B, -1), own[:, None]], 1).contiguous()
    P = shared * page
    k, v = (torch.randn(1, H, P, d, device="cuda", generator=g) for _ in range(2))
    ko, vo = (torch.randn(B, H, 50, d, device="cuda", generator=g) for _ in range(2))
    q = torch.randn(B, Hq, 1, d, device="cuda", generator=g).to(DT[dtype])
    qc = torch.randn(2, Hq, m, d, device="cuda", generator=g).to(DT[dtype])
    pos = i32([P + (13 * b) % 50 for b in range(B)])
    outs = []
    for base in (0, far):
        data = torch.zeros((base + shared + B) * one, dtype=torch.uint8, device="cuda")
        at = plsh.Q4Cache(data, table + base, H, d, page)
        whole = plsh.Q4Cache(data, (prefix + base)[None].contiguous(), H, d, page)
        plsh.q4_cache_write(whole, k, v, i32([0]))
        plsh.q4_cache_write(at, ko, vo, i32([P] * B))
        two = plsh.Q4Cache(data, (table[:2] + base).contiguous(), H, d, page)
        sig = np.full(Hq, 2000.0)
        outs.append((plsh.alibi_exact_prefix_decode_q4(q, at, sig, pos, prefix + base),
                     plsh.alibi_exact_chunk_q4(qc, two, sig, i32([P + 50 - m, 100]))))
        plsh.stream_status()
        del data, at, whole, two
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert all(torch.isfinite(o).all() and (o != 0).any() for pair in outs for o in pair)


@pytest.mark.parametrize("B,shared", [(64, 390), (6, 3)])
def test_prefix_streams_graphs_and_workspaces(B, shared):
    """Captured, replayed at other positions on two streams at once, beside the same
    call made directly; a workspace no smaller than it must be."""
    s = Shared(B, 4, 1, 128, 64, shared, 70, "bf16", seed=8)
    sig = alibi_sigmas(4)
    pos = i32([s.P + (11 * b) % 70 for b in range(B)])
    plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, s.d_prefix)
    torch.cuda.synchronize()
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for g in graphs:
        with torch.cuda.graph(g):
            outs.append(plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, s.d_prefix))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for at in ([s.P + (7 * b) % 60 for b in range(B)], [(997 * b) % s.P if b % 3 else -1 for b in range(B)]):
        pos.copy_(i32(at))
        s.q.copy_(torch.randn_like(s.q))
        torch.cuda.synchronize()
        for _ in range(3):
            for g, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    g.replay()
            got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, s.d_prefix)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], got) and torch.equal(outs[1], got)
        s.check(got, at, sig)
    need = plsh.q4_prefix_work_bytes(s.q, s.cache)
    w = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert torch.equal(plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, s.d_prefix, work=w), got)
    with pytest.raises(plsh.PlshError, match="work must be"):
        plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, s.d_prefix, work=w[:-16])
    plsh.stream_status()


def test_a_server_s_loop_of_prompts_and_tokens():
    """The calls as they are used together: pages reserved, a shared prompt written
    and attended to in pieces, sequences of their own behind it, a token each."""
    H, Hq, d, page, B = 2, 8, 128, 16, 6
    pages, cap = 80, 12
    pool = i32(np.concatenate([[pages], np.random.default_rng(0).permutation(pages)]))
    held, table = i32([0]), i32(np.full((1, 1024), -1))
    data = torch.randint(0, 256, (pages, H, 1, 20 * d), dtype=torch.uint8, device="cuda")
    one = plsh.Q4Cache(data, table, H, d, page)
    sigma = alibi_sigmas(Hq)
    n = 96                                           # the prompt: six pages
    plsh.q4_cache_reserve(one, i32([n]), held, pool)
    K, V = torch.randn(2, 1, H, n, d, device="cuda")
    q = torch.randn(1, Hq, n, d, device="cuda").bfloat16()
    whole, parts = None, []
    for at in (0, 40, 80):
        m = min(40, n - at)
        plsh.q4_cache_write(one, K[:, :, at:at + m].contiguous(), V[:, :, at:at + m].contiguous(), i32([at]))
        parts.append(plsh.alibi_exact_chunk_q4(q[:, :, at:at + m].contiguous(), one, sigma, i32([at])))
    whole = plsh.alibi_exact_chunk_q4(q, one, sigma, i32([0])).double()
    got = torch.cat(parts, 2).double()
    assert ((got - whole).norm() / whole.norm()).item() < 2.5e-3 * 2 ** 0.5
    prefix = table[0, :6].clone()
    tables, many = i32(np.full((B, cap), -1)), i32([0] * B)
    cache = plsh.Q4Cache(data, tables, H, d, page)
    pos = i32([n - 1] * B)
    ks, vs = [], []
    for step in range(20):
        pos += 1
        plsh.q4_cache_reserve(cache, pos + 1, many, pool, prefix)
        k, v = torch.randn(2, B, H, 1, d, device="cuda")
        ks.append(k)
        vs.append(v)
        plsh.q4_cache_write(cache, k, v, pos)
        slots = plsh.q4_cache_slots(cache, pos, m=1)
        assert (slots >= 0).all() and slots.unique().numel() == B
        qs = torch.randn(B, Hq, 1, d, device="cuda").bfloat16()
        a = plsh.alibi_exact_prefix_decode_q4(qs, cache, sigma, pos, prefix).double()
        b = plsh.alibi_exact_decode_q4(qs, cache, sigma, pos).double()
        c = plsh.alibi_exact_chunk_q4(qs, cache, sigma, pos).double()
        assert ((a - b).norm() / b.norm()).item() < 2.5e-3 * 2 ** 0.5
        assert ((c - b).norm() / b.norm()).item() < 2.5e-3 * 2 ** 0.5
    plsh.q4_cache_reserve(cache, i32([0] * B), many, pool, prefix)
    assert pool[0].item() == pages - 6 and (tables == -1).all()
    plsh.stream_status()


def test_refusals():
    s = Rows(2, 4, 2, 64, 16, 40, "bf16", 6)
    sig, pos = [1.0] * 4, i32([0, 3])
    with pytest.raises(ValueError, match="lens"):
        plsh.alibi_exact_chunk_q4(s.q, s.cache, sig, pos, i32([1]))
    with pytest.raises(ValueError, match="sigma"):
        plsh.alibi_exact_chunk_q4(s.q, s.cache, sig[:3], pos)
    with pytest.raises(ValueError, match="contiguous"):
        plsh.alibi_exact_chunk_q4(s.q[..., ::1].transpose(1, 2).contiguous().transpose(1, 2), s.cache, sig, pos)
    with pytest.raises(plsh.PlshError, match="overlap"):
        plsh.alibi_exact_chunk_q4(s.q, s.cache, sig, pos, out=s.q)
    with pytest.raises(plsh.PlshError, match="shape"):
        plsh.alibi_exact_chunk_q4(s.q, s.cache, sig, pos, out=torch.empty_like(s.q, dtype=torch.float32))
    with pytest.raises(ValueError, match="prefix"):
        plsh.alibi_exact_prefix_decode_q4(s.q[:, :, :1].contiguous(), s.cache, sig, pos, i32([[1]]))
    with pytest.raises(plsh.PlshError, match="prefix_pages"):
        plsh.alibi_exact_prefix_decode_q4(s.q[:, :, :1].contiguous(), s.cache, sig, pos, i32([0, 1, 2, 3]))
    with pytest.raises(plsh.PlshError, match="q must be"):
        plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, pos, i32([0]))
