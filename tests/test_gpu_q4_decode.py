"""The decode steps over the 4-bit cache against the fp64 oracle, on the values
the cache holds.

Tolerance, from the arithmetic (derived, not fitted).  With A a bound of
sum_e |q_e| |k_e| / sqrt(d) over the keys (+ 40 for the bias of keys that still
weigh 2^-40), R the largest |lo| + 15 step of V and S the largest 15 step:
  - a score is a sum of at most 32 rounded partial sums (four groups of two
    matrix products, each counted as three roundings of an fp32 accumulator
    that may truncate, a product with step, two with lo and the bias): off by
    at most 32 * 2^-23 A in natural units, which moves o, a convex combination
    of values within R, by at most twice that times R;
    (bf16 queries: the codes are f16 subnormals, whose products the matrix
    instruction may truncate at 2^-18 of the largest in a sum; with q's and the
    codes' signs and sizes mixed that is far inside the bound above, and P V's
    is inside the next but one);
  - sums over L keys accumulate L / 16 + 64 terms one after the other at most:
    2 (L / 16 + 64) 2^-24 R for the numerator and the row sum together;
  - ex2 is within 2^-21: 2^-20 R for both;
  - fp32 keeps the weights of P V to 2^-22 (two f16 terms), bf16 to 2^-11 (one
    f16 term), times a code's S;
  - the output's rounding: 2^-24 or 2^-8 of |o|.
"""
import threading

import numpy as np
import pytest
import torch

import oracle
import positional_lsh_approximation_gb300 as plsh
from oracle import q4
from positional_lsh_approximation_gb300.inputs import alibi_sigmas

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


def tolerance(q, K, V, o, dtype, G):
    """Bound of |got - o| per query head [Hq, 1] + relative part; K, V fp64
    values [H, n, d] (finite rows only)."""
    d, n = K.shape[2], K.shape[1]
    A = np.abs(q).max(-1) * np.repeat(np.abs(K).sum(-1).max(-1), G) / np.sqrt(d) + 40
    g = V.reshape(V.shape[0], n, -1, 32)
    S = np.repeat((g.max(-1) - g.min(-1)).max((1, 2)), G) * 1.07   # 15 step: the codes' span, a step wider
    R = np.repeat(np.abs(V).max((1, 2)), G) + S
    fixed = R * (2 * 32 * 2.0 ** -23 * A + 2 * (n / 16 + 64) * 2.0 ** -24 + 2.0 ** -20)
    fixed = fixed + S * (2.0 ** -11 if dtype == "bf16" else 2.0 ** -22)
    return fixed[:, None] + np.abs(o) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24)


class Setup:
    """A cache of random rows written by the library, its bytes on the host."""

    def __init__(self, B, Hq, H, d, page, n, dtype, seed=0, scale=1.0, spare=3):
        rng = np.random.default_rng(seed)
        per = -(-n // page)
        pages = B * per + spare
        self.table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
        self.B, self.Hq, self.H, self.d, self.page, self.n, self.dtype = B, Hq, H, d, page, n, dtype
        data = torch.randint(0, 256, (pages, H, page // 16, 20 * d), dtype=torch.uint8, device="cuda",
                             generator=torch.Generator("cuda").manual_seed(seed))
        self.cache = plsh.Q4Cache(data, torch.from_numpy(self.table).cuda(), H, d, page)
        g = torch.Generator("cuda").manual_seed(seed + 1)
        self.k, self.v = (torch.randn(B, H, n, d, device="cuda", generator=g) * scale + 0.3 for _ in range(2))
        plsh.q4_cache_write(self.cache, self.k, self.v, i32([0] * B))
        self.q = torch.randn(B, Hq, 1, d, device="cuda", generator=g).to(DT[dtype])
        self.rng = rng

    def host(self):
        return self.cache.data.cpu().numpy().reshape(self.cache.pages, self.H, -1, 20 * self.d)

    def check(self, got, pos, log_w):
        """got [B, Hq, 1, d]; log_w(b, pos, n) the weights of sequence b."""
        data = self.host()
        q = self.q.double().cpu().numpy()[:, :, 0]
        got = got.double().cpu().numpy()[:, :, 0]
        for b in range(self.B):
            if pos[b] < 0:
                assert (got[b] == 0).all()
                continue
            n = pos[b] + 1
            K, V = q4.read_sequence(data, self.table[b], self.page, self.d, n)
            want = q4.decode_row(q[b], K, V, log_w(pos[b], n))
            tol = tolerance(q[b], K, V, want, self.dtype, self.Hq // self.H)
            off = np.abs(got[b] - want)
            assert (off <= tol).all(), f"sequence {b}: off by {(off / tol).max():.2f} tolerances"


CASES = [
    # B, Hq, H, d, page, n, dtype, positions
    (1, 1, 1, 128, 16, 1, "bf16", [0]),
    (1, 1, 1, 64, 16, 1, "f32", [0]),
    (3, 8, 2, 128, 64, 300, "bf16", [299, 0, 15]),
    (5, 8, 2, 64, 32, 530, "bf16", [529, -1, 16, 511, 512]),          # an idle slot
    (2, 3, 1, 128, 256, 700, "f32", [699, 255]),
    (3, 12, 1, 64, 16, 400, "f32", [399, 31, 32]),                    # twelve heads on one
    (2, 24, 2, 128, 64, 900, "bf16", [899, 63]),
    (1, 20, 4, 128, 128, 1500, "bf16", [1487]),                       # five heads on one
    (40, 4, 4, 128, 64, 200, "bf16", [(37 * b) % 200 for b in range(40)]),
    (2, 32, 8, 128, 64, 4100, "bf16", [4099, 2048]),
    (1, 16, 1, 64, 64, 6000, "f32", [5999]),
    (2, 17, 1, 128, 32, 333, "bf16", [332, 100]),                     # seventeen: three chunks
]
IDS = [str(i) for i in range(len(CASES))]


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_exact_decode_matches_the_oracle(case):
    *shape, pos = case
    s = Setup(*shape, seed=shape[5])
    sigma = alibi_sigmas(s.Hq)
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, n: q4.log_weights_exact(sigma, p, n))


@pytest.mark.parametrize("hashes", [1, 6, 64])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_approximate_decode_matches_the_oracle(case, hashes):
    *shape, pos = case
    s = Setup(*shape, seed=shape[5] + hashes)
    sigma = np.exp2(np.linspace(0.5, 9, s.Hq))
    n = s.n + 5                                      # bins of another length than the cache
    bins = plsh.sample_bins(n, sigma, hashes, seed=hashes)
    off, st = bins.to_host()
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, m: q4.log_weights_approx(off, st, s.Hq, hashes, p, m))
    bins.free()


WIDE = [
    # shape as above, scales, positions: rows of 2, 4 and 8 CTAs, some with
    # nothing for most of them; the last two by a second kernel
    ((3, 3, 1, 64, 16, 3000, "f32"), [700.0, 20, 300], [2999, 5, -1]),
    ((2, 5, 1, 128, 64, 1100, "bf16"), [900.0, 3, 40, 500, 2], [1099, 640]),
    ((2, 8, 2, 64, 32, 1200, "bf16"), [1.0, 2, 4, 8, 60, 80, 100, 120], [1199, 33]),
    ((1, 34, 34, 64, 32, 2100, "f32"), [300.0] * 34, [2077]),           # more KV heads than are ordered
    ((2, 11, 1, 128, 128, 5000, "bf16"), [1e4] * 11, [4999, 4095]),     # two chunks of heads
    ((1, 4, 1, 64, 64, 12001, "bf16"), [1e5] * 4, [12000]),
    ((30, 4, 2, 64, 64, 2000, "f32"), [1e4] * 4, [1999 - 61 * b for b in range(30)]),
    # and more rows than fit at once, idle ones among them
    ((700, 4, 2, 64, 64, 400, "bf16"), [1.0, 5, 40, 300], [(97 * b) % 401 - 1 for b in range(700)]),
]


@pytest.mark.parametrize("case", WIDE, ids=[str(i) for i in range(len(WIDE))])
def test_rows_that_several_ctas_share(case):
    shape, sigma, pos = case
    s = Setup(*shape, seed=5)
    bins = plsh.sample_bins(s.n, sigma, 7, seed=3)
    off, st = bins.to_host()
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, m: q4.log_weights_approx(off, st, s.Hq, 7, p, m))
    again = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    assert torch.equal(got, again)
    bins.free()


@pytest.mark.parametrize("sigma", [0.05, 1e6])
def test_one_bin_and_the_steepest_and_flattest_slopes(sigma):
    s = Setup(2, 4, 2, 128, 64, 3000, "f32", seed=8)
    pos = [2999, 1024]
    sig = np.full(4, sigma)
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sig, i32(pos))
    s.check(got, pos, lambda p, n: q4.log_weights_exact(sig, p, n))
    # one bin over everything: every key, every hash; then singletons
    for starts in (np.array([0, 3000]), np.arange(3001)):
        off = np.arange(0, 4 * 3 * len(starts) + 1, len(starts))
        st = np.tile(starts, 12)
        bins = plsh.bins_from_host(3000, 4, 3, off, st)
        got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
        plsh.stream_status()
        s.check(got, pos, lambda p, n: q4.log_weights_approx(off, st, 4, 3, p, n))
        bins.free()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_values(dtype):
    """Queries far from unit scale in both directions, values of every group
    of very different sizes: the weights' and codes' scales follow them."""
    s = Setup(2, 8, 2, 128, 64, 500, dtype, seed=5)
    size = torch.tensor([1e4, 1.0, 1e-4, 1e-8], device="cuda").repeat_interleave(32)
    s.v = s.v * size
    s.k[:, :, 100:130] *= 3
    for qs, ks in ((1e3, 1e-3), (1e-6, 1e6), (30.0, 1.0)):
        k = s.k * ks
        plsh.q4_cache_write(s.cache, k, s.v, i32([0, 0]))
        s.q = torch.randn(2, 8, 1, 128, device="cuda").to(DT[dtype]) * qs
        pos = [499, 77]
        sigma = alibi_sigmas(8)
        got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
        plsh.stream_status()
        data = s.host()
        q = s.q.double().cpu().numpy()[:, :, 0]
        for b in range(2):
            K, V = q4.read_sequence(data, s.table[b], 64, 128, pos[b] + 1)
            want = q4.decode_row(q[b], K, V, q4.log_weights_exact(sigma, pos[b], pos[b] + 1))
            # group by group, so that a small group is held to its own size
            for y in range(4):
                sl = slice(32 * y, 32 * y + 32)
                tol = tolerance(q[b], K, V[:, :, sl], want[:, sl], dtype, 4)
                off = np.abs(got.double().cpu().numpy()[b, :, 0, sl] - want[:, sl])
                assert (off <= tol).all(), f"group {y}: {(off / tol).max():.2f}"


def poison(s, b, p, which):
    """NaN into position p of sequence b (a value of K or V of every head)."""
    k = s.k[b:b + 1, :, p:p + 1].clone()
    v = s.v[b:b + 1, :, p:p + 1].clone()
    (k if which == "k" else v)[..., 5] = float("nan")
    table = torch.from_numpy(s.table[b:b + 1].copy()).cuda()
    plsh.q4_cache_write(plsh.Q4Cache(s.cache.data, table, s.H, s.d, s.page), k, v, i32([p]))


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_past_the_position_or_outside_the_bins_has_no_effect(which, dtype):
    s = Setup(2, 4, 1, 128, 64, 400, dtype, seed=2)
    pos = [207, 399]
    starts = [np.array([0, 150, 401]), np.array([0, 190, 401]), np.array([0, 203, 401]),
              np.array([0, 207, 401])]
    off = np.concatenate([[0], np.cumsum([len(x) for x in starts])])
    st = np.concatenate(starts)
    bins = plsh.bins_from_host(401, 4, 1, off, st)
    sigma = alibi_sigmas(4)
    want = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    want_e = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    poison(s, 0, 208, which)                  # the next position, in the same tile
    poison(s, 0, 300, which)
    assert torch.equal(plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos)), want_e)
    poison(s, 0, 200, which)                  # seen by heads 0 and 1 alone, in the others' tile
    poison(s, 0, 148, which)                  # seen by none
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    plsh.stream_status()
    assert torch.equal(got[1], want[1]) and torch.equal(got[0, 2:], want[0, 2:])
    seen = torch.isnan(got[0, :2, 0])
    if which == "k":
        assert seen.all()                     # a NaN score makes the row NaN
    else:                                     # a NaN value its group of the row
        assert seen[:, :32].all() and torch.equal(got[0, :2, 0, 32:], want[0, :2, 0, 32:])
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    assert torch.isnan(got[0]).any() and torch.equal(got[1], want_e[1])
    bins.free()


@pytest.mark.parametrize("heads", [(4, 4), (8, 2), (8, 1)])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_what_was_never_written_has_no_effect(heads, d, dtype):
    """Pages of zeros and pages of NaN around the same rows: the same bits.
    The rows begin inside a tile, behind positions that no head sees."""
    Hq, H = heads
    s = Setup(2, Hq, H, d, 32, 130, dtype, seed=21)
    pos, start = [93, 129], 21
    starts = np.array([0, start, 131])            # the second bin: positions start ..
    off = np.arange(0, 3 * Hq + 1, 3)
    bins = plsh.bins_from_host(131, Hq, 1, off, np.tile(starts, Hq))
    sigma = alibi_sigmas(Hq)
    got = []
    for fill in (0, 255):
        s.cache.data.fill_(fill)
        plsh.q4_cache_write(s.cache, s.k[:, :, :109].contiguous(), s.v[:, :, :109].contiguous(),
                            i32([start] * 2), i32([93 - start + 1, 109]))
        a = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
        plsh.q4_cache_write(s.cache, s.k, s.v, i32([0, 0]), i32([94, 130]))
        got.append((a, plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))))
        plsh.stream_status()
    for a, b in zip(*got):
        assert torch.isfinite(a).all() and torch.equal(a, b)
    bins.free()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_that_is_not_finite_spoils_its_own_head_alone(bad):
    s = Setup(1, 4, 1, 64, 16, 100, "f32", seed=2)
    sigma = alibi_sigmas(4)
    want = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32([99]))
    s.q[0, 2, 0, 7] = bad
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32([99]))
    assert torch.isnan(got[0, 2]).all()
    keep = [0, 1, 3]
    assert torch.equal(got[0, keep], want[0, keep])


def test_places_out_of_range_are_reported():
    s = Setup(3, 4, 2, 128, 16, 64, "bf16", seed=3)
    sigma = alibi_sigmas(4)
    bins = plsh.sample_bins(60, sigma, 4, 0)

    def failed():
        with pytest.raises(plsh.PlshError) as err:
            plsh.stream_status()
        assert err.value.status == plsh.PLSH_ERR_INVALID
    # past the pages, and below them but past the bins
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32([64, 2 ** 31 - 1, 63]))
    failed()
    assert (got[:2] == 0).all() and (got[2] != 0).any()
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32([60, 59, -2 ** 31]))
    failed()
    assert (got[0] == 0).all() and (got[1] != 0).any() and (got[2] == 0).all()
    # a bad page: its keys are absent (sequence 1's second page)
    pos = [40, 40, 40]
    want = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    plsh.stream_status()
    for bad in (-1, s.cache.pages, -2 ** 31):
        s.cache.table[1, 1] = bad
        got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
        failed()
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        data, q = s.host(), s.q.double().cpu().numpy()[1, :, 0]
        t = s.table[1].copy()
        t[1] = 0
        K, V = q4.read_sequence(data, t, 16, 128, 41)
        w = q4.log_weights_exact(sigma, 40, 41)
        w[:, 16:32] = -np.inf
        o = q4.decode_row(q, K, V, w)
        assert (np.abs(got[1, :, 0].double().cpu().numpy() - o) <= tolerance(q, K, V, o, "bf16", 2)).all()
    # every page bad: nothing is seen
    s.cache.table[1] = -1
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    failed()
    assert (got[1] == 0).all()
    # pages past the position are not read
    s.cache.table.copy_(torch.from_numpy(s.table))
    s.cache.table[:, 3] = -5
    assert torch.equal(plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos)), want)
    plsh.stream_status()
    bins.free()


def test_the_decode_loop_of_a_batch():
    """As a serving loop uses them: prompts written, then one token at a time
    appended and attended to, approximate and exact; after each step both rows
    against the oracle, and the approximate one against the decode step over
    the fp32 rows that the cache reads back as."""
    B, Hq, H, d, page, n = 3, 8, 2, 128, 16, 120
    s = Setup(B, Hq, H, d, page, n, "f32", seed=11)
    sigma = alibi_sigmas(Hq)
    bins = plsh.sample_bins(n, sigma, 5, 1)
    off, st = bins.to_host()
    lens = [100, 37, 64]
    prompt = torch.randn(2, B, H, 100, d, device="cuda")
    plsh.q4_cache_write(s.cache, prompt[0], prompt[1], i32([0, 0, 0]), i32(lens))
    pos = i32(lens)
    for step in range(4):
        k, v = torch.randn(2, B, H, 1, d, device="cuda")
        s.q = torch.randn(B, Hq, 1, d, device="cuda")
        plsh.q4_cache_write(s.cache, k, v, pos)
        o = plsh.alibi_decode_q4(s.q, s.cache, bins, pos)
        e = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, pos)
        plsh.stream_status()
        at = [x + step for x in lens]
        s.check(o, at, lambda p, m: q4.log_weights_approx(off, st, Hq, 5, p, m))
        s.check(e, at, lambda p, m: q4.log_weights_exact(sigma, p, m))
        K, V = plsh.q4_cache_read(s.cache, i32([0] * B), m=n, dtype=torch.float32)
        for b in range(B):
            row = plsh.alibi_decode(s.q[b:b + 1].contiguous(), K[b:b + 1].contiguous(),
                                    V[b:b + 1].contiguous(), bins, at[b])
            torch.testing.assert_close(o[b:b + 1], row, atol=1e-4, rtol=1e-4)
        pos += 1
    bins.free()


def test_two_streams_and_two_graphs_with_their_own_workspaces():
    """Calls that run at once, each with its workspace, give what they give
    alone; so do replays of two graphs at once, with positions changed."""
    a = Setup(2, 8, 2, 128, 64, 3000, "bf16", seed=1)
    b = Setup(3, 8, 2, 64, 32, 2500, "bf16", seed=2)
    sig = alibi_sigmas(8)
    bins = plsh.sample_bins(3000, sig, 6, 2)
    pa, pb = i32([2999, 1500]), i32([2499, 3, 700])
    wa = plsh.alibi_exact_decode_q4(a.q, a.cache, sig, pa)
    wb = plsh.alibi_decode_q4(b.q, b.cache, bins, pb)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        ga = plsh.alibi_exact_decode_q4(a.q, a.cache, sig, pa, stream=s1)
        gb = plsh.alibi_decode_q4(b.q, b.cache, bins, pb, stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        ga = plsh.alibi_exact_decode_q4(a.q, a.cache, sig, pa)
    with torch.cuda.graph(g2):
        gb = plsh.alibi_decode_q4(b.q, b.cache, bins, pb)
    for qa, qb in (([2999, 1500], [2499, 3, 700]), ([17, -1], [2000, 2499, 0])):
        pa.copy_(i32(qa))
        pb.copy_(i32(qb))
        wa = plsh.alibi_exact_decode_q4(a.q, a.cache, sig, pa)
        wb = plsh.alibi_decode_q4(b.q, b.cache, bins, pb)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s1):
                g1.replay()
            with torch.cuda.stream(s2):
                g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(ga, wa) and torch.equal(gb, wb)
    plsh.stream_status()
    bins.free()


def test_two_threads_on_one_stream():
    """Calls of two threads on one stream share the cache's workspace; the
    kernels of one are not parted by the other's."""
    s = Setup(6, 8, 2, 128, 64, 3000, "bf16", seed=11)
    sig = alibi_sigmas(8)
    at = [i32([2999 - 17 * b for b in range(6)]), i32([100 + 450 * b for b in range(6)])]
    want = [plsh.alibi_exact_decode_q4(s.q, s.cache, sig, p) for p in at]
    got = [[], []]

    def work(k):
        for _ in range(200):
            got[k].append(plsh.alibi_exact_decode_q4(s.q, s.cache, sig, at[k]))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 200 and all(torch.equal(o, want[k]) for o in got[k])


def test_the_same_call_gives_the_same_bits():
    s = Setup(9, 8, 2, 128, 64, 2000, "bf16", seed=4)
    pos = i32([(431 * b) % 2000 for b in range(9)])
    sig = alibi_sigmas(8)
    first = plsh.alibi_exact_decode_q4(s.q, s.cache, sig, pos)
    work = torch.full((plsh.q4_decode_work_bytes(s.q, s.cache),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(plsh.alibi_exact_decode_q4(s.q, s.cache, sig, pos, work=work), first)


def test_many_sequences_with_idle_ones_among_them():
    """More sequences than a block has threads, a third of them idle, some one
    block long: the exact step's split runs over them all."""
    B = 300
    s = Setup(B, 2, 1, 64, 16, 100, "f32", seed=31)
    pos = [-1 if b % 3 == 1 else (7 * b) % 100 if b % 2 else b % 20 for b in range(B)]
    sigma = np.array([3.0, 40.0])
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, n: q4.log_weights_exact(sigma, p, n))
    bins = plsh.sample_bins(100, sigma, 3, 5)
    off, st = bins.to_host()
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, n: q4.log_weights_approx(off, st, 2, 3, p, n))
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32([-1] * B))
    assert (got == 0).all()
    bins.free()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [1, 6])
def test_more_kv_heads_than_are_ordered(dtype, group):
    """Forty KV heads (the approximate step orders up to 32 by their scales)."""
    H = 40
    s = Setup(2, H * group, H, 64, 64, 700, dtype, seed=33)
    sigma = np.exp2(np.linspace(0, 11, H * group))
    bins = plsh.sample_bins(700, sigma, 4, 6)
    off, st = bins.to_host()
    pos = [699, 310]
    got = plsh.alibi_decode_q4(s.q, s.cache, bins, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, n: q4.log_weights_approx(off, st, H * group, 4, p, n))
    got = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32(pos))
    plsh.stream_status()
    s.check(got, pos, lambda p, n: q4.log_weights_exact(sigma, p, n))
    bins.free()


def test_pages_whose_bytes_begin_past_32_bits():
    """The same rows in the first pages and in pages past 2^32 bytes."""
    H, d, page = 8, 128, 256
    one = plsh.q4_cache_bytes(1, H, page, d)
    pages = 2 ** 32 // one + 40
    table = i32([[0, 1, 2], [pages - 1, pages - 30, pages - 2]])
    cache = plsh.Q4Cache.empty(pages, H, d, table, page)
    g = torch.Generator("cuda").manual_seed(4)
    k, v = (torch.randn(1, H, 700, d, device="cuda", generator=g).expand(2, -1, -1, -1).contiguous()
            for _ in range(2))
    q = torch.randn(1, 32, 1, d, device="cuda", generator=g).expand(2, -1, -1, -1).contiguous().bfloat16()
    plsh.q4_cache_write(cache, k, v, i32([0, 0]))
    sigma = alibi_sigmas(32)
    bins = plsh.sample_bins(768, sigma, 6, 1)
    o = plsh.alibi_decode_q4(q, cache, bins, i32([699, 699]))
    assert torch.equal(o[0], o[1]) and torch.isfinite(o).all()
    # alone, a row is cut as it is cut alone in the other place
    e = [plsh.alibi_exact_decode_q4(q, cache, sigma, i32(p)) for p in ([699, -1], [-1, 699])]
    plsh.stream_status()
    assert torch.equal(e[0][0], e[1][1]) and torch.isfinite(e[0][0]).all() and (e[0][0] != 0).any()
    bins.free()


def test_shared_prefix_pages():
    """Two sequences whose tables name the same pages read the same keys.  (The
    exact step cuts the two rows at different tiles, so that their sums are
    taken in another order: each is held to the oracle, not to the other.)"""
    s = Setup(2, 4, 2, 64, 16, 200, "f32", seed=9)
    s.cache.table[1] = s.cache.table[0]
    s.table[1] = s.table[0]
    s.q[1] = s.q[0]
    sigma = alibi_sigmas(4)
    o = plsh.alibi_exact_decode_q4(s.q, s.cache, sigma, i32([150, 150]))
    plsh.stream_status()
    s.check(o, [150, 150], lambda p, n: q4.log_weights_exact(sigma, p, n))


def test_binding_and_workspace_refusals():
    s = Setup(2, 4, 2, 64, 16, 50, "f32", seed=9)
    sig, pos = alibi_sigmas(4), i32([3, 4])
    small = torch.empty(plsh.q4_decode_work_bytes(s.q, s.cache) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(plsh.PlshError):
        plsh.alibi_exact_decode_q4(s.q, s.cache, sig, pos, work=small)
    with pytest.raises(ValueError):
        plsh.alibi_exact_decode_q4(s.q, s.cache, sig[:2], pos)
    with pytest.raises(ValueError):
        plsh.alibi_exact_decode_q4(s.q, s.cache, sig, pos.long())
    with pytest.raises(ValueError):
        plsh.alibi_exact_decode_q4(s.q.cpu(), s.cache, sig, pos)
    with pytest.raises(plsh.PlshError):
        plsh.alibi_exact_decode_q4(s.q, s.cache, sig, pos, out=torch.empty(2, 4, 1, 128, device="cuda"))
    bins = plsh.sample_bins(50, [1.0, 2.0], 2, 0)
    with pytest.raises(plsh.PlshError):
        plsh.alibi_decode_q4(s.q, s.cache, bins, pos)              # bins of two heads
    bins.free()
