"""Writing and reading the 4-bit paged cache against the numpy oracle: stored
bytes bit for bit, values exact up to the output's rounding, and everything a
call does not name left as it was."""
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


def make(B, H, d, page, per, seed, spare=2):
    """A cache filled with random bytes, a shuffled page table."""
    rng = np.random.default_rng(seed)
    pages = B * per + spare
    data = rng.integers(0, 256, (pages, H, page // 16, 20 * d), dtype=np.uint8)
    table = rng.permutation(pages)[:B * per].reshape(B, per).astype(np.int32)
    cache = plsh.Q4Cache(torch.from_numpy(data).cuda(), torch.from_numpy(table).cuda(), H, d, page)
    return cache, data, table, rng


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def host_write(data, table, page, K, V, pos, lens):
    B, H, m, d = K.shape
    for b in range(B):
        for i in range(max(0, min(lens[b], m))):
            p = pos[b] + i
            for h in range(H):
                q4.write_row(data[table[b, p // page], h, p % page // 16], p % 16, K[b, h, i], V[b, h, i])


def rows(rng, shape, dtype):
    """fp32 arrays of values that `dtype` holds, and the same on the device."""
    x = [torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * 2 + 0.5).to(DT[dtype])
         for _ in range(2)]
    return [t.float().numpy() for t in x], [t.cuda() for t in x]


CASES = [
    # B, H, d, page, pages a sequence, m, first positions, lengths, dtype
    (1, 1, 128, 16, 1, 1, [0], None, "bf16"),
    (1, 1, 64, 16, 1, 16, [0], None, "f32"),
    (3, 2, 128, 64, 3, 70, [0, 63, 122], None, "bf16"),       # across pages, inside tiles
    (4, 3, 64, 32, 4, 33, [5, 16, 31, 90], [33, 0, 1, 17], "f32"),
    (3, 2, 64, 128, 2, 200, [56, 0, 1], [200, -4, 900], "bf16"),   # lengths taken within 0..m
    (2, 5, 128, 256, 1, 47, [209, 13], [47, 46], "f32"),
    (70, 1, 128, 16, 2, 1, [b % 32 for b in range(70)], None, "bf16"),   # a token each
    (2, 2, 128, 64, 5, 257, [0, 48], [256, 257], "bf16"),     # whole tiles and ragged ends
    (1, 2, 64, 64, 5, 301, [15], None, "f32"),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
def test_write_and_read_match_the_oracle(case):
    B, H, d, page, per, m, pos, lens, dtype = case
    cache, data, table, rng = make(B, H, d, page, per, m + d)
    (K, V), (k, v) = rows(rng, (B, H, m, d), dtype)
    n = lens if lens is not None else [m] * B
    ln = i32(lens) if lens is not None else None
    plsh.q4_cache_write(cache, k, v, i32(pos), ln)
    plsh.stream_status()
    host_write(data, table, page, K, V, pos, n)
    np.testing.assert_array_equal(cache.data.cpu().numpy(), data)
    # read back as both types; rows past the length keep what was there
    for out in ("f32", "bf16"):
        pair = tuple(torch.full((B, H, m, d), 7.0, dtype=DT[out], device="cuda") for _ in range(2))
        plsh.q4_cache_read(cache, i32(pos), ln, out=pair)
        plsh.stream_status()
        for b in range(B):
            L = max(0, min(n[b], m))
            want = q4.read_sequence(data, table[b], page, d, pos[b] + L) if L else (None, None)
            for got, w in zip(pair, want):
                assert (got[b, :, L:] == 7.0).all()
                if L:
                    # fp32: one rounding of lo + step c; bf16: that, rounded again
                    f = torch.from_numpy(w[:, pos[b]:].astype(np.float32))
                    assert torch.equal(got[b, :, :L].cpu(), f.to(DT[out]))


def test_read_allocates_zeros_past_the_lengths():
    cache, data, table, _ = make(2, 1, 64, 16, 2, 5)
    k, v = plsh.q4_cache_read(cache, i32([0, 3]), i32([4, 9]), m=9, dtype=torch.float32)
    assert k.shape == (2, 1, 9, 64) and (k[0, :, 4:] == 0).all() and (v[0, :, 4:] == 0).all()
    with pytest.raises(ValueError):
        plsh.q4_cache_read(cache, i32([0, 3]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_unusual_values_match_the_oracle(dtype, d):
    """Constants, zeros of both signs, ties, subnormals, the largest numbers,
    values far apart, infinities and NaN, each in groups of its own."""
    cache, data, table, rng = make(1, 1, d, 16, 8, 1)
    m = 96
    x = rng.standard_normal((1, 1, m, d)).astype(np.float32)
    x[0, 0, 0] = 0.0
    x[0, 0, 1, ::2] = -0.0
    x[0, 0, 1, 1::2] = 0.0
    x[0, 0, 2] = -2.5
    x[0, 0, 3] = np.arange(d) % 16 + 0.0
    x[0, 0, 4] = np.where(np.arange(d) % 32 < 2, 15 * (np.arange(d) % 2), np.arange(d) % 15 + 0.5)
    x[0, 0, 5] *= 1e-39
    x[0, 0, 6] *= 1e37
    x[0, 0, 7] = np.where(rng.random(d) < 0.5, 1e30, 1e-30)
    x[0, 0, 8, 3] = np.inf
    x[0, 0, 9, 33] = -np.inf
    x[0, 0, 10, 40] = np.nan
    x[0, 0, 11] = 3.3e38
    x[0, 0, 12] = np.where(np.arange(d) % 2, 3.3e38, -3.3e38)
    x[0, 0, 13] = -np.nan
    x[0, 0, 14] = 100.0 + 0.01 * rng.standard_normal(d)
    x[0, 0, 15] = np.where(np.arange(d) % 32 == 0, -3.4e38, 0.0)
    t = torch.from_numpy(x).to(DT[dtype])
    x = t.float().numpy()
    plsh.q4_cache_write(cache, t.cuda(), t.cuda(), i32([5]))
    plsh.stream_status()
    host_write(data, table, 16, x, x, [5], [m])
    np.testing.assert_array_equal(cache.data.cpu().numpy(), data)


def test_many_random_quotients_match_the_oracle():
    """Quotients next to a half, where a quotient formed in another way than
    by one rounded division would pick the other code."""
    cache, data, table, rng = make(1, 1, 128, 256, 9, 2)
    m = 2304
    x = (rng.integers(-400, 400, (2, 1, 1, m, 128)) / 16.0).astype(np.float32)
    x[1] *= np.float32(1 / 3)
    k, v = torch.from_numpy(x[0]).cuda(), torch.from_numpy(x[1]).cuda()
    plsh.q4_cache_write(cache, k, v, i32([0]))
    plsh.stream_status()
    got = plsh.q4_cache_read(cache, i32([0]), m=m, dtype=torch.float32)
    for g, x_ in zip(got, x):
        c, lo, step = q4.quantise(x_)
        want = (np.repeat(lo, 32, -1).astype(np.float64)
                + np.repeat(step, 32, -1).astype(np.float64) * c).astype(np.float32)
        np.testing.assert_array_equal(g.cpu().numpy(), want)


def status():
    with pytest.raises(plsh.PlshError) as err:
        plsh.stream_status()
    plsh.stream_status()                                   # reported once
    return err.value.status


def test_places_out_of_range_are_skipped_and_reported():
    B, H, d, page, per, m = 3, 2, 128, 16, 2, 20
    cache, data, table, rng = make(B, H, d, page, per, 9)
    (K, V), (k, v) = rows(rng, (B, H, m, d), "bf16")
    # sequence 0 starts before its first position, 1 runs past its pages, 2 has
    # a bad second page
    pos = [-3, 20, 0]
    for bad in (-1, cache.pages, 2 ** 31 - 1, -2 ** 31):
        table[2, 1] = bad
        cache.table.copy_(torch.from_numpy(table))
        before = cache.data.cpu().numpy()
        want = before.copy()
        plsh.q4_cache_write(cache, k, v, i32(pos))
        assert status() == plsh.PLSH_ERR_INVALID
        host_write(want, table, page, K[:1, :, 3:], V[:1, :, 3:], [0], [17])
        host_write(want, table[1:2], page, K[1:2], V[1:2], [20], [12])
        host_write(want, table[2:], page, K[2:], V[2:], [0], [16])
        np.testing.assert_array_equal(cache.data.cpu().numpy(), want)
        pair = tuple(torch.full((B, H, m, d), 7.0, device="cuda") for _ in range(2))
        plsh.q4_cache_read(cache, i32(pos), out=pair)
        assert status() == plsh.PLSH_ERR_INVALID
        for x in pair:
            assert (x[0, :, :3] == 7).all() and (x[1, :, 12:] == 7).all() and (x[2, :, 16:] == 7).all()
            assert (x[0, :, 3:] != 7).any() and (x[1, :, :12] != 7).any()


def test_positions_near_the_largest_are_refused_without_wrapping():
    cache, data, _, rng = make(1, 1, 64, 16, 1, 4)
    _, (k, v) = rows(rng, (1, 1, 40, 64), "f32")
    plsh.q4_cache_write(cache, k, v, i32([2 ** 31 - 20]))
    assert status() == plsh.PLSH_ERR_INVALID
    plsh.q4_cache_write(cache, k, v, i32([-2 ** 31]))
    assert status() == plsh.PLSH_ERR_INVALID
    np.testing.assert_array_equal(cache.data.cpu().numpy(), data)


def test_offsets_past_32_bits():
    """Pages whose bytes begin past 2^32."""
    H, d, page = 8, 128, 256
    one = plsh.q4_cache_bytes(1, H, page, d)
    pages = 2 ** 32 // one + 40
    cache = plsh.Q4Cache.empty(pages, H, d, i32([[pages - 1, 2, pages - 30]]), page)
    rng = np.random.default_rng(0)
    (K, V), (k, v) = rows(rng, (1, H, 700, d), "bf16")
    plsh.q4_cache_write(cache, k, v, i32([10]))
    got = plsh.q4_cache_read(cache, i32([10]), m=700, dtype=torch.float32)
    plsh.stream_status()
    for g, x in zip(got, (K, V)):
        c, lo, step = q4.quantise(x)
        want = (np.repeat(lo, 32, -1).astype(np.float64)
                + np.repeat(step, 32, -1).astype(np.float64) * c).astype(np.float32)
        np.testing.assert_array_equal(g.cpu().numpy(), want)


def test_another_stream_and_a_replayed_graph():
    cache, data, table, rng = make(2, 2, 64, 32, 4, 6)
    (K, V), (k, v) = rows(rng, (2, 2, 3, 64), "bf16")
    pos = i32([0, 50])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plsh.q4_cache_write(cache, k, v, pos, stream=side)
    got = plsh.q4_cache_read(cache, pos, m=3, dtype=torch.float32, stream=side)
    side.synchronize()
    host_write(data, table, 32, K, V, [0, 50], [3, 3])
    np.testing.assert_array_equal(cache.data.cpu().numpy(), data)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plsh.q4_cache_write(cache, k, v, pos)
        out = plsh.q4_cache_read(cache, pos, m=3, dtype=torch.float32)
    for step in range(3):
        (K, V), (a, b) = rows(rng, (2, 2, 3, 64), "bf16")
        k.copy_(a)
        v.copy_(b)
        pos.copy_(i32([3 * step + 3, 53 + step]))
        graph.replay()
        torch.cuda.synchronize()
        host_write(data, table, 32, K, V, [3 * step + 3, 53 + step], [3, 3])
        np.testing.assert_array_equal(cache.data.cpu().numpy(), data)
        want = q4.read_sequence(data, table[1], 32, 64, 56 + step)[0][:, 53 + step:]
        np.testing.assert_array_equal(out[0][1].cpu().numpy(), want.astype(np.float32))
    del got


def test_binding_refuses_what_it_cannot_pass_on():
    cache, _, _, rng = make(2, 2, 64, 32, 2, 6)
    _, (k, v) = rows(rng, (2, 2, 3, 64), "bf16")
    pos = i32([0, 1])
    for bad in (pos.long(), pos[:1], pos.cpu(), torch.stack([pos, pos], 1)[:, 0]):
        with pytest.raises(ValueError):
            plsh.q4_cache_write(cache, k, v, bad)
    with pytest.raises(ValueError):
        plsh.q4_cache_write(cache, k.transpose(1, 2), v, pos)
    with pytest.raises(ValueError):
        plsh.q4_cache_write(cache, k.half(), v.half(), pos)
    with pytest.raises(ValueError):
        plsh.q4_cache_write(cache, k.cpu(), v, pos)
    with pytest.raises(plsh.PlshError):
        plsh.q4_cache_write(cache, k[:1].contiguous(), v[:1].contiguous(), pos)


def test_tensors_of_a_cache_are_not_exchanged():
    """A call's addresses are taken when the cache is made."""
    cache = plsh.Q4Cache.empty(4, 1, 64, torch.zeros(1, 4, dtype=torch.int32, device="cuda"), 16)
    with pytest.raises(AttributeError):
        cache.table = cache.table.clone()
    with pytest.raises(AttributeError):
        cache.data = cache.data.clone()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows_are_written_as_few_are(dtype, d):
    """A call of many rows and calls of ten leave the same bytes (the latter are
    held to the oracle above): ragged positions and lengths, groups of ties,
    constants, infinities and NaN among them."""
    B, H, m, page, per = 16, 8, 350, 32, 12
    gen = torch.Generator("cuda").manual_seed(d)
    table = torch.randperm(B * per, device="cuda", generator=gen).to(torch.int32).view(B, per)
    a, b = (plsh.Q4Cache(torch.full((plsh.q4_cache_bytes(B * per, H, page, d),), 9, dtype=torch.uint8,
                                    device="cuda"), table, H, d, page) for _ in range(2))
    k, v = (torch.randn(B, H, m, d, device="cuda", generator=gen) for _ in range(2))
    k[:, :, ::7] = (k[:, :, ::7] * 4).round() / 2                    # halves of codes
    k[:, ::3, 5::11] = 1.5
    v[1, :, 3::9, 40] = float("inf")
    v[2, 1, 4::9, 7] = float("nan")
    v[3] *= 1e-39
    v[4] *= 1e37
    k, v = k.to(DT[dtype]), v.to(DT[dtype])
    pos = torch.arange(B, dtype=torch.int32, device="cuda") * 2 % 31
    lens = m - torch.arange(B, dtype=torch.int32, device="cuda") * 13
    plsh.q4_cache_write(a, k, v, pos, lens)
    for i in range(0, m, 10):
        plsh.q4_cache_write(b, k[:, :, i:i + 10].contiguous(), v[:, :, i:i + 10].contiguous(),
                            pos + i, (lens - i).clamp(-1, 10))
    plsh.stream_status()
    assert torch.equal(a.data, b.data)
