"""The 4-bit cache's calls at the ends of what their interface admits."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def filled(B, H, n, page, pages, d=64, max_pages=None, seed=0):
    """A cache with n random positions of each sequence, and K, V as held."""
    g = torch.Generator("cuda").manual_seed(seed)
    per = -(-n // page)
    table = torch.zeros(B, max_pages or per, dtype=torch.int32, device="cuda")
    table[:, :per] = torch.randperm(pages, device="cuda", generator=g)[:B * per].view(B, per).to(torch.int32)
    cache = plsh.Q4Cache.empty(pages, H, d, table, page)
    k, v = (torch.randn(B, H, n, d, device="cuda", generator=g) for _ in range(2))
    plsh.q4_cache_write(cache, k, v, i32([0] * B))
    K, V = plsh.q4_cache_read(cache, i32([0] * B), m=n, dtype=torch.float32)
    return cache, K.double().cpu().numpy(), V.double().cpu().numpy()


def test_the_most_pages_a_sequence_may_have():
    """max_pages * page = 2^31 - 16: the exact step's plan, which counts the
    blocks a row may have, and both steps' results at small positions."""
    n, Hq, d = 100, 4, 64
    cache, K, V = filled(1, 2, n, 16, 12, max_pages=2 ** 27 - 1)
    assert cache.max_pages * cache.page == 2 ** 31 - 16
    q = torch.randn(1, Hq, 1, d, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    sigma = np.array([3.0, 10.0, 30.0, 90.0])
    bins = plsh.sample_bins(n, sigma, 3, seed=1)
    off, st = bins.to_host()
    for pos in (0, 17, 99):
        e = plsh.alibi_exact_decode_q4(q, cache, sigma, i32([pos]))
        o = plsh.alibi_decode_q4(q, cache, bins, i32([pos]))
        plsh.stream_status()
        for got, lw in ((e, q4.log_weights_exact(sigma, pos, n)),
                        (o, q4.log_weights_approx(off, st, Hq, 3, pos, n))):
            want = q4.decode_row(q[0, :, 0].double().cpu().numpy(), K[0], V[0], lw)
            # scores of size ~ 4 and values of size ~ 4, some 60 fp32 roundings
            # of either: 60 * 2^-24 * 4 * 4 < 6e-5
            assert np.abs(got[0, :, 0].double().cpu().numpy() - want).max() < 6e-5
    bins.free()


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("first", [16, 30, 47, 160, 175])
def test_pages_before_the_bins_may_be_gone(page, first):
    """An approximate row reaches back to its bins' first start: the pages
    before it may have been handed back (an index out of range), and those
    behind the position may not have been given yet; nothing is reported."""
    n, Hq, d, pos = 200, 4, 128, 177
    cache, _, _ = filled(2, 1, n, page, 40, d=d)
    q = torch.randn(2, Hq, 1, d, device="cuda").bfloat16()
    bins = plsh.bins_from_host(n, Hq, 1, np.arange(0, 3 * Hq + 1, 3), np.tile([0, first, n], Hq))
    want = plsh.alibi_decode_q4(q, cache, bins, i32([pos, pos]))
    plsh.stream_status()
    cache.table[:, :first // page] = -1
    cache.table[:, pos // page + 1:] = 10 ** 9
    got = plsh.alibi_decode_q4(q, cache, bins, i32([pos, pos]))
    plsh.stream_status()
    assert torch.equal(got, want)
    # the page that the first start lies in counts
    cache.table[:, first // page] = -1
    plsh.alibi_decode_q4(q, cache, bins, i32([pos, pos]))
    with pytest.raises(plsh.PlshError):
        plsh.stream_status()
    bins.free()


STEEP = [1e-30, 1e-37, 1e-39, 1e-45, 1e-300]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scales_whose_slope_fp32_does_not_hold(dtype):
    """Every sigma above 0 is admitted; so steep a bias leaves the key at the
    row's own position alone: o is its value."""
    n, Hq, d = 70, len(STEEP), 64
    cache, _, V = filled(2, 1, n, 32, 8, d=d)
    q = torch.randn(2, Hq, 1, d, device="cuda").to(dtype)
    pos = [69, 32]
    got = plsh.alibi_exact_decode_q4(q, cache, STEEP, i32(pos))
    plsh.stream_status()
    # one rounding of P step to f16 (2^-11 of 15 steps, a span of 8 at most),
    # fp32 sums, the output's 2^-8
    for b in range(2):
        want = np.broadcast_to(V[b, 0, pos[b]], (Hq, d))
        np.testing.assert_allclose(got[b, :, 0].double().cpu().numpy(), want, atol=8 * 2.0 ** -11, rtol=2.0 ** -8)
