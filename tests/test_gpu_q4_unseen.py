"""What no row sees has no effect on any: behind a shared prefix whose end no sequence
has come to (pages not yet written, or not yet there), on either kernel."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from test_gpu_q4_chunk import Shared
from test_gpu_q4_decode import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


SIZES = [(64, 390, 64, "bf16"), (128, 1040, 16, "bf16"), (5, 12, 64, "bf16"), (5, 12, 64, "f32")]


def within(B, shared, page, dtype):
    s = Shared(B, 4, 1, 128, page, shared, 20, dtype, seed=7)
    half = shared // 2
    pos = [max(0, (half * page) - 1 - 11 * b) if b % 9 else -1 for b in range(B)]      # the largest: b = 1
    last = max(pos)
    return s, pos, last


@pytest.mark.parametrize("B,shared,page,dtype", SIZES)
@pytest.mark.parametrize("sigma", [50.0, 1e6])
def test_pages_of_a_prefix_that_nobody_has_come_to(B, shared, page, dtype, sigma):
    s, pos, last = within(B, shared, page, dtype)
    sig = np.full(4, sigma)
    want = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(pos), s.d_prefix)
    plsh.stream_status()
    s.check(want, pos, sig)
    first = last // page + 1                         # the first page that no row needs
    unseen = s.d_prefix[first:].long()
    for fill in (0, 127, 255, 0x7e, 0x44):           # (0x7e7e, as bf16: 8e37)
        s.cache.data.view(s.cache.pages, -1)[unseen] = fill
        got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(pos), s.d_prefix)
        plsh.stream_status()
        assert torch.equal(got, want), fill
    for bad in (-1, s.cache.pages, -2 ** 31):        # not there at all
        prefix = s.d_prefix.clone()
        prefix[first:] = bad
        assert torch.equal(plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(pos), prefix), want)
        plsh.stream_status()


@pytest.mark.parametrize("B,shared,page,dtype", SIZES)
def test_positions_of_a_page_that_nobody_has_come_to(B, shared, page, dtype):
    s, pos, last = within(B, shared, page, dtype)
    pos = [p if p < 0 else max(0, p - 37 * (p > 40)) for p in pos]
    last = max(pos)
    sig = np.full(4, 1e6)
    want = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(pos), s.d_prefix)
    one = plsh.Q4Cache(s.cache.data, i32(s.prefix[None]), 1, 128, page)
    n = min(60, s.P - last - 1)
    for value in (1e25, -3e38, float("inf"), float("nan")):
        k, v = torch.full((2, 1, 1, n, 128), value, device="cuda")
        v[..., ::7] = 0.5
        plsh.q4_cache_write(one, k, v, i32([last + 1]))
        got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(pos), s.d_prefix)
        plsh.stream_status()
        assert torch.equal(got, want), value
    # all idle, or out of range but for one: nothing is seen of what lies behind that one
    far = [-1] * (B - 1) + [5]
    want = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32(far), s.d_prefix)
    plsh.stream_status()
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sig, i32([10 ** 9] * (B - 1) + [5]), s.d_prefix)
    with pytest.raises(plsh.PlshError) as e:
        plsh.stream_status()
    assert e.value.status == plsh.PLSH_ERR_INVALID
    assert torch.equal(got, want) and (got[:-1] == 0).all() and torch.isfinite(got[-1]).all()
