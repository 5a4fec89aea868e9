"""Failure detection of the tensor cores' kernel over the 4-bit cache without a GPU
fault: its waits run out, the call is reported, and the next one is right.

PLSH_FAULT=stall: no item is listed, so that every warp but one waits for what nothing
will complete, with nothing in flight.  A limit of a nanosecond: waits that last longer than
the hardware itself suspends a thread at a try (two tries come before the clock is
looked at) give up, wherever the kernel is, with products in flight; the thread blocks
let these end, whatever the limit, before they free their tensor memory.  Which waits
those are is a matter of timing: a call is reported, or right.
"""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from positional_lsh_approximation_gb300.inputs import alibi_sigmas

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def chunk_call(d):
    """Sixteen sequences' chunks, several items a thread block, of one and two tiles."""
    B, H, G, m, page, cap = 16, 8, 4, 160, 64, 32
    g = torch.Generator("cuda").manual_seed(d)
    data = torch.zeros(plsh.q4_cache_bytes(B * cap, H, page, d), dtype=torch.uint8, device="cuda")
    table = torch.randperm(B * cap, device="cuda", generator=g).to(torch.int32).view(B, cap)
    cache = plsh.Q4Cache(data, table, H, d, page)
    k, v = (torch.randn(B, H, cap * page, d, device="cuda", generator=g) for _ in range(2))
    plsh.q4_cache_write(cache, k, v, i32([0] * B))
    q = torch.randn(B, H * G, m, d, device="cuda", generator=g).bfloat16()
    pos = i32([(137 * b) % (cap * page - m) for b in range(B)])
    lens = i32([160 - 9 * b for b in range(B)])
    return lambda: plsh.alibi_exact_chunk_q4(q, cache, alibi_sigmas(H * G), pos, lens)


def prefix_call(d):
    B, H, G, page, shared, cap = 64, 8, 4, 64, 128, 130
    g = torch.Generator("cuda").manual_seed(d)
    pages = shared + 2 * B
    data = torch.zeros(plsh.q4_cache_bytes(pages, H, page, d), dtype=torch.uint8, device="cuda")
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    prefix = order[:shared].contiguous()
    table = torch.cat([prefix.expand(B, -1), order[shared:].view(B, 2)], 1).contiguous()
    assert table.shape[1] == cap
    cache = plsh.Q4Cache(data, table, H, d, page)
    whole = plsh.Q4Cache(data, prefix[None].contiguous(), H, d, page)
    k, v = (torch.randn(1, H, shared * page, d, device="cuda", generator=g) for _ in range(2))
    plsh.q4_cache_write(whole, k, v, i32([0]))
    k, v = (torch.randn(B, H, 2 * page, d, device="cuda", generator=g) for _ in range(2))
    plsh.q4_cache_write(cache, k, v, i32([shared * page] * B))
    q = torch.randn(B, H * G, 1, d, device="cuda", generator=g).bfloat16()
    pos = i32([shared * page + (7 * b) % (2 * page) for b in range(B)])
    return lambda: plsh.alibi_exact_prefix_decode_q4(q, cache, np.full(H * G, 3000.0), pos, prefix)


@pytest.mark.parametrize("call", [chunk_call, prefix_call])
def test_a_stalled_call_is_reported_and_the_next_is_right(call, monkeypatch):
    f = call(128)
    want = f()
    plsh.stream_status()
    plsh.set_wait_limit_ns(1_000_000)          # 1 ms; 64 of these for an item
    try:
        monkeypatch.setenv("PLSH_FAULT", "stall")
        f()
        with pytest.raises(plsh.PlshError) as err:
            plsh.stream_status()
        assert err.value.status == plsh.PLSH_ERR_TIMEOUT
        plsh.stream_status()                   # the report cleared the flag
    finally:
        monkeypatch.delenv("PLSH_FAULT", raising=False)
        plsh.set_wait_limit_ns(0)
    assert torch.equal(f(), want)
    plsh.stream_status()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("call", [chunk_call, prefix_call])
def test_waits_that_give_up_at_once_leave_the_next_call_right(call, d):
    f = call(d)
    want = f()
    plsh.stream_status()
    for _ in range(3):
        plsh.set_wait_limit_ns(1)
        try:
            got = f()
            plsh.stream_status()
            assert torch.equal(got, want)
        except plsh.PlshError as err:
            assert err.status == plsh.PLSH_ERR_TIMEOUT
        finally:
            plsh.set_wait_limit_ns(0)
        assert torch.equal(f(), want)
        plsh.stream_status()


@pytest.mark.parametrize("limit", [2 ** 58, 2 ** 63, 2 ** 64 - 1])
@pytest.mark.parametrize("call", [chunk_call, prefix_call])
def test_a_limit_that_nothing_reaches(call, limit):
    """An item's waits have 64 times a step's limit: of the largest limits, no less."""
    f = call(128)
    want = f()
    plsh.stream_status()
    plsh.set_wait_limit_ns(limit)
    try:
        for _ in range(3):
            got = f()
            plsh.stream_status()
            assert torch.equal(got, want)
    finally:
        plsh.set_wait_limit_ns(0)
