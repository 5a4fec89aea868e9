"""Items of one and of two row tiles in turn, many of them in every thread block of
the tensor cores' kernel over the 4-bit cache: whatever follows what, a row is the one
that the decode step gives for its token."""
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


@pytest.mark.parametrize("lens", [(32, 9), (9, 32), (32, 9, 32, 32, 9, 9), (32, 9, 0, 17, 16, 1)],
                         ids=lambda t: "-".join(map(str, t)))
@pytest.mark.parametrize("far", [40, 400])           # items of one step, and of up to four
def test_a_second_tile_after_items_without_one(lens, far):
    B, G, d, page, m, cap = 1500, 8, 128, 64, 32, 8
    g = torch.Generator("cuda").manual_seed(far)
    # (256 rows are two tiles, 72 one; a CTA has about ten items)
    pages = B * cap
    data = torch.zeros(plsh.q4_cache_bytes(pages, 1, page, d), dtype=torch.uint8, device="cuda")
    table = torch.randperm(pages, device="cuda", generator=g).to(torch.int32).view(B, cap)
    cache = plsh.Q4Cache(data, table, 1, d, page)
    k, v = (torch.randn(B, 1, far + m, d, device="cuda", generator=g) for _ in range(2))
    plsh.q4_cache_write(cache, k, v, i32([0] * B))
    q = torch.randn(B, G, m, d, device="cuda", generator=g).bfloat16()
    sigma = alibi_sigmas(G)
    pos = torch.randint(0, far, (B,), device="cuda", generator=g).to(torch.int32)
    count = i32([lens[b % len(lens)] for b in range(B)])
    got = plsh.alibi_exact_chunk_q4(q, cache, sigma, pos, count)
    plsh.stream_status()
    for i in range(m):
        one = plsh.alibi_exact_decode_q4(q[:, :, i:i + 1].contiguous(), cache, sigma, pos + i).double()[:, :, 0]
        seen = (i < count)
        off = (got[:, :, i].double() - one)[seen].norm(dim=-1) / one[seen].norm(dim=-1)
        # two bf16 roundings of 2^-8 at most, and f16's 2^-11 of K (twice, by scores of a few units), P and V
        assert off.numel() == 0 or off.max().item() < 2 * 2.0 ** -8 + 2.0 ** -7, (i, off.max().item())
        assert (got[:, :, i][~seen] == 0).all()
    plsh.stream_status()
    for _ in range(20):
        assert torch.equal(plsh.alibi_exact_chunk_q4(q, cache, sigma, pos, count), got)
    plsh.stream_status()
