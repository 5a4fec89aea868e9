"""A key or value that is no number at every offset of the rows that share a pass of
the decode step's kernel (as many tokens as eight columns hold), and on the tensor
cores: the rows before it are as they were, bit for bit, the others tell of it."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from test_gpu_q4_chunk import Rows, poison
from test_gpu_q4_decode import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("dtype,wide", [("bf16", False), ("f32", False), ("bf16", True)])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5])       # eight, four, two, two tokens a pass, and one
@pytest.mark.parametrize("first", [299, 308])        # the rows' first position; blocks of 32 end inside
def test_rows_before_it_are_as_they_were(first, G, dtype, wide, which):
    m, d = 17, 128
    s = Rows(2, G, 1, d, 64, 400, dtype, m, wide=wide, seed=2)
    sigma, pos = np.full(G, 40.0), [first, 360]
    want = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos))
    for off in range(m):
        poison(s, 0, first + off, which)
        got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos))
        plsh.stream_status()
        assert torch.equal(got[1], want[1])
        assert torch.equal(got[0, :, :off], want[0, :, :off]), off
        seen = torch.isnan(got[0, :, off:])
        if which == "k":
            assert seen.all(), off
        else:                                        # a value's group: 32 .. 63
            assert seen[..., 32:64].all() and not seen[..., :32].any() and not seen[..., 64:].any(), off
        # as it was
        table = torch.from_numpy(s.table[:1].copy()).cuda()
        one = plsh.Q4Cache(s.cache.data, table, s.H, s.d, s.page)
        at = slice(first + off, first + off + 1)
        plsh.q4_cache_write(one, s.k[:1, :, at].contiguous(), s.v[:1, :, at].contiguous(), i32([first + off]))
    assert torch.equal(plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32(pos)), want)
