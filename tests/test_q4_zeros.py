"""Zeros of both signs in a group of the 4-bit cache: -0 counts as less than
+0, so that the stored bytes do not hang on the order of the values."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4


def groups():
    """Groups of 32: zeros of both signs in many orders, some with larger values."""
    rng = np.random.default_rng(4)
    x = np.where(rng.random((64, 32)) < 0.5, np.float32(-0.0), np.float32(0.0))
    x[:8], x[8:16] = -0.0, 0.0
    x[16:24, 0], x[24:32, 31] = -0.0, -0.0
    x[16:24, 1:], x[24:32, :31] = 0.0, 0.0
    x[40:, ::5] = rng.random((24, 7)) * 3
    return x


def test_the_oracle_takes_the_lesser_zero():
    x = groups()
    for order in (slice(None), slice(None, None, -1)):
        c, lo, step = q4.quantise(x[:, order])
        for g, low in zip(x, lo[:, 0]):
            assert low == 0 and np.signbit(low) == (np.signbit(g) & (g == 0)).any()
        assert not np.signbit(step).any()
        assert (c[:40] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows", [16, 7])
def test_stored_bytes(dtype, rows):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    x = torch.from_numpy(groups().reshape(1, 1, 16, 128)).to(dtype)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cache = plsh.Q4Cache(torch.zeros(20 * 128, dtype=torch.uint8, device="cuda"), table, 1, 128, 16)
    d = x[:, :, :rows].contiguous().cuda()
    plsh.q4_cache_write(cache, d, d.flip(3).contiguous(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    plsh.stream_status()
    want = np.zeros(20 * 128, np.uint8)
    v = x.float().numpy()[0, 0]
    for r in range(rows):
        q4.write_row(want, r, v[r], v[r, ::-1])
    np.testing.assert_array_equal(cache.data.cpu().numpy(), want)
