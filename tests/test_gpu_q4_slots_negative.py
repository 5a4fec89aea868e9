"""Slots of rows that begin before position 0 are where the same call of a write puts
them; an idle sequence is one without rows."""
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from test_gpu_q4_pages import Pages, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


@pytest.mark.parametrize("pos,lens", [([-2, -1, -7], [5, 1, 6]), ([-1, -1, 3], [0, 4, 2])])
def test_slots_of_rows_before_the_first_position(pos, lens):
    t = Pages(3, 5, 16, 11)
    t.step([20, 20, 20])
    m = 6
    slots = plsh.q4_cache_slots(t.cache, i32(pos), i32(lens), m=m).tolist()
    plsh.stream_status()
    k = torch.arange(1, 3 * m + 1, device="cuda", dtype=torch.float32).view(3, 1, m, 1).expand(3, 1, m, 64).contiguous()
    t.cache.data.zero_()
    plsh.q4_cache_write(t.cache, k, k, i32(pos), i32(lens))
    with pytest.raises(plsh.PlshError):              # (rows before position 0 are reported by a write)
        plsh.stream_status()
    # every page as a sequence of its own
    pages = plsh.Q4Cache(t.cache.data, i32([[p] for p in range(11)]), 1, 64, 16)
    held, _ = plsh.q4_cache_read(pages, i32([0] * 11), m=16, dtype=torch.float32)
    held = held[:, 0, :, 0].flatten().tolist()
    want = [0.0] * len(held)
    for b in range(3):
        for i in range(m):
            there = i < lens[b] and pos[b] + i >= 0
            assert (slots[b][i] >= 0) == there
            if there:
                want[slots[b][i]] = float(b * m + i + 1)
    assert held == want
    plsh.stream_status()
