"""Row counts near the limits of the steps of several rows."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from test_gpu_q4_decode import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def test_an_idle_sequence_of_2_27_rows():
    """Its rows are 0, all 34 GB of them: 2^31 stores of 16 bytes.  (Its queries are
    not read: two rows of them overlap nothing, but the tensor has to be there.)"""
    m, d = 2 ** 27, 128
    if torch.cuda.mem_get_info()[0] < 80 * 2 ** 30:
        pytest.skip("needs 80 GB of device memory")
    q = torch.empty(1, 1, m, d, dtype=torch.bfloat16, device="cuda")
    out = torch.full((1, 1, m, d), 7.0, dtype=torch.bfloat16, device="cuda")
    data = torch.zeros(plsh.q4_cache_bytes(4, 1, 64, d), dtype=torch.uint8, device="cuda")
    cache = plsh.Q4Cache(data, i32([[0, 1, 2, 3]]), 1, d, 64)
    try:
        plsh.alibi_exact_chunk_q4(q, cache, np.ones(1), i32([-1]), out=out)
        plsh.stream_status()
        flat = out.view(-1)
        assert (flat[::2 ** 16] == 0).all() and (flat[-2 ** 16:] == 0).all() and (flat[:2 ** 16] == 0).all()
    finally:
        del q, out
        torch.cuda.empty_cache()
