"""A row whose query is far larger than the others', or far smaller, is a matter of that
row alone: behind a shared prefix the rows of a tile are other requests'.

On the tensor cores other rows are the same, bit for bit.  In the decode step's kernel
the columns of a pass share the decision to move their references, by factors that are
no powers of two: other rows differ by roundings (each side's as derived in
test_gpu_q4_chunk.py), however large the row is."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from positional_lsh_approximation_gb300.inputs import alibi_sigmas
from test_gpu_q4_chunk import Rows, Shared
from test_gpu_q4_decode import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def alike(got, want, dtype, exactly):
    if exactly:
        assert torch.equal(got, want)
    off = ((got.double() - want.double()).norm() / want.double().norm()).item()
    assert off < (2.5e-3 if dtype == "bf16" else 2e-6) * 2 ** 0.5


@pytest.mark.parametrize("power", [10, 40, 100, -40, -100])
@pytest.mark.parametrize("d,wide,dtype", [(64, True, "bf16"), (128, True, "bf16"), (128, False, "bf16"), (128, False, "f32")])
def test_rows_of_a_chunk(power, d, wide, dtype):
    s = Rows(2, 4, 1, d, 64, 500, dtype, 40, wide=wide, seed=2)
    sigma, pos = alibi_sigmas(4), i32([460, 100])
    want = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, pos)
    s.q[0, 2, 9] *= 2.0 ** power
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, pos)
    plsh.stream_status()
    rest = torch.ones(2, 4, 40, dtype=torch.bool)
    rest[0, 2, 9] = False
    alike(got.cpu()[rest], want.cpu()[rest], dtype, wide)
    near = torch.zeros(2, 4, 40, dtype=torch.bool)       # of its head, token, pass
    near[0, 2, 8:11] = near[0, :, 9] = near[0, :, 8] = True
    near[0, 2, 9] = False
    alike(got.cpu()[near], want.cpu()[near], dtype, wide)
    assert torch.isfinite(got).all()
    if power < 0:                                    # no scores to speak of: the bias alone
        flat, *_ = s.want(0, 469, 9, sigma)
        off = np.linalg.norm(got[0, 2, 9].double().cpu().numpy() - flat[2]) / np.linalg.norm(flat[2])
        assert off < 2.0 ** -8 + 4 * 2.0 ** -11


@pytest.mark.parametrize("power", [10, 40, 100, -40, -100])
@pytest.mark.parametrize("B,shared", [(64, 390), (5, 12)])
def test_sequences_behind_a_prefix(power, B, shared):
    s = Shared(B, 4, 1, 128, 64, shared, 64, "bf16", seed=4)
    sigma, pos = np.full(4, 60.0), i32([s.P + b for b in range(B)])
    want = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, pos, s.d_prefix)
    s.q[3] *= 2.0 ** power
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, pos, s.d_prefix)
    plsh.stream_status()
    others = [b for b in range(B) if b != 3]
    alike(got[others], want[others], "bf16", B == 64)
    assert torch.isfinite(got).all()
