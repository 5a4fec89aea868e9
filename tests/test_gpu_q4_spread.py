"""Values of V of very different sizes over the 4-bit cache: a large group of one
position takes nothing from other columns, nor from other positions than the ones
beside it, on either kernel of the steps of several rows and behind a prefix.

Every group of 32 columns is held to its own size.  Its relative 2-norm error over
all rows is below 2.5e-3 (as derived in test_gpu_q4_chunk.py: the output's rounding
1.7e-3, at most 2.26e-3; K's, P's and V's roundings to f16 add 1e-4).  The columns that
one value rules have an error of one sign where that value and its weight have: 2^-8
of the output's rounding at most, 2^-11 each of V, of P and (twice) of K's scores.
"""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4
from test_gpu_q4_chunk import Rows, Shared
from test_gpu_q4_decode import i32

pytestmark = pytest.mark.gpu

RULED = 2.0 ** -8 + 4 * 2.0 ** -11


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def rows_of(q, K, V, sigma, pos):
    """fp64, all rows at once: q [Hq, m, d], row i at pos + i; K, V [H, n, d]."""
    Hq, m, d = q.shape
    G, n = Hq // K.shape[0], K.shape[1]
    p = pos + np.arange(m)[:, None]
    j = np.arange(n)[None]
    out = np.empty((Hq, m, d))
    for h in range(Hq):
        x = q[h] @ K[h // G].T / np.sqrt(d) - (p - j) / sigma[h]
        x = np.where(j <= p, x, -np.inf)
        w = np.exp(x - x.max(1, keepdims=True))
        out[h] = w @ V[h // G] / w.sum(1, keepdims=True)
    return out


def check(got, want, ruled=()):
    """[..., d]: each group of 32 columns against its own norm."""
    for y in range(want.shape[-1] // 32):
        a, b = got[..., 32 * y:32 * y + 32], want[..., 32 * y:32 * y + 32]
        off = np.linalg.norm(a - b) / np.linalg.norm(b)
        assert off < (RULED if y in ruled else 2.5e-3), (y, off)


def chunk(s, sigma, pos, which=(0,)):
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, sigma, i32([pos] * s.B)).double().cpu().numpy()
    plsh.stream_status()
    data, out = s.host(), []
    for b in which:
        K, V = q4.read_sequence(data, s.table[b], s.page, s.d, pos + s.m)
        out.append((got[b], rows_of(s.q[b].double().cpu().numpy(), K, V, sigma, pos)))
    return out


POWERS = [0, 16, 20, 24, 29]


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("at", [150, 300, 545])      # older steps, and the newest
@pytest.mark.parametrize("B,wide", [(1, True), (300, True), (1, False)])
def test_one_group_of_one_position(B, wide, at, power):
    """B = 300: all steps of a sequence in one piece.  Not wide: the decode step's kernel."""
    s = Rows(B, 4, 1, 128, 64, 600, "bf16", 32, wide=wide, seed=9)
    s.v[:, :, at, 32:64] *= 2.0 ** power
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * B))
    for sigma in (np.full(4, 1e6), np.full(4, 80.0)):
        for got, want in chunk(s, sigma, 568, (0, B - 1)):
            check(got, want, (1,) if power else ())


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("d,groups", [(64, (0,)), (64, (0, 1)), (128, (3,)), (128, (0, 1, 2, 3))])
def test_groups_of_several_positions(d, groups, power):
    """In three steps, and so that what is large comes, goes and comes again."""
    s = Rows(300, 4, 1, d, 32, 900, "bf16", 20, seed=3)
    for at in (40, 500, 520, 870):
        for y in groups:
            s.v[:, :, at, 32 * y:32 * y + 32] *= 2.0 ** power
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * 300))
    for got, want in chunk(s, np.full(4, 1e6), 880, (0, 299)):
        check(got, want, groups if power else ())


@pytest.mark.parametrize("power", [16, 29, 60, 70])
@pytest.mark.parametrize("B", [1, 300])
def test_whole_positions_far_apart(B, power):
    """Steps whose values differ by a factor each: rows rule, whatever their order."""
    for sign in (1, -1):
        s = Rows(B, 4, 1, 128, 64, 640, "bf16", 32, seed=4)
        for i in range(5):
            s.v[:, :, 128 * i:128 * (i + 1)] *= 2.0 ** (sign * power * (i - 2) / 2)
        plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * B))
        # rows of the newest step alone, and of all
        for sigma in (np.full(4, 0.5), np.full(4, 1e6)):
            for got, want in chunk(s, sigma, 600, (0, B - 1)):
                check(got, want)


@pytest.mark.parametrize("power", [16, 20, 22])
@pytest.mark.parametrize("lean", [-4, 0, 4])
@pytest.mark.parametrize("B,wide", [(1, True), (300, True), (1, False)])
def test_large_values_of_small_weights(B, wide, lean, power):
    """A position so far back that its weight and its group's size make up for one
    another (to 2^lean): the weight, 2^-power and less of the row's largest, counts.
    It is held to 2^-33 of that largest: 2^(power - 33), less than 2^-11, of the group's."""
    s = Rows(B, 4, 1, 128, 64, 600, "bf16", 32, wide=wide, seed=9)
    at, pos = 150, 568
    s.v[:, :, at, 32:64] *= 2.0 ** power
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * B))
    sigma = np.full(4, (pos - at) / ((power - lean) * np.log(2)))
    for got, want in chunk(s, sigma, pos, (0, B - 1)):
        check(got, want, (1,))


@pytest.mark.parametrize("power", [16, 20, 24])
@pytest.mark.parametrize("wide", [True, False])
def test_a_later_token_takes_nothing_from_an_earlier_one(wide, power):
    """Rows before a new token whose group is large, of its step but not its 32 positions."""
    s = Rows(1, 4, 1, 128, 64, 640, "bf16", 64, wide=wide, seed=6)
    s.v[:, :, 610, 64:96] *= 2.0 ** power
    plsh.q4_cache_write(s.cache, s.k, s.v, i32([0]))
    for sigma in (np.full(4, 1e6), np.full(4, 3.0)):
        (got, want), = chunk(s, sigma, 576)
        check(got[:, :32], want[:, :32])                     # positions 576 .. 607
        check(got[:, 34:], want[:, 34:], (2,))


@pytest.mark.parametrize("power", POWERS)
@pytest.mark.parametrize("B,shared", [(64, 390), (5, 12)])     # tensor cores; the decode step's kernel
def test_one_group_of_a_shared_position(B, shared, power):
    s = Shared(B, 4, 1, 128, 64, shared, 64, "bf16", seed=4)
    P = s.P
    pos = [P + b for b in range(B)]
    for at in (100, P // 2 + 3, P - 20):
        k, v = (torch.randn(1, 1, 1, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(at)) for _ in range(2))
        v[..., 96:] *= 2.0 ** power
        plsh.q4_cache_write(plsh.Q4Cache(s.cache.data, i32(s.prefix[None]), 1, 128, 64), k, v, i32([at]))
    sigma = np.full(4, 1e6)
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, sigma, i32(pos), s.d_prefix).double().cpu().numpy()
    plsh.stream_status()
    data = s.host()
    Kp, Vp = q4.read_sequence(data, s.prefix, s.page, s.d, P)
    a, b = [], []
    for i in range(B):
        K, V = q4.read_sequence(data, s.table[i, shared:], s.page, s.d, pos[i] + 1 - P)
        a.append(got[i])
        b.append(rows_of(s.q[i].double().cpu().numpy(), np.concatenate([Kp, K], 1), np.concatenate([Vp, V], 1),
                         sigma, pos[i]))
    check(np.stack(a), np.stack(b), (3,) if power else ())


@pytest.mark.parametrize("B", [1, 300])
def test_what_cannot_be_held_is_refused_however_the_list_is_cut(B):
    """A group 2^33 above and more what other 32 positions of its step hold; below, the
    rows are right."""
    for power, wrong in ((29, False), (36, True), (80, True)):
        s = Rows(B, 4, 1, 128, 64, 600, "bf16", 32, seed=9)
        s.v[:, :, 300, 32:64] *= 2.0 ** power
        plsh.q4_cache_write(s.cache, s.k, s.v, i32([0] * B))
        if not wrong:
            for sigma in (np.full(4, 50.0), np.full(4, 1e6)):
                for got, want in chunk(s, sigma, 568, (0, B - 1)):
                    check(got, want, (1,))
            continue
        plsh.alibi_exact_chunk_q4(s.q, s.cache, np.full(4, 50.0), i32([568] * B))
        with pytest.raises(plsh.PlshError) as e:
            plsh.stream_status()
        assert e.value.status == plsh.PLSH_ERR_RANGE


@pytest.mark.parametrize("sigma", [0.05, 1e-4, 2e-6, 1.4e-6, 1e-6, 1e-8, 1e-9, 1e-35, 1e-300])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,wide", [(1, True), (300, True), (1, False)])
def test_slopes_so_steep_that_a_row_is_its_own_value(B, wide, d, sigma):
    """Rows at every alignment: o is v at the row's own position, but for its rounding
    and those of V and of the one weight."""
    s = Rows(B, 4, 1, d, 64, 400, "bf16", 150, wide=wide, seed=12)
    pos = 217
    got = plsh.alibi_exact_chunk_q4(s.q, s.cache, np.full(4, sigma), i32([pos] * B)).double().cpu().numpy()
    plsh.stream_status()
    for b in {0, B - 1}:
        _, V = q4.read_sequence(s.host(), s.table[b], s.page, d, pos + 150)
        want = V[:, pos:]
        lost = np.abs(V).max() * 2.0 ** -18              # f16's step beside a step's largest value
        assert (np.abs(got[b] - want) <= np.abs(want) * (2.0 ** -8 + 2 * 2.0 ** -11) + lost).all()


@pytest.mark.parametrize("sigma", [2e-6, 1e-8, 1e-35])
def test_steep_slopes_behind_a_prefix(sigma):
    s = Shared(64, 4, 1, 128, 64, 390, 64, "bf16", seed=4)
    pos = [s.P - 64 + 2 * b for b in range(64)]              # within, at its end and behind
    got = plsh.alibi_exact_prefix_decode_q4(s.q, s.cache, np.full(4, sigma), i32(pos), s.d_prefix).double().cpu().numpy()
    plsh.stream_status()
    data = s.host()
    _, Vp = q4.read_sequence(data, s.prefix, s.page, s.d, s.P)
    for b in range(64):
        _, V = q4.read_sequence(data, s.table[b, 390:], s.page, s.d, 64)
        want = Vp[:, pos[b]] if pos[b] < s.P else V[:, pos[b] - s.P]
        lost = np.abs(Vp).max() * 2.0 ** -18
        assert (np.abs(got[b, :, 0] - want) <= np.abs(want) * (2.0 ** -8 + 2 * 2.0 ** -11) + lost).all(), b
