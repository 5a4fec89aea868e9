"""4-bit paged cache without a GPU: the oracle's format and quantiser against
their statements, and the refusals of every entry point (validated before any
CUDA call)."""
import ctypes

import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4


@pytest.fixture(scope="module")
def lib():
    plsh.build()
    return plsh.load()


@pytest.mark.parametrize("d", [64, 128])
def test_every_byte_of_a_tile_is_used_once(d):
    use = np.zeros(20 * d, dtype=int)
    for r in range(16):
        for value in (False, True):
            for e in range(0, d, 2):
                use[q4.code_byte(d, r, e, value)] += 1
                assert q4.code_byte(d, r, e, value) == q4.code_byte(d, r, e + 1, value)
            for y in range(d // 32):
                use[q4.pair_byte(d, r, y, value):][:4] += 1
    assert (use == 1).all()


@pytest.mark.parametrize("scale", [1e-38, 1e-3, 1.0, 1e4, 1e30])
@pytest.mark.parametrize("shift", [0.0, 1.0, -50.0])
def test_quantiser_holds_its_bound(scale, shift):
    """Every value is within half a step (and the fp32 roundings of x - lo and
    of the quotient, 15 steps wide at most) of what it reads back as, and the
    extremes stay inside the codes."""
    rng = np.random.default_rng(3)
    x = ((rng.standard_normal((200, 128)) + shift) * scale).astype(np.float32)
    c, lo, step = q4.quantise(x)
    lo, step = np.repeat(lo, 32, -1).astype(np.float64), np.repeat(step, 32, -1).astype(np.float64)
    assert c.max() <= 15
    assert (lo <= x).all()
    off = np.abs(lo + step * c - x)
    assert (off <= step * (0.5 + 15 * 2.0 ** -22) + 2.0 ** -149).all()
    # both bf16 values
    for v in (lo, step):
        assert (v.astype(np.float32).view(np.uint32) & 0xFFFF == 0).all()


def test_quantiser_ties_go_to_even_and_constants_are_exact():
    x = np.zeros((1, 32), np.float32)
    x[0, :4] = [0.0, 15.0, 2.5, 3.5]           # lo 0, step 1
    c, lo, step = q4.quantise(x)
    assert lo[0, 0] == 0 and step[0, 0] == 1
    assert list(c[0, :4]) == [0, 15, 2, 4]
    c, lo, step = q4.quantise(np.full((1, 32), -2.5, np.float32))
    assert step[0, 0] == 0 and lo[0, 0] == -2.5 and (c == 0).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, 3.4e38])
def test_a_group_that_fp32_cannot_span_reads_back_as_nan(bad):
    x = np.ones((1, 64), np.float32)
    x[0, 5] = bad
    x[0, 6] = -3.4e38 if bad == 3.4e38 else 0.0
    tile = np.zeros(20 * 64, np.uint8)
    q4.write_row(tile, 3, x[0], x[0])
    k, v = q4.read_tiles(tile, 64)
    for t in (k, v):
        assert np.isnan(t[3, :32]).all() and (t[3, 32:] == 1).all()


def test_tiles_read_back_what_was_written():
    rng = np.random.default_rng(0)
    tile = np.zeros(20 * 128, np.uint8)
    x = rng.standard_normal((2, 16, 128)).astype(np.float32)
    for r in rng.permutation(16):
        q4.write_row(tile, r, x[0, r], x[1, r])
    for got, x_ in zip(q4.read_tiles(tile, 128), x):
        c, lo, step = q4.quantise(x_)
        want = np.repeat(lo, 32, -1).astype(np.float64) + np.repeat(step, 32, -1).astype(np.float64) * c
        np.testing.assert_array_equal(got, want)


# ------------------------------------------------------------------- refusals
PTR = 4096
T, C = plsh._Tensor, plsh._Q4Cache


def cache(data=PTR, table=PTR, B=2, H=2, pages=8, max_pages=4, page=64, d=128):
    return C(data, table, B, H, pages, max_pages, page, d)


def test_cache_bytes(lib):
    assert plsh.q4_cache_bytes(3, 8, 64, 128) == 3 * 8 * 4 * 2560
    assert plsh.q4_cache_bytes(1, 1, 16, 64) == 1280
    for bad in ((0, 8, 64, 128), (2 ** 31, 8, 64, 128), (3, 0, 64, 128), (3, 8, 48, 128),
                (3, 8, 512, 128), (3, 8, 64, 96)):
        with pytest.raises(plsh.PlshError) as err:
            plsh.q4_cache_bytes(*bad)
        assert err.value.status == plsh.PLSH_ERR_INVALID


BAD_CACHES = [cache(data=0), cache(data=PTR + 8), cache(table=0), cache(table=PTR + 2), cache(B=0),
              cache(B=65536), cache(H=0), cache(pages=0), cache(max_pages=0), cache(max_pages=2 ** 25),
              cache(page=24), cache(d=96), None]


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_bad_caches_are_refused(lib, i):
    c = BAD_CACHES[i]
    ref = ctypes.byref(c) if c is not None else None
    B, H, d = (c.B, c.H, c.d) if c is not None else (2, 2, 128)
    k = T(PTR, plsh.PLSH_BF16, B, H, 5, d)
    q = T(PTR, plsh.PLSH_BF16, B, H, 1, d)
    sig = np.ones(4)
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    r = ctypes.byref
    out = ctypes.c_int64()
    calls = [lib.plsh_q4_cache_write(r(k), r(k), ref, PTR, None, None),
             lib.plsh_q4_cache_read(ref, PTR, None, r(k), r(k), None),
             lib.plsh_q4_decode_work_bytes(r(q), ref, r(out))]
    if 1 <= H <= 4:
        calls.append(lib.plsh_alibi_exact_decode_q4(r(q), ref, sp, PTR, r(q), PTR, 1 << 40, None))
    assert all(st == plsh.PLSH_ERR_INVALID for st in calls)
    assert lib.plsh_last_error()


@pytest.mark.parametrize("K,V,pos,len_", [
    (T(PTR, 1, 2, 2, 5, 128), T(PTR, 0, 2, 2, 5, 128), PTR, None),       # dtypes differ
    (T(PTR, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 6, 128), PTR, None),       # shapes differ
    (T(PTR, 1, 3, 2, 5, 128), T(PTR, 1, 3, 2, 5, 128), PTR, None),       # B
    (T(PTR, 1, 2, 4, 5, 128), T(PTR, 1, 2, 4, 5, 128), PTR, None),       # H
    (T(PTR, 1, 2, 2, 5, 64), T(PTR, 1, 2, 2, 5, 64), PTR, None),         # d
    (T(PTR, 1, 2, 2, 0, 128), T(PTR, 1, 2, 2, 0, 128), PTR, None),       # no rows
    (T(PTR, 7, 2, 2, 5, 128), T(PTR, 7, 2, 2, 5, 128), PTR, None),       # no such dtype
    (T(PTR + 4, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 5, 128), PTR, None),   # alignment
    (T(0, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 5, 128), PTR, None),
    (T(PTR, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 5, 128), None, None),      # no positions
    (T(PTR, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 5, 128), PTR + 1, None),
    (T(PTR, 1, 2, 2, 5, 128), T(PTR, 1, 2, 2, 5, 128), PTR, PTR + 2),
])
def test_bad_rows_are_refused(lib, K, V, pos, len_):
    r = ctypes.byref
    c = cache()
    assert lib.plsh_q4_cache_write(r(K), r(V), r(c), pos, len_, None) == plsh.PLSH_ERR_INVALID
    assert lib.plsh_q4_cache_read(r(c), pos, len_, r(K), r(V), None) == plsh.PLSH_ERR_INVALID


def test_more_rows_than_a_launch_holds_are_refused(lib):
    c = cache(B=65535, H=65535, d=128)
    k = T(PTR, 1, 65535, 65535, 2 ** 31 - 1, 128)
    r = ctypes.byref
    assert lib.plsh_q4_cache_write(r(k), r(k), r(c), PTR, None, None) == plsh.PLSH_ERR_UNSUPPORTED


def test_bad_queries_are_refused(lib):
    r = ctypes.byref
    c = cache()
    good = T(PTR, 1, 2, 4, 1, 128)
    sig = np.ones(1024)
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))

    def call(q=good, o=good, pos=PTR, sigma=sp):
        return lib.plsh_alibi_exact_decode_q4(r(q), r(c), sigma, pos, r(o), PTR, 1 << 40, None)
    for q in (T(PTR, 1, 2, 4, 2, 128), T(PTR, 1, 1, 4, 1, 128), T(PTR, 1, 2, 3, 1, 128),
              T(PTR, 1, 2, 4, 1, 64), T(PTR + 2, 1, 2, 4, 1, 128)):
        assert call(q=q, o=q) == plsh.PLSH_ERR_INVALID
    assert call(o=T(PTR, 0, 2, 4, 1, 128)) == plsh.PLSH_ERR_INVALID
    assert call(o=T(PTR, 1, 2, 2, 1, 128)) == plsh.PLSH_ERR_INVALID
    assert call(pos=None) == plsh.PLSH_ERR_INVALID
    assert call(pos=PTR + 2) == plsh.PLSH_ERR_INVALID
    assert call(sigma=None) == plsh.PLSH_ERR_INVALID
    zero = np.zeros(4)
    assert call(sigma=zero.ctypes.data_as(ctypes.POINTER(ctypes.c_double))) == plsh.PLSH_ERR_INVALID
    many = T(PTR, 1, 2, 514, 1, 128)
    assert call(q=many, o=many) == plsh.PLSH_ERR_UNSUPPORTED
    huge = T(PTR, 1, 2, 2 ** 62, 1, 128)
    out = ctypes.c_int64()
    assert lib.plsh_q4_decode_work_bytes(r(huge), r(c), r(out)) == plsh.PLSH_ERR_UNSUPPORTED
    assert lib.plsh_q4_decode_work_bytes(r(good), r(c), None) == plsh.PLSH_ERR_INVALID
    assert lib.plsh_alibi_decode_q4(r(good), r(c), None, PTR, r(good), PTR, 1 << 40, None) \
        == plsh.PLSH_ERR_INVALID                                       # bins NULL


def test_outputs_that_overlap_are_refused(lib):
    r = ctypes.byref
    c = cache()
    sig = np.ones(4)
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    base = 1 << 20
    k = T(base, 1, 2, 2, 5, 128)
    q = T(base, 1, 2, 4, 1, 128)
    rows, row = 2 * 2 * 5 * 128 * 2, 2 * 4 * 128 * 2
    for off in (0, 16, rows - 16, 16 - rows):
        v = T(base + off, 1, 2, 2, 5, 128)
        assert lib.plsh_q4_cache_read(r(c), PTR, None, r(k), r(v), None) == plsh.PLSH_ERR_INVALID
        assert b"overlap" in lib.plsh_last_error()
    for off in (0, 16, row - 16, 16 - row):
        o = T(base + off, 1, 2, 4, 1, 128)
        assert lib.plsh_alibi_exact_decode_q4(r(q), r(c), sp, PTR, r(o), PTR, 1 << 40, None) \
            == plsh.PLSH_ERR_INVALID
        assert b"overlap" in lib.plsh_last_error()


def test_binding_refuses_host_tensors():
    data = torch.zeros(plsh.q4_cache_bytes(2, 1, 16, 64), dtype=torch.uint8)
    table = torch.zeros(1, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        plsh.Q4Cache(data, table, 1, 64, 16)                           # not on a GPU
    with pytest.raises(ValueError):
        plsh.Q4Cache(data[:-1], table, 1, 64, 16)                      # not whole pages
    with pytest.raises(ValueError):
        plsh.Q4Cache(data, table.long(), 1, 64, 16)
    with pytest.raises(ValueError):
        plsh.Q4Cache(data.float(), table, 1, 64, 16)
