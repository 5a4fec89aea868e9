"""Refusals of the 4-bit cache's steps of several rows a sequence, and of a batch
behind a shared prefix, each told apart by its message (the tensors of a call lie
apart: only the fault in question is there to refuse)."""
import ctypes

import numpy as np
import pytest

import positional_lsh_approximation_gb300 as plsh
from test_q4_refusals_cpu import AT, BAD_CACHES, F32, cache, r, refused, ten

AT = {**AT, "prefix": 1 << 40}
ROWS = "plsh_alibi_exact_chunk_q4"
SHARED = "plsh_alibi_exact_prefix_decode_q4"


@pytest.fixture(scope="module")
def lib():
    plsh.build()
    return plsh.load()


def call(lib, name, q, o, c, pos=AT["pos"], len=None, sigma=(1, 1, 1, 1), prefix=AT["prefix"], pages=2,
         work=AT["work"], size=1 << 40):
    s = None if sigma is None else np.asarray(sigma, np.float64)
    sp = None if s is None else s.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    p = [x if x is None else r(x) for x in (q, c, o)]
    if name == ROWS:
        return lib.plsh_alibi_exact_chunk_q4(p[0], p[1], sp, pos, len, p[2], work, size, None)
    return lib.plsh_alibi_exact_prefix_decode_q4(p[0], p[1], sp, pos, prefix, pages, p[2], work, size, None)


def both(m=5):
    return [(ROWS, ten("q", 2, 4, m, 128), ten("o", 2, 4, m, 128)),
            (SHARED, ten("q", 2, 4, 1, 128), ten("o", 2, 4, 1, 128))]


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_each_fault_of_a_cache(lib, i):
    kw, word = BAD_CACHES[i]
    c, out = cache(**kw), ctypes.c_int64()
    for name, q, o in both():
        refused(lib, call(lib, name, q, o, c, pages=1), plsh.PLSH_ERR_INVALID,
                word if kw.get("max_pages") != 0 or name == ROWS else "prefix_pages must be")
    q1 = ten("q", 2, 4, 1, 128)
    for st in (lambda: lib.plsh_q4_chunk_work_bytes(r(both()[0][1]), r(c), r(out)),
               lambda: lib.plsh_q4_prefix_work_bytes(r(q1), r(c), r(out))):
        refused(lib, st(), plsh.PLSH_ERR_INVALID, word)


def test_no_cache_no_tensors_no_bytes(lib):
    out = ctypes.c_int64()
    for name, q, o in both():
        refused(lib, call(lib, name, q, o, None), plsh.PLSH_ERR_INVALID, "cache is NULL")
        refused(lib, call(lib, name, None, o, cache()), plsh.PLSH_ERR_INVALID, "q")
        refused(lib, call(lib, name, q, None, cache()), plsh.PLSH_ERR_INVALID, "o")
    q = ten("q", 2, 4, 1, 128)
    for f in (lib.plsh_q4_chunk_work_bytes, lib.plsh_q4_prefix_work_bytes):
        refused(lib, f(r(q), None, r(out)), plsh.PLSH_ERR_INVALID, "cache is NULL")
        refused(lib, f(None, r(cache()), r(out)), plsh.PLSH_ERR_INVALID, "q")
        refused(lib, f(r(q), r(cache()), None), plsh.PLSH_ERR_INVALID, "bytes is NULL")


# (entry points, q's shape, o's, arguments, words)
BAD = [
    ((SHARED,), (2, 4, 2, 128), (2, 4, 2, 128), {}, "q must be [B, Hq, 1, d]"),
    ((ROWS,), (2, 4, 0, 128), (2, 4, 0, 128), {}, "q: every dimension"),
    ((ROWS, SHARED), (1, 4, 1, 128), (1, 4, 1, 128), {}, "q must have the cache's B and d"),
    ((ROWS, SHARED), (2, 4, 1, 64), (2, 4, 1, 64), {}, "q must have the cache's B and d"),
    ((ROWS, SHARED), (2, 3, 1, 128), (2, 3, 1, 128), {}, "multiple of the cache's H"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 2, 1, 128), {}, "o must have q's shape and dtype"),
    ((ROWS,), (2, 4, 3, 128), (2, 4, 4, 128), {}, "o must have q's shape and dtype"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 4, 1, 128), dict(pos=None), "pos and len must be"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 4, 1, 128), dict(pos=AT["pos"] + 2), "pos and len must be"),
    ((ROWS,), (2, 4, 3, 128), (2, 4, 3, 128), dict(len=AT["len"] + 1), "pos and len must be"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 4, 1, 128), dict(sigma=None), "sigma_h is NULL"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 4, 1, 128), dict(sigma=[1, 0, 1, 1]), "sigma_h[1]"),
    ((ROWS, SHARED), (2, 4, 1, 128), (2, 4, 1, 128), dict(sigma=[1, 1, 1, np.nan]), "sigma_h[3]"),
    ((SHARED,), (2, 4, 1, 128), (2, 4, 1, 128), dict(prefix=None), "prefix must be"),
    ((SHARED,), (2, 4, 1, 128), (2, 4, 1, 128), dict(prefix=AT["prefix"] + 2), "prefix must be"),
    ((SHARED,), (2, 4, 1, 128), (2, 4, 1, 128), dict(pages=0), "prefix_pages must be"),
    ((SHARED,), (2, 4, 1, 128), (2, 4, 1, 128), dict(pages=-1), "prefix_pages must be"),
    ((SHARED,), (2, 4, 1, 128), (2, 4, 1, 128), dict(pages=5), "prefix_pages must be"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_each_fault_of_a_call(lib, i):
    names, qs, os, kw, word = BAD[i]
    for name in names:
        refused(lib, call(lib, name, ten("q", *qs), ten("o", *os), cache(), **kw), plsh.PLSH_ERR_INVALID, word)


@pytest.mark.parametrize("kw,word", [
    (dict(q=dict(off=2)), "q->data must be 16-byte aligned"), (dict(o=dict(off=8)), "o->data must be 16-byte aligned"),
    (dict(q=dict(off=-AT["q"])), "q->data is NULL"), (dict(o=dict(off=-AT["o"])), "o->data is NULL"),
    (dict(q=dict(dtype=5)), "q: dtype"), (dict(o=dict(dtype=F32)), "o must have q's shape and dtype"),
    (dict(o=dict(off=AT["q"] - AT["o"] + 256)), "must not overlap"),
])
def test_each_fault_of_a_tensor(lib, kw, word):
    for name, m in ((ROWS, 3), (SHARED, 1)):
        q, o = ten("q", 2, 4, m, 128, **kw.get("q", {})), ten("o", 2, 4, m, 128, **kw.get("o", {}))
        refused(lib, call(lib, name, q, o, cache()), plsh.PLSH_ERR_INVALID, word)


def test_more_heads_and_rows_than_are_served(lib):
    sig = np.ones(1024)
    for name, m in ((ROWS, 2), (SHARED, 1)):
        refused(lib, call(lib, name, ten("q", 2, 1024, m, 128), ten("o", 2, 1024, m, 128), cache(), sigma=sig),
                plsh.PLSH_ERR_UNSUPPORTED, "512 heads")
    m = 1 << 28                                          # 2 x 4 x 2^28 rows
    st = call(lib, ROWS, ten("q", 2, 4, m, 128), ten("o", 2, 4, m, 128), cache())
    assert st != plsh.PLSH_OK and "2^30" in lib.plsh_last_error().decode()
