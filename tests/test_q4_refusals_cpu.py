"""Refusals of the 4-bit cache's entry points, each told apart by its message:
the tensors of a call lie apart, so that only the fault in question is there to
refuse.  (The status alone would not say which check refused.)"""
import ctypes

import numpy as np
import pytest

import positional_lsh_approximation_gb300 as plsh

T, C = plsh._Tensor, plsh._Q4Cache
AT = {name: (i + 1) << 32 for i, name in enumerate(("data", "table", "q", "o", "K", "V", "pos", "len", "work"))}
r = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    plsh.build()
    return plsh.load()


def cache(data=AT["data"], table=AT["table"], B=2, H=2, pages=8, max_pages=4, page=64, d=128):
    return C(data, table, B, H, pages, max_pages, page, d)


def ten(name, *shape, dtype=plsh.PLSH_BF16, off=0):
    return T(AT[name] + off, dtype, *shape)


def refused(lib, status, code, word):
    assert status == code, lib.plsh_last_error()
    assert word in lib.plsh_last_error().decode()


BAD_CACHES = [
    (dict(data=0), "data must be"), (dict(data=AT["data"] + 8), "data must be"),
    (dict(table=0), "table must be"), (dict(table=AT["table"] + 2), "table must be"),
    (dict(B=0), "B must be"), (dict(B=65536), "B must be"), (dict(H=0), "H must be"), (dict(H=65536), "H must be"),
    (dict(pages=0), "pages must be"), (dict(pages=2 ** 31), "pages must be"),
    (dict(max_pages=0), "max_pages must be"), (dict(max_pages=2 ** 25), "max_pages must be"),
    (dict(page=24), "page must be"), (dict(page=8), "page must be"), (dict(d=96), "d must be 64 or 128"),
]


@pytest.mark.parametrize("i", range(len(BAD_CACHES)))
def test_each_fault_of_a_cache(lib, i):
    kw, word = BAD_CACHES[i]
    c = cache(**kw)
    K, V = ten("K", 2, 2, 5, 128), ten("V", 2, 2, 5, 128)
    q, o = ten("q", 2, 4, 1, 128), ten("o", 2, 4, 1, 128)
    sig, out = np.ones(4), ctypes.c_int64()
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    for st in (lambda: lib.plsh_q4_cache_write(r(K), r(V), r(c), AT["pos"], None, None),
               lambda: lib.plsh_q4_cache_read(r(c), AT["pos"], None, r(K), r(V), None),
               lambda: lib.plsh_q4_decode_work_bytes(r(q), r(c), r(out)),
               lambda: lib.plsh_alibi_exact_decode_q4(r(q), r(c), sp, AT["pos"], r(o), AT["work"], 1 << 40, None)):
        refused(lib, st(), plsh.PLSH_ERR_INVALID, word)


def test_no_cache(lib):
    K, V = ten("K", 2, 2, 5, 128), ten("V", 2, 2, 5, 128)
    q, o = ten("q", 2, 4, 1, 128), ten("o", 2, 4, 1, 128)
    sig, out = np.ones(4), ctypes.c_int64()
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    for st in (lambda: lib.plsh_q4_cache_write(r(K), r(V), None, AT["pos"], None, None),
               lambda: lib.plsh_q4_cache_read(None, AT["pos"], None, r(K), r(V), None),
               lambda: lib.plsh_q4_decode_work_bytes(r(q), None, r(out)),
               lambda: lib.plsh_alibi_exact_decode_q4(r(q), None, sp, AT["pos"], r(o), AT["work"], 1 << 40, None)):
        refused(lib, st(), plsh.PLSH_ERR_INVALID, "cache is NULL")


K0, V0 = ("K", 2, 2, 5, 128), ("V", 2, 2, 5, 128)
F32 = plsh.PLSH_F32
BAD_ROWS = [
    (K0, V0, dict(v=dict(dtype=F32)), "V must have K's shape and dtype"),
    (K0, ("V", 2, 2, 6, 128), {}, "V must have K's shape and dtype"),
    (K0, ("V", 2, 1, 5, 128), {}, "V must have K's shape and dtype"),
    (("K", 3, 2, 5, 128), ("V", 3, 2, 5, 128), {}, "cache's B, H and d"),
    (("K", 2, 4, 5, 128), ("V", 2, 4, 5, 128), {}, "cache's B, H and d"),
    (("K", 2, 2, 5, 64), ("V", 2, 2, 5, 64), {}, "cache's B, H and d"),
    (("K", 2, 2, 0, 128), ("V", 2, 2, 0, 128), {}, "K: every dimension"),
    (K0, ("V", 2, 2, 0, 128), {}, "V: every dimension"),
    (K0, V0, dict(k=dict(dtype=7), v=dict(dtype=7)), "K: dtype"),
    (K0, V0, dict(v=dict(dtype=7)), "V: dtype"),
    (K0, V0, dict(k=dict(off=4)), "K->data must be 16-byte aligned"),
    (K0, V0, dict(v=dict(off=8)), "V->data must be 16-byte aligned"),
    (K0, V0, dict(k=dict(off=-AT["K"])), "K->data is NULL"),
    (K0, V0, dict(v=dict(off=-AT["V"])), "V->data is NULL"),
    (K0, V0, dict(pos=None), "pos is NULL"),
    (K0, V0, dict(pos=AT["pos"] + 1), "pos and len must be int32"),
    (K0, V0, dict(len=AT["len"] + 2), "pos and len must be int32"),
]


@pytest.mark.parametrize("i", range(len(BAD_ROWS)))
def test_each_fault_of_rows(lib, i):
    k, v, kw, word = BAD_ROWS[i]
    K, V, c = ten(*k, **kw.get("k", {})), ten(*v, **kw.get("v", {})), cache()
    pos, ln = kw.get("pos", AT["pos"]), kw.get("len")
    refused(lib, lib.plsh_q4_cache_write(r(K), r(V), r(c), pos, ln, None), plsh.PLSH_ERR_INVALID, word)
    refused(lib, lib.plsh_q4_cache_read(r(c), pos, ln, r(K), r(V), None), plsh.PLSH_ERR_INVALID, word)


Q0, O0 = ("q", 2, 4, 1, 128), ("o", 2, 4, 1, 128)
BAD_QUERIES = [
    (("q", 2, 4, 2, 128), O0, {}, "q must be [B, Hq, 1, d]"),
    (("q", 1, 4, 1, 128), O0, {}, "q must have the cache's B and d"),
    (("q", 2, 4, 1, 64), O0, {}, "q must have the cache's B and d"),
    (("q", 2, 3, 1, 128), O0, {}, "multiple of the cache's H"),
    (Q0, O0, dict(q=dict(off=2)), "q->data must be 16-byte aligned"),
    (Q0, O0, dict(q=dict(dtype=5)), "q: dtype"),
    (Q0, O0, dict(q=dict(off=-AT["q"])), "q->data is NULL"),
    (Q0, O0, dict(o=dict(dtype=F32)), "o must have q's shape and dtype"),
    (Q0, ("o", 2, 2, 1, 128), {}, "o must have q's shape and dtype"),
    (Q0, ("o", 2, 4, 2, 128), {}, "o must have q's shape and dtype"),
    (Q0, O0, dict(o=dict(off=8)), "o->data must be 16-byte aligned"),
    (Q0, O0, dict(o=dict(off=-AT["o"])), "o->data is NULL"),
    (Q0, O0, dict(pos=None), "pos must be"),
    (Q0, O0, dict(pos=AT["pos"] + 2), "pos must be"),
    (Q0, O0, dict(sigma=None), "sigma_h is NULL"),
    (Q0, O0, dict(sigma=[1, 0, 1, 1]), "sigma_h[1]"),
    (Q0, O0, dict(sigma=[1, 1, -2, 1]), "sigma_h[2]"),
    (Q0, O0, dict(sigma=[1, 1, 1, np.inf]), "sigma_h[3]"),
    (Q0, O0, dict(sigma=[np.nan, 1, 1, 1]), "sigma_h[0]"),
]


@pytest.mark.parametrize("i", range(len(BAD_QUERIES)))
def test_each_fault_of_a_decode_call(lib, i):
    q, o, kw, word = BAD_QUERIES[i]
    q, o, c = ten(*q, **kw.get("q", {})), ten(*o, **kw.get("o", {})), cache()
    sig = kw.get("sigma", [1, 1, 1, 1])
    sig = None if sig is None else np.array(sig, dtype=np.float64)
    sp = None if sig is None else sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    pos = kw.get("pos", AT["pos"])
    refused(lib, lib.plsh_alibi_exact_decode_q4(r(q), r(c), sp, pos, r(o), AT["work"], 1 << 40, None),
            plsh.PLSH_ERR_INVALID, word)


def test_no_bins_no_bytes_and_more_heads_than_are_served(lib):
    q, o, c, out = ten(*Q0), ten(*O0), cache(), ctypes.c_int64()
    refused(lib, lib.plsh_alibi_decode_q4(r(q), r(c), None, AT["pos"], r(o), AT["work"], 1 << 40, None),
            plsh.PLSH_ERR_INVALID, "bins is NULL")
    refused(lib, lib.plsh_q4_decode_work_bytes(r(q), r(c), None), plsh.PLSH_ERR_INVALID, "bytes is NULL")
    many, to = ten("q", 2, 514, 1, 128), ten("o", 2, 514, 1, 128)
    sig = np.ones(514)
    sp = sig.ctypes.data_as(ctypes.POINTER(ctypes.c_double))
    refused(lib, lib.plsh_alibi_exact_decode_q4(r(many), r(c), sp, AT["pos"], r(to), AT["work"], 1 << 40, None),
            plsh.PLSH_ERR_UNSUPPORTED, "512 heads")
    huge = ten("q", 2, 2 ** 62, 1, 128)
    refused(lib, lib.plsh_q4_decode_work_bytes(r(huge), r(c), r(out)), plsh.PLSH_ERR_UNSUPPORTED, "B * Hq")
