"""Page tables and slot maps: the oracle against examples done by hand, and the
entry points' refusals."""
import ctypes

import numpy as np
import pytest

import positional_lsh_approximation_gb300 as plsh
from oracle import q4

C = plsh._Q4Cache
AT = {name: (i + 1) << 32 for i, name in enumerate(("data", "table", "need", "held", "pool", "prefix", "pos", "len",
                                                    "slots"))}


@pytest.fixture(scope="module")
def lib():
    plsh.build()
    return plsh.load()


def cache(**kw):
    a = dict(data=AT["data"], table=AT["table"], B=2, H=2, pages=8, max_pages=4, page=64, d=128, **{})
    a.update(kw)
    return C(*(a[k] for k in ("data", "table", "B", "H", "pages", "max_pages", "page", "d")))


def test_oracle_by_hand():
    table = np.full((3, 4), -1, np.int32)
    held, pool = np.zeros(3, np.int32), np.array([5, 10, 11, 12, 13, 14], np.int32)
    q4.reserve(table, held, pool, [17, 0, 16], 16)
    assert held.tolist() == [2, 0, 1] and table[0, :2].tolist() == [14, 13] and table[2, 0] == 12 and pool[0] == 2
    q4.reserve(table, held, pool, [1, 64, 16], 16)               # the first gives one, the second does not fit
    assert held.tolist() == [1, 0, 1] and pool[:4].tolist() == [3, 10, 11, 13] and table[0].tolist() == [14, -1, -1, -1]
    q4.reserve(table, held, pool, [0, 48, 48], 16)               # the second fits then, the third no more
    assert held.tolist() == [0, 3, 1] and table[1].tolist() == [14, 13, 11, -1] and pool[0] == 1
    assert q4.slots(table, 20, 16, [0, 31, 15], [1, 3, 2], 3).tolist() == [
        [-1, -1, -1], [13 * 16 + 15, 11 * 16, 11 * 16 + 1], [12 * 16 + 15, -1, -1]]


def test_oracle_prefix_by_hand():
    table, held = np.full((2, 4), -1, np.int32), np.zeros(2, np.int32)
    pool = np.array([2, 5, 6, 0], np.int32)
    q4.reserve(table, held, pool, [1, 40], 16, [8, 9])
    assert table.tolist() == [[8, 9, -1, -1], [8, 9, 6, -1]] and held.tolist() == [2, 3] and pool[0] == 1
    q4.reserve(table, held, pool, [64, 0], 16, [8, 9])
    assert table.tolist() == [[8, 9, 6, 5], [-1, -1, -1, -1]] and held.tolist() == [4, 0] and pool[0] == 0


BAD = [
    ("reserve", dict(need=None), "must not be NULL"), ("reserve", dict(held=None), "must not be NULL"),
    ("reserve", dict(pool=None), "must not be NULL"), ("reserve", dict(need=AT["need"] + 1), "int32 device"),
    ("reserve", dict(held=AT["held"] + 2), "int32 device"), ("reserve", dict(pool=AT["pool"] + 2), "int32 device"),
    ("reserve", dict(prefix=AT["prefix"] + 2), "int32 device"), ("reserve", dict(pool_pages=-1), "pool_pages"),
    ("reserve", dict(pool_pages=2 ** 31), "pool_pages"), ("reserve", dict(prefix_pages=-1), "prefix_pages"),
    ("reserve", dict(prefix_pages=5), "prefix_pages"), ("reserve", dict(prefix=None, prefix_pages=1), "prefix is NULL"),
    ("reserve", dict(cache=dict(page=24)), "page must be"), ("reserve", dict(cache=dict(table=0)), "table must be"),
    ("slots", dict(pos=None), "must not be NULL"), ("slots", dict(slots=None), "must not be NULL"),
    ("slots", dict(pos=AT["pos"] + 2), "int32 device"), ("slots", dict(len=AT["len"] + 1), "int32 device"),
    ("slots", dict(slots=AT["slots"] + 8), "16-byte aligned"), ("slots", dict(m=0), "m must be"),
    ("slots", dict(m=-1), "m must be"), ("slots", dict(cache=dict(B=0)), "B must be"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_each_fault(lib, i):
    call, kw, word = BAD[i]
    c = cache(**kw.get("cache", {}))
    a = dict(need=AT["need"], held=AT["held"], pool=AT["pool"], pool_pages=8, prefix=AT["prefix"], prefix_pages=0,
             pos=AT["pos"], len=None, m=3, slots=AT["slots"])
    a.update(kw)
    if call == "reserve":
        st = lib.plsh_q4_cache_reserve(ctypes.byref(c), a["need"], a["held"], a["pool"], a["pool_pages"], a["prefix"],
                                       a["prefix_pages"], None)
    else:
        st = lib.plsh_q4_cache_slots(ctypes.byref(c), a["pos"], a["len"], a["m"], a["slots"], None)
    assert st == plsh.PLSH_ERR_INVALID
    assert word in lib.plsh_last_error().decode()


def test_more_rows_than_are_served(lib):
    c = cache(B=65535)
    assert lib.plsh_q4_cache_slots(ctypes.byref(c), AT["pos"], None, 2 ** 20, AT["slots"], None) == plsh.PLSH_ERR_UNSUPPORTED
    assert lib.plsh_q4_cache_slots(ctypes.byref(c), AT["pos"], None, 2 ** 62, AT["slots"], None) == plsh.PLSH_ERR_UNSUPPORTED
    assert lib.plsh_q4_cache_slots(None, AT["pos"], None, 1, AT["slots"], None) == plsh.PLSH_ERR_INVALID
    assert lib.plsh_q4_cache_reserve(None, AT["need"], AT["held"], AT["pool"], 1, None, 0, None) == plsh.PLSH_ERR_INVALID
