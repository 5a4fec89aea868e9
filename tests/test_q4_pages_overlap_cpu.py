"""Page tables: arrays that lie in one another are refused (a prefix that is a row of
the table being written, most likely)."""
import ctypes

import pytest

import positional_lsh_approximation_gb300 as plsh
from test_q4_pages_cpu import AT, cache


@pytest.fixture(scope="module")
def lib():
    plsh.build()
    return plsh.load()


def reserve(lib, **kw):
    a = dict(need=AT["need"], held=AT["held"], pool=AT["pool"], pool_pages=8, prefix=AT["prefix"], prefix_pages=2)
    a.update(kw)
    c = cache()                                          # a table of 2 x 4
    return lib.plsh_q4_cache_reserve(ctypes.byref(c), a["need"], a["held"], a["pool"], a["pool_pages"], a["prefix"],
                                     a["prefix_pages"], None)


@pytest.mark.parametrize("kw", [
    dict(prefix=AT["table"]), dict(prefix=AT["table"] + 28), dict(prefix=AT["table"] - 4), dict(prefix=AT["pool"] + 4),
    dict(prefix=AT["held"] - 4), dict(need=AT["held"]), dict(need=AT["held"] + 4), dict(need=AT["table"] + 16),
    dict(need=AT["pool"] + 32), dict(held=AT["table"]), dict(held=AT["pool"] + 32), dict(pool=AT["table"] - 32),
    dict(pool=AT["held"] - 32),
])
def test_overlaps_are_refused(lib, kw):
    assert reserve(lib, **kw) == plsh.PLSH_ERR_INVALID
    assert "must not overlap" in lib.plsh_last_error().decode()


@pytest.mark.parametrize("kw", [
    dict(prefix=AT["table"] + 32), dict(prefix=AT["table"] - 8), dict(need=AT["held"] + 8), dict(pool=AT["held"] - 36),
    dict(need=AT["prefix"]),                             # both are only read
    dict(prefix=AT["table"], prefix_pages=0),            # none of it is
])
def test_neighbours_are_not(lib, kw):
    reserve(lib, **kw)
    assert "must not overlap" not in lib.plsh_last_error().decode()
