"""Page tables and slot maps kept on the GPU, against a plain loop over requests
and pages (whole numbers: equal)."""
import numpy as np
import pytest
import torch

import positional_lsh_approximation_gb300 as plsh
from oracle import q4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    plsh.build()
    plsh.load()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Pages:
    """Tables on the device and on the host, nothing held yet."""

    def __init__(self, B, cap, page, pages, S=0, seed=0):
        rng = np.random.default_rng(seed)
        order = rng.permutation(pages).astype(np.int32)
        self.B, self.cap, self.page, self.pages = B, cap, page, pages
        self.prefix = order[:S]
        self.table = np.full((B, cap), -1, np.int32)
        self.held = np.zeros(B, np.int32)
        self.pool = np.zeros(1 + pages, np.int32)
        self.pool[0] = pages - S
        self.pool[1:1 + pages - S] = order[S:]
        self.upload()
        data = torch.empty(plsh.q4_cache_bytes(pages, 1, page, 64), dtype=torch.uint8, device="cuda")
        self.cache = plsh.Q4Cache(data, self.d_table, 1, 64, page)
        self.d_prefix = i32(self.prefix) if S else None

    def upload(self):
        self.d_table, self.d_held, self.d_pool = i32(self.table), i32(self.held), i32(self.pool)

    def step(self, need):
        plsh.q4_cache_reserve(self.cache, i32(need), self.d_held, self.d_pool, self.d_prefix)
        q4.reserve(self.table, self.held, self.pool, need, self.page, self.prefix)
        self.same()

    def same(self):
        np.testing.assert_array_equal(self.d_held.cpu().numpy(), self.held)
        np.testing.assert_array_equal(self.d_table.cpu().numpy(), self.table)
        np.testing.assert_array_equal(self.d_pool.cpu().numpy(), self.pool)
        plsh.stream_status()


SHAPES = [
    # B, max_pages, page, pages, shared
    (1, 1, 16, 1, 0), (1, 5, 256, 9, 3), (3, 40, 16, 50, 0), (64, 128, 64, 5000, 0), (64, 16, 64, 300, 5),
    (200, 300, 32, 20000, 40), (1023, 9, 16, 4000, 0), (1025, 9, 16, 4000, 2), (2500, 33, 128, 30000, 0),
    (7, 64, 16, 70, 64),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
def test_calls_one_after_the_other(shape):
    B, cap, page, pages, S = shape
    t = Pages(B, cap, page, pages, S, seed=B)
    rng = np.random.default_rng(B + 1)
    need = np.zeros(B, np.int64)
    for k in range(12):
        u = rng.random(B)
        need = np.where(u < 0.3, 0, np.where(u < 0.6, rng.integers(1, cap * page + 1, B), np.minimum(need + 1, cap * page)))
        if k == 5:
            need[:] = cap * page                        # more than there is, most of the time
        if k == 9:
            need[:] = rng.integers(-3, 2, B)
        t.step(need)


def test_growing_and_releasing_leaves_the_stack_as_it_was():
    t = Pages(50, 30, 32, 900, 3)
    first = np.random.default_rng(0).integers(0, 500, 50)
    t.step(first)
    table, pool = t.table.copy(), t.pool.copy()
    then = np.where(np.arange(50) % 3 == 0, 0, first + 400)
    t.step(then)
    assert (t.table != table).any()
    t.step(first)
    np.testing.assert_array_equal(t.d_table.cpu().numpy(), table)
    np.testing.assert_array_equal(t.d_pool.cpu().numpy()[:1 + pool[0]], pool[:1 + pool[0]])


def test_more_than_a_row_holds_or_a_count_out_of_range_is_left_and_reported():
    t = Pages(4, 3, 16, 20)
    t.step([10, 20, 30, 0])
    plsh.q4_cache_reserve(t.cache, i32([49, 48, 2 ** 31 - 1, 1]), t.d_held, t.d_pool)
    with pytest.raises(plsh.PlshError) as e:
        plsh.stream_status()
    assert e.value.status == plsh.PLSH_ERR_INVALID
    q4.reserve(t.table, t.held, t.pool, [49, 48, 2 ** 31 - 1, 1], 16)
    t.same()
    for wrong in (-1, 4):
        t.d_held[2] = wrong                             # more than the row has, or less than nothing
        before = t.d_table.clone()
        plsh.q4_cache_reserve(t.cache, i32([1, 48, 16, 1]), t.d_held, t.d_pool)
        with pytest.raises(plsh.PlshError):
            plsh.stream_status()
        assert torch.equal(t.d_table[2], before[2])
    t = Pages(2, 3, 16, 6)
    t.d_pool[0] = 7                                     # counts as six
    plsh.q4_cache_reserve(t.cache, i32([48, 48]), t.d_held, t.d_pool)
    with pytest.raises(plsh.PlshError):
        plsh.stream_status()
    assert t.d_held.tolist() == [3, 3] and t.d_pool[0].item() == 0
    t.d_pool[0] = 5                                     # pages that come back past the stack's end are dropped
    plsh.q4_cache_reserve(t.cache, i32([0, 0]), t.d_held, t.d_pool)
    with pytest.raises(plsh.PlshError):
        plsh.stream_status()
    assert t.d_held.tolist() == [0, 0] and t.d_pool[0].item() == 6


@pytest.mark.parametrize("m", [1, 2, 7, 100])
def test_slots(m):
    t = Pages(37, 6, 16, 150, 1)
    rng = np.random.default_rng(m)
    t.step(rng.integers(0, 97, 37))
    pos = rng.integers(0, 96 - min(m, 96) + 1, 37)
    pos[3] = -1
    lens = rng.integers(0, m + 1, 37)
    pos = np.where(pos + lens > 96, 0, pos)
    lens = np.minimum(lens, 96)
    got = plsh.q4_cache_slots(t.cache, i32(pos), i32(lens), m=m)
    want = q4.slots(t.table, t.pages, 16, pos, lens, m)
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    plsh.stream_status()
    if m <= 96:
        out = torch.full((37, m), 5, dtype=torch.int64, device="cuda")
        assert plsh.q4_cache_slots(t.cache, i32([96 - m] * 37), out=out) is out
        np.testing.assert_array_equal(out.cpu().numpy(), q4.slots(t.table, t.pages, 16, [96 - m] * 37, [m] * 37, m))
        plsh.stream_status()
        plsh.q4_cache_slots(t.cache, i32([97 - m] * 37), out=out)      # one past the end
        with pytest.raises(plsh.PlshError):
            plsh.stream_status()
        assert (out[:, -1] == -1).all()


def test_slots_say_where_a_write_goes():
    B, m, page = 3, 21, 16
    t = Pages(B, 5, page, 11)
    pos, lens = [0, 30, 15], [21, 10, 0]
    t.step([p + n for p, n in zip(pos, lens)])
    k = torch.randn(B, 1, m, 64, device="cuda")
    t.cache.data.fill_(7)
    plsh.q4_cache_write(t.cache, k, k, i32(pos), i32(lens))
    slots = plsh.q4_cache_slots(t.cache, i32(pos), i32(lens), m=m).cpu().numpy()
    K, _ = q4.read_tiles(t.cache.data.cpu().numpy().reshape(-1, 20 * 64), 64)
    flat = K.reshape(-1, 64)
    for b in range(B):
        for i in range(m):
            if i < lens[b]:
                c, lo, step = q4.quantise(k[b, 0, i].cpu().numpy()[None])
                np.testing.assert_array_equal(flat[slots[b, i]], (np.repeat(lo, 32) + np.repeat(step, 32).astype(np.float64) * c[0]))
            else:
                assert slots[b, i] == -1


def test_a_captured_step_follows_the_lengths():
    t = Pages(20, 8, 16, 200, 1)
    t.step(np.arange(20))
    need, pos = i32(np.arange(20)), i32(np.arange(20) - 1)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros(20, 1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        need += 1
        pos += 1
        plsh.q4_cache_reserve(t.cache, need, t.d_held, t.d_pool, t.d_prefix)
        plsh.q4_cache_slots(t.cache, pos, out=out)
    for k in range(1, 70):
        g.replay()
        want = np.arange(20) + k
        q4.reserve(t.table, t.held, t.pool, want, 16, t.prefix)
        t.same()
        np.testing.assert_array_equal(out.cpu().numpy(), q4.slots(t.table, 200, 16, want - 1, [1] * 20, 1))


def test_refusals():
    t = Pages(4, 3, 16, 20)
    good = dict(need=i32([1] * 4), held=t.d_held, pool=t.d_pool)
    for name, bad in (("need", i32([1] * 3)), ("need", i32([1] * 4).long()), ("held", i32([0] * 5)),
                      ("pool", i32([])), ("pool", t.d_pool.view(1, -1)), ("pool", t.d_pool.cpu()),
                      ("need", torch.zeros(8, dtype=torch.int32, device="cuda")[::2])):
        with pytest.raises(ValueError, match=name):
            plsh.q4_cache_reserve(t.cache, **{**good, name: bad})
    with pytest.raises(ValueError, match="prefix"):
        plsh.q4_cache_reserve(t.cache, **good, prefix=i32([[1]]))
    with pytest.raises(plsh.PlshError, match="prefix_pages"):
        plsh.q4_cache_reserve(t.cache, **good, prefix=i32([1, 2, 3, 4]))
    with pytest.raises(ValueError, match="give m"):
        plsh.q4_cache_slots(t.cache, i32([0] * 4))
    for out in (torch.zeros(4, 2, dtype=torch.int32, device="cuda"), torch.zeros(3, 2, dtype=torch.int64, device="cuda"),
                torch.zeros(2, 4, dtype=torch.int64, device="cuda").T):
        with pytest.raises(ValueError, match="out"):
            plsh.q4_cache_slots(t.cache, i32([0] * 4), out=out)
    t.same()
