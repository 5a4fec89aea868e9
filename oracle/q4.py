"""The 4-bit paged K/V cache and its decode steps, in plain numpy.

Quantising follows the recipe operation by operation in fp32 (each rounded
once), so that stored bytes agree bit for bit with any other implementation of
it; the decode steps are fp64 from the values the cache holds.
"""
from __future__ import annotations

import numpy as np

GROUP, TILE = 32, 16


def _round_bf16(x: np.ndarray, up: bool) -> np.ndarray:
    """fp32 rounded to a bf16 value towards +inf (up) or -inf, by steps of the
    bit pattern."""
    b = x.astype(np.float32).view(np.uint32)
    cut = (b & np.uint32(0xFFFF0000)).view(np.float32)
    away = ((b & np.uint32(0xFFFF0000)) + np.uint32(0x10000)).view(np.float32)
    with np.errstate(invalid="ignore"):
        off = cut < x if up else cut > x
    return np.where(off, away, cut).astype(np.float32)


def quantise(x: np.ndarray):
    """x [..., d] fp32 -> codes uint8 [..., d], lo, step fp32 [..., d / 32]."""
    g = x.astype(np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        mn = g.min(-1)
        # (-0 is less than +0, whichever of them numpy's minimum picks)
        lo = _round_bf16(np.where((mn == 0) & (np.signbit(g) & (g == 0)).any(-1), np.float32(-0.0), mn), False)
        spread = (g.max(-1) - lo).astype(np.float32)
        bad = ~np.isfinite(spread)
        step = _round_bf16((spread / np.float32(15)).astype(np.float32), True)
        t = ((g - lo[..., None]).astype(np.float32) / step[..., None]).astype(np.float32)
        c = np.where(step[..., None] > 0, np.clip(np.rint(t), 0, 15), 0)
    c[bad] = 0
    lo = np.where(bad, np.float32(0), lo)
    step = np.where(bad, np.float32(np.nan), step)
    return c.astype(np.uint8).reshape(x.shape), lo, step


def code_byte(d: int, r: int, e: int, value: bool) -> int:
    """Byte of a tile that holds the code of value e of position r of K, or of
    V (value); odd e in the high nibble."""
    y, i = divmod(e, GROUP)
    if not value:
        return r * (d // 2) + (i // 8) * (d // 8) + 4 * y + (i % 8) // 2
    blk, t, par = r // 8, r % 8 // 2, r % 2
    return 8 * d + (y // 2) * 512 + (4 * (i // 4) + t) * 16 + (y % 2) * 8 + 4 * blk + 2 * par \
        + (i % 4) // 2


def pair_byte(d: int, r: int, y: int, value: bool) -> int:
    """First of the four bytes (lo, step) of group y of position r."""
    return (18 if value else 16) * d + (r * (d // GROUP) + y) * 4


def write_row(tile: np.ndarray, r: int, k: np.ndarray, v: np.ndarray):
    """Rows k, v [d] into position r of a tile (uint8 [20 d])."""
    d = k.shape[0]
    for value, x in ((False, k), (True, v)):
        c, lo, step = quantise(x)
        for e in range(0, d, 2):
            tile[code_byte(d, r, e, value)] = c[e] | (c[e + 1] << 4)
        for y in range(d // GROUP):
            at = pair_byte(d, r, y, value)
            if np.isnan(step[y]):
                tile[at:at + 4] = (0, 0, 0xC0, 0x7F)
            else:
                tile[at:at + 2] = np.frombuffer(lo[y].tobytes(), np.uint8)[2:]
                tile[at + 2:at + 4] = np.frombuffer(step[y].tobytes(), np.uint8)[2:]


def read_tiles(tiles: np.ndarray, d: int):
    """tiles uint8 [..., 20 d] -> the fp64 values of K, V [..., 16, d]."""
    out = []
    for value in (False, True):
        at = np.array([[code_byte(d, r, e, value) for e in range(d)] for r in range(TILE)])
        c = tiles[..., at] >> (4 * (np.arange(d) % 2)).astype(np.uint8) & 15
        pa = np.array([[pair_byte(d, r, y, value) for y in range(d // GROUP)] for r in range(TILE)])
        two = lambda k: (tiles[..., pa + k].astype(np.uint32) << 16  # noqa: E731
                         | tiles[..., pa + k + 1].astype(np.uint32) << 24).view(np.float32)
        lo, step = np.repeat(two(0), GROUP, -1), np.repeat(two(2), GROUP, -1)
        with np.errstate(invalid="ignore"):
            out.append(lo.astype(np.float64) + step.astype(np.float64) * c)
    return out


def read_sequence(data: np.ndarray, table: np.ndarray, page: int, d: int, n: int):
    """data uint8 [pages, H, page / 16, 20 d], one sequence's page row ->
    K, V [H, n, d] fp64 of its first n positions."""
    need = -(-n // page)
    H = data.shape[1]
    tiles = data[table[:need]].transpose(1, 0, 2, 3).reshape(H, -1, 20 * d)
    k, v = read_tiles(tiles, d)
    return k.reshape(H, -1, d)[:, :n], v.reshape(H, -1, d)[:, :n]


def decode_row(q: np.ndarray, K: np.ndarray, V: np.ndarray, log_w: np.ndarray) -> np.ndarray:
    """q [Hq, d], K, V [H, n, d], log_w [Hq, n] (log of the mask's weights,
    -inf: not seen) -> o [Hq, d]; a row that sees nothing gives 0."""
    Hq, d = q.shape
    G = Hq // K.shape[0]
    o = np.zeros((Hq, d))
    for h in range(Hq):
        see = log_w[h] > -np.inf
        if not see.any():
            continue
        x = K[h // G][see] @ q[h].astype(np.float64) / np.sqrt(d) + log_w[h][see]
        p = np.exp(x - x.max())
        o[h] = p @ V[h // G][see] / p.sum()
    return o


def log_weights_exact(sigma: np.ndarray, pos: int, n: int) -> np.ndarray:
    """Exact ALiBi: -(pos - j) / sigma_h for j <= pos, [Hq, n]."""
    j = np.arange(n)
    w = -(pos - j)[None] / np.asarray(sigma, dtype=np.float64)[:, None]
    return np.where(j[None] <= pos, w, -np.inf)


def log_weights_approx(offsets, starts, H: int, s: int, pos: int, n: int) -> np.ndarray:
    """log #{t : j and pos share a bin of hash t}, j <= pos, [H, n]."""
    j = np.arange(n)
    c = np.zeros((H, n))
    for hs in range(H * s):
        st = starts[offsets[hs]:offsets[hs + 1]]
        lo = st[np.searchsorted(st, pos, side="right") - 1]
        c[hs // s] += (j >= lo) & (j <= pos)
    with np.errstate(divide="ignore"):
        return np.log(c)


def reserve(table, held, pool, need, page: int, prefix=()):
    """A page table kept from the positions that sequences ask for: table [B,
    max_pages], held [B] and pool (free count, then the stack) are updated in
    place, one sequence and one page after the other."""
    S, (B, cap) = len(prefix), table.shape
    want = [max(-(-int(n) // page), S) if n > 0 else 0 for n in need]
    want = [w if w <= cap else int(h) for w, h in zip(want, held)]
    for b in reversed(range(B)):
        for i in reversed(range(want[b], int(held[b]))):
            if i >= S:
                pool[0] += 1
                pool[pool[0]] = table[b, i]
            table[b, i] = -1
        held[b] = min(held[b], want[b])
    full = False
    for b in range(B):
        if want[b] <= held[b]:
            continue
        missing = range(max(int(held[b]), S), want[b])
        full = full or len(missing) > pool[0]
        if full:
            continue
        if held[b] < S:
            table[b, held[b]:S] = prefix[held[b]:]
        for i in missing:
            table[b, i] = pool[pool[0]]
            pool[0] -= 1
        held[b] = want[b]


def slots(table, pages: int, page: int, pos, lens, m: int):
    """[B, m]: page * page size + row of positions pos[b] + i, i < lens[b]; -1
    where there is none."""
    B, cap = table.shape
    out = np.full((B, m), -1, np.int64)
    for b in range(B):
        for i in range(min(m, int(lens[b]))):
            p = int(pos[b]) + i
            if 0 <= p < cap * page and 0 <= table[b, p // page] < pages:
                out[b, i] = int(table[b, p // page]) * page + p % page
    return out
