"""Definitions of the block-scaled fp8 paged cache, in float64 and plain loops.

TEST INFRASTRUCTURE (same rules as the rest of oracle/): page bookkeeping,
the cache write, and the gather of a sequence's rows from the pages, written
from the definitions in the library's header and sharing no code with it.
"""
import numpy as np

from .fp8 import e4m3_to_float64

E4M3_MAX = 448.0
MIN_EXP, MAX_EXP = -60, 60
_GRID = e4m3_to_float64(np.arange(127, dtype=np.uint8))  # nonnegative values, ascending


def encode_e4m3(x):
    """float64 -> e4m3 codes: nearest, ties to the even code, clamped to +-448, NaN 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    x = np.where(nan, 0.0, x)
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 126)
    lo = hi - 1
    below, above = a - _GRID[lo], _GRID[hi] - a
    code = np.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return np.where(nan, 0x7F, code + 128 * np.signbit(x)).astype(np.uint8)


def scale_exponent(amax):
    """Smallest e in [-60, 60] with amax <= 448 * 2^e (60 where there is none)."""
    for e in range(MIN_EXP, MAX_EXP):
        if amax <= E4M3_MAX * 2.0 ** e:
            return e
    return MAX_EXP


def page_map(lens, cu, total_q, table, free, head, page_size):
    """Returns (slots, offsets, head_out, table, code): lens Lk_b, cu new-token
    offsets or None (one each), table int [batch, max_pages] (copied)."""
    table = np.array(table, dtype=np.int64)
    batch, max_pages = table.shape
    slots = np.full(total_q, -1, dtype=np.int64)
    offsets, at, code = [int(head)], int(head), 0
    for b in range(batch):
        q0, lq = (b, 1) if cu is None else (int(cu[b]), int(cu[b + 1] - cu[b]))
        lk = int(lens[b])
        if lk < 0 or lk > max_pages * page_size:
            code = code or 3
        lk = max(lk, 0)
        for i in range(lq):
            pos = lk - lq + i
            pg = pos // page_size
            if pos < 0 or pg >= max_pages:
                continue
            if pos % page_size == 0:  # the token starts a page: a new one
                table[b, pg] = free[at] if at < len(free) else -1
                at += 1
            if table[b, pg] >= 0:
                slots[q0 + i] = table[b, pg] * page_size + pos % page_size
        offsets.append(at)
    if at > len(free):
        code = code or 4
    return slots, np.array(offsets), min(at, len(free)), table, code


def append(rows, slots, cache, scale):
    """rows float64 [n, hkv, D] into (cache uint8, scale float32), both copied.
    A token at a time is not enough (a block's scale covers all its new rows),
    so the rows are first grouped by block."""
    cache, scale = np.array(cache), np.array(scale)
    pages, hkv, page, _ = cache.shape
    block = page // scale.shape[2]
    groups = {}
    for i, s in enumerate(np.asarray(slots)):
        if 0 <= s < pages * page:
            groups.setdefault(int(s) // block, []).append((int(s) % block, i))
    for blk, members in groups.items():
        p, c = divmod(blk, page // block)
        first = min(off for off, _ in members)
        for g in range(hkv):
            mags = np.abs(np.stack([rows[i, g] for _, i in members]))
            amax = float(mags[np.isfinite(mags)].max(initial=0.0))
            s = 2.0 ** scale_exponent(amax)
            if first > 0:
                had = float(scale[p, g, c])
                while s < had and s < 2.0 ** MAX_EXP:
                    s *= 2.0
                old = slice(c * block, c * block + first)
                if s != had:
                    cache[p, g, old] = encode_e4m3(e4m3_to_float64(cache[p, g, old]) * (had / s))
            scale[p, g, c] = s
            for off, i in members:
                cache[p, g, c * block + off] = encode_e4m3(rows[i, g] / s)
    return cache, scale


def rows_of(cache, scale, table_row, length):
    """float64 [length, hkv, D]: the dequantised rows of one sequence; the rows of
    pages outside the cache count as zeros."""
    pages, hkv, page, d = cache.shape
    block = page // scale.shape[2]
    out = np.zeros((length, hkv, d))
    for p0 in range(0, length, page):
        pid = int(table_row[p0 // page])
        n = min(page, length - p0)
        if 0 <= pid < pages:
            sc = np.repeat(scale[pid].astype(np.float64), block, axis=1)[:, :n]
            out[p0:p0 + n] = (e4m3_to_float64(cache[pid, :, :n]) * sc[..., None]).transpose(1, 0, 2)
    return out
