"""Plain 64-bit reference of the 4-bit paged cache on the CPU: format, quantisation, attention of one
token, eviction.  Written from the definitions in include/vs_prefill.h, in numpy."""
from __future__ import annotations

import numpy as np

PAGE = 64


def bf16_round(x: np.ndarray) -> np.ndarray:
    """float64 -> the nearest bf16 value through fp32 (as float64)."""
    with np.errstate(over="ignore", invalid="ignore"):
        b = np.ascontiguousarray(x, np.float64).astype(np.float32).view(np.uint32).astype(np.uint64)
    nan = (b & 0x7FFFFFFF) > 0x7F800000
    r = ((b + 0x7FFF + ((b >> np.uint64(16)) & np.uint64(1))) >> np.uint64(16)).astype(np.uint32)
    r = np.where(nan, np.uint32(0x7FC0), r)
    return (r << np.uint32(16)).view(np.float32).astype(np.float64)


def bf16_bits(x: np.ndarray) -> np.ndarray:
    return (np.ascontiguousarray(x, np.float64).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)


def quantize(x: np.ndarray):
    """x [..., 64] float64 (bf16 values) -> codes, s, m."""
    with np.errstate(all="ignore"):
        bad = ~np.isfinite(x).all(-1)
        y = np.where(bad[..., None], 0.0, x)
        m, hi = y.min(-1), y.max(-1)
        s = bf16_round((hi - m) / 15.0)
        n = np.rint((y - m[..., None]) / np.where(s == 0, 1.0, s)[..., None])
        n = np.where((s == 0)[..., None], 0, np.clip(n, 0, 15))
        n = np.where(bad[..., None], 0, n).astype(np.uint32)
    return n, np.where(bad, np.nan, s), np.where(bad, np.nan, m)


class Cache:
    """Codes [pages, Hkv, 2, GR, 64 slots, 64] and pairs [pages, Hkv, 2, GR, 64 slots] of a pool."""

    def __init__(self, pool_bytes: np.ndarray):
        p, h, nb = pool_bytes.shape
        self.raw = pool_bytes
        self.GR = nb // 4608
        g = self.GR
        c = pool_bytes[..., :g * 4096].reshape(p, h, 2, g, PAGE, 32)
        self.codes = np.stack([c & 15, c >> 4], -1).reshape(p, h, 2, g, PAGE, 64)
        pair = np.ascontiguousarray(pool_bytes[..., g * 4096:]).view(np.uint16).reshape(p, h, 2, g, PAGE, 2)
        val = (pair.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        self.s, self.m = val[..., 0], val[..., 1]

    def rows(self, table_row, head, slots, kv):
        """Values [len(slots), d] of one sequence and head."""
        slots = np.asarray(slots)
        pg = np.asarray(table_row)[slots // PAGE]
        x = self.codes[pg, head, kv, :, slots % PAGE].astype(np.float64)  # [n, GR, 64]
        s, m = self.s[pg, head, kv, :, slots % PAGE], self.m[pg, head, kv, :, slots % PAGE]
        return (x * s[..., None] + m[..., None]).reshape(len(slots), -1)


def pool_write(pool, table_row, head, slot, kv, n, s, m):
    """Writes one slot's group codes n [GR, 64] and pairs into the bytes of a pool."""
    g = n.shape[0]
    page, r = int(table_row[slot // PAGE]), slot % PAGE
    by = (n[:, 0::2] | (n[:, 1::2] << 4)).astype(np.uint8)
    for i in range(g):
        a = (kv * g + i) * 2048 + r * 32
        pool[page, head, a:a + 32] = by[i]
        a = 2 * g * 2048 + (kv * g + i) * 256 + r * 4
        nan = np.isnan(s[i])
        two = np.array([0x7FC0, 0x7FC0], np.uint16) if nan else bf16_bits(np.array([s[i], m[i]]))
        pool[page, head, a:a + 4] = two.view(np.uint8)


def visible(n, window, sinks):
    t = np.arange(n)
    return t if window == 0 else t[(t >= n - window) | (t < sinks)]


def decode(q, cache: Cache, table_row, n, window=0, sinks=0, scale=None):
    """q [Hq, d] float64 -> O [Hq, d], lse [Hq], weights [Hkv, n] (sums over the group's heads)."""
    Hq, d = q.shape
    Hkv = cache.codes.shape[1]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    O, lse, w = np.zeros((Hq, d)), np.full(Hq, -np.inf), np.zeros((Hkv, n))
    t = visible(n, window, sinks)
    if not len(t):
        return O, lse, w
    for g in range(Hkv):
        k, v = (cache.rows(table_row, g, t, kv) for kv in (0, 1))
        for h in range(g * G, (g + 1) * G):
            z = k @ q[h] * scale
            mx = z.max()
            e = np.exp(z - mx)
            O[h] = e @ v / e.sum()
            lse[h] = mx + np.log(e.sum())
            w[g, t] += e / e.sum()
    return O, lse, w


def evict_order(acc, pos, n_tokens, keep, sinks, recent):
    """Source slot of every slot of the cut row."""
    n = len(acc)
    k = min(n, keep)
    fixed = (pos < sinks) | (pos >= n_tokens - recent)

    def key(t):
        if fixed[t]:
            return (0, 0.0, t)
        if np.isnan(acc[t]):
            return (2, 0.0, t)
        return (1, -float(acc[t]) + 0.0, t)

    stay = set(sorted(range(n), key=key)[:k])
    movers = iter(t for t in range(k, n) if t in stay)
    return np.array([t if t in stay else next(movers) for t in range(k)], np.int64)
