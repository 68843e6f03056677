"""Dropout from a counter, in whole numbers and float64.

Philox 4x32 with ten rounds (Salmon, Moraes, Dror, Shaw: "Parallel random
numbers: as easy as 1, 2, 3", SC 2011, section 3 and table 2): a round takes the
counter (c0, c1, c2, c3) and the key (k0, k1) to
    (hi(M1 c2) ^ c1 ^ k0,  lo(M1 c2),  hi(M0 c0) ^ c3 ^ k1,  lo(M0 c0))
and adds the Weyl constants to the key.
"""
from __future__ import annotations

import numpy as np

M0, M1 = 0xD2511F53, 0xCD9E8D57
W0, W1 = 0x9E3779B9, 0xBB67AE85
MASK = 0xFFFFFFFF


def philox(counter, key):
    """Ten rounds on four uint32 arrays (or whole numbers) and two whole numbers: four uint64 arrays below 2^32."""
    c0, c1, c2, c3 = (np.asarray(c, dtype=np.uint64) for c in counter)
    k0, k1 = (int(k) for k in key)
    u32, mask = np.uint64(32), np.uint64(MASK)
    for _ in range(10):
        a, b = c0 * np.uint64(M0), c2 * np.uint64(M1)
        c0, c1, c2, c3 = (b >> u32) ^ c1 ^ np.uint64(k0), b & mask, (a >> u32) ^ c3 ^ np.uint64(k1), a & mask
        k0, k1 = (k0 + W0) & MASK, (k1 + W1) & MASK
    return c0, c1, c2, c3


def fields(seed: int, step: int, site: int, first: int, count: int):
    """The 16-bit fields of elements first .. first + count - 1 (uint16)."""
    i = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    words = philox((i & np.uint64(MASK), (i >> np.uint64(32)) + np.uint64(site * 4096), np.full_like(i, step & MASK),
                    np.full_like(i, step >> 32 & MASK)), (seed & MASK, seed >> 32 & MASK))
    out = np.stack([h for w in words for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).astype(np.uint16)
    return out.reshape(-1)[first % 8:first % 8 + count]


def threshold(p: float) -> int:
    return min(int(np.rint(p * 65536.0)), 65535)


def kept(seed: int, step: int, site: int, p: float, shape):
    """(bool mask of the elements that stay, their factor)."""
    T = threshold(p)
    f = fields(seed, step, site, 0, int(np.prod(shape, dtype=np.int64)))
    return (f >= T).reshape(shape), 65536.0 / (65536.0 - T)


def dropout(x, seed: int, step: int, site: int, p: float):
    """float64, not rounded."""
    mask, factor = kept(seed, step, site, p, np.shape(x))
    return np.where(mask, np.asarray(x, dtype=np.float64), 0.0) * np.where(mask, factor, 0.0)
