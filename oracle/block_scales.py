"""Reference for an e4m3 cache with a scale for each block and KV head (test
infrastructure only; see the package docstring).

Key (and value) of physical block b, slot t, KV head g: code * scale[b, g].

Appending a step's elements x (keys after their rotation) to the block's slots
from `first` on, with A the largest finite |x| of the block and head:

  first = 0:  scale = 2^k, the least k with A <= 448 * 2^k, held to
              [2^-100, 2^100]; 2^-100 when A = 0
  first > 0:  scale = old * 2^n, the least n >= 0 with A <= 448 * old * 2^n
              (and scale <= 2^100); the codes of the slots before `first`
              become e4m3(code / 2^n). An old scale outside [2^-100, 2^100]
              counts as none: the first rule, and the codes stay.
  code = e4m3(x / scale)

The codes of new elements are left as the exact quotients x / scale, in
binary64: what is at most half a step from them is right. Reading: powers of
two, because e4m3 has the same relative step in every binade, so that moving a
block's scale leaves its earlier codes exact (but for subnormal ones).
"""
from __future__ import annotations

import numpy as np

from .fp8_products import round_e4m3

LEAST, MOST = 2.0 ** -100, 2.0 ** 100
E4M3_MAX = 448.0


def _power(a: float) -> float:
    """The least power of two of at least a / 448, by search."""
    s = LEAST
    while a > E4M3_MAX * s and s < MOST:
        s *= 2.0
    return s


def next_scale(amax: float, old: float, first: int):
    """(scale, n) of a block and head after a step."""
    if first == 0 or not LEAST <= old <= MOST:
        return _power(amax), 0
    scale, n = float(np.float32(old)), 0
    limit = float(np.float32(448.0) * np.float32(old))
    while amax > limit * 2.0 ** n and scale * 2.0 <= MOST:
        scale, n = scale * 2.0, n + 1
    return scale, n


def append(x: np.ndarray, codes: np.ndarray, scales: np.ndarray, cu, kv_lens, block_tables,
           block_size: int, skip=()):
    """(values, scales): x [tokens, Hkv, d] (binary64) appended to codes (the e4m3
    values, [blocks, block_size, Hkv, d]) under scales [blocks, Hkv]. skip:
    sequences whose page does not exist."""
    codes, scales = np.array(codes, dtype=np.float64), np.array(scales, dtype=np.float64)
    cu = [int(c) for c in cu]
    for s in range(len(cu) - 1):
        n = cu[s + 1] - cu[s]
        ctx = int(kv_lens[s]) - n
        if s in skip:
            continue
        for page in sorted({p // block_size for p in range(ctx, ctx + n)}):
            lo, hi = max(ctx, page * block_size), min(ctx + n, (page + 1) * block_size)
            b, first = int(block_tables[s, page]), lo % block_size
            new = x[cu[s] + lo - ctx:cu[s] + hi - ctx]
            for g in range(codes.shape[2]):
                size = np.abs(new[:, g])
                size = size[np.isfinite(size)]
                scale, n2 = next_scale(float(size.max(initial=0.0)), scales[b, g], first)
                if n2:
                    codes[b, :first, g] = round_e4m3(codes[b, :first, g] / 2.0 ** n2)
                scales[b, g] = scale
                codes[b, first:first + hi - lo, g] = new[:, g] / scale
    return codes, scales


def dequantised(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Values of a cache's codes ([blocks, block_size, Hkv, d], as values)."""
    return np.asarray(codes, dtype=np.float64) * np.asarray(scales, dtype=np.float64)[:, None, :, None]
