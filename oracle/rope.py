"""Reference for rotary positions (test infrastructure only; see the package
docstring).

The pair (a, b) of a head at position p with frequency w (radians per position)
is the complex number a + ib turned by p w and stretched by the amplitude:

  a' + i b' = m e^{i p w} (a + i b)

over the pairs (x[i], x[i + rotary_dim / 2]) (half layout) or (x[2i], x[2i + 1])
(interleaved), i < rotary_dim / 2; elements from rotary_dim on are unchanged.
Frequencies of a configuration with context length L stretched by `factor`:

  plain   w_i = base^(-2 i / rotary_dim)
  linear  w_i / factor
  ntk     plain with base * factor^(rotary_dim / (rotary_dim - 2))
  bands   by the turns r_i = L w_i / 2 pi a pair makes over L: unchanged from
          `high` on, w_i / factor up to `low`, a linear blend in r between
  yarn    a linear blend in the pair index between the indices whose plain
          frequency makes `high` and `low` turns; amplitude 0.1 ln factor + 1
"""
from __future__ import annotations

import math

import numpy as np


def rotate(x: np.ndarray, positions, inv_freq, interleaved: bool, amplitude: float = 1.0) -> np.ndarray:
    """x [tokens, heads, d] (any float type) rotated, in binary64."""
    y = np.array(x, dtype=np.float64)
    w = np.asarray(inv_freq, dtype=np.float64)
    n = w.size
    a = np.arange(n) * 2 if interleaved else np.arange(n)
    b = a + 1 if interleaved else a + n
    angle = np.asarray(positions, dtype=np.float64)[:, None] * w[None, :]
    turn = amplitude * np.exp(1j * angle)[:, None, :]
    z = (y[..., a] + 1j * y[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def pair_size(x: np.ndarray, rotary_dim: int, interleaved: bool) -> np.ndarray:
    """|a| + |b| of the pair each element belongs to (0 beyond rotary_dim):
    what an error of cos and sin is multiplied by."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    out = np.zeros_like(x)
    n = rotary_dim // 2
    a = np.arange(n) * 2 if interleaved else np.arange(n)
    b = a + 1 if interleaved else a + n
    out[..., a] = out[..., b] = x[..., a] + x[..., b]
    return out


def frequencies(rotary_dim: int, base: float, scaling: str = "plain", factor: float = 1.0,
                length: float = 0.0, low: float = 1.0, high: float = 4.0):
    """([w_i], amplitude) of a configuration."""
    n = rotary_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    w = [math.exp(-2 * i / rotary_dim * math.log(base)) for i in range(n)]
    if scaling == "linear":
        return [x / factor for x in w], 1.0
    if scaling == "bands":
        out = []
        for x in w:
            turns = length * x / (2 * math.pi)
            if turns >= high:
                out.append(x)
            elif turns <= low:
                out.append(x / factor)
            else:
                s = (turns - low) / (high - low)
                out.append((1 - s) * x / factor + s * x)
        return out, 1.0
    if scaling == "yarn":
        def index(turns):
            return rotary_dim * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo = max(0, math.floor(index(high)))
        hi = min(rotary_dim - 1, math.ceil(index(low)))
        out = []
        for i, x in enumerate(w):
            r = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            out.append(x * (1 - r) + x / factor * r)
        return out, 0.1 * math.log(factor) + 1.0
    return w, 1.0
