"""Reference for shaped attention scores (test infrastructure only; see the
package docstring).

The attention of oracle.attention with three changes to the definition, each
off by default:

  x = scale * <q, k_t>                                 (k dequantised)
  x = softcap * tanh(x / softcap)                      softcap > 0
  x = x - slopes[h] * |pos - t|                        slopes given (ALiBi; the
      alibi_slopes of Flash_fwd_params, "flashatten takeaways EP2 工程")
  visible t: t < kv_len, (not causal or t <= pos or t < prefix_s),
             (window <= 0 or t > pos - window or t < sinks)

An e4m3 cache may have a scale for each block and KV head (oracle.block_scales);
`staged` rounds the dequantised keys and values to bf16, as the copy does that
prefills read.

Everything in binary64, one query row at a time, no running maximum over
blocks. Besides the output it returns what error bounds are made of: for every
output element sum_t p_t |v_t|, and for every row the softmax weights.
"""
from __future__ import annotations

from typing import Optional, Sequence

import numpy as np

from .attention import BF16, decode_bf16, gather_kv, kv_head_of


def visible_with_prefix(kv_len: int, q_len: int, i: int, causal: bool, window: int,
                        prefix: int, sinks: int = 0) -> np.ndarray:
    """Key positions query i of a sequence sees."""
    pos = kv_len - q_len + i
    t = np.arange(kv_len, dtype=np.int64)
    keep = np.ones(kv_len, dtype=bool)
    if causal:
        keep &= (t <= pos) | (t < prefix)
    if window > 0:
        keep &= (t > pos - window) | (t < sinks)
    return t[keep]


def round_bf16(x: np.ndarray) -> np.ndarray:
    """binary64 values to 8 significant bits, nearest, ties to even."""
    f, e = np.frexp(np.asarray(x, dtype=np.float64))
    return np.ldexp(np.rint(f * 256.0) / 256.0, e)


def shape_scores(x: np.ndarray, distance: np.ndarray, softcap: float, slope: float) -> np.ndarray:
    """Cap, then bias, of one row's scaled scores."""
    x = np.asarray(x, dtype=np.float64)
    if softcap > 0:
        x = softcap * np.tanh(x / softcap)
    return x - slope * np.abs(distance)


def paged_attention_shaped(q_bits: np.ndarray, k_cache: np.ndarray, v_cache: np.ndarray,
                           cu_query_lens, kv_lens, block_tables: np.ndarray, block_size: int,
                           scale: float, kv_dtype: str = BF16, k_scale: float = 1.0,
                           v_scale: float = 1.0, causal: bool = True, window: int = 0,
                           softcap: float = 0.0, slopes: Optional[Sequence[float]] = None,
                           prefix_lens: Optional[Sequence[int]] = None, with_probs: bool = False,
                           sinks: int = 0, k_scales: Optional[np.ndarray] = None,
                           v_scales: Optional[np.ndarray] = None, staged: bool = False):
    """(out [Tq, Hq, d], spread [Tq, Hq, d] = sum_t p_t |v_t|[, rows]) in fp64;
    rows[(token, head)] = (visible keys, p, V rows) on request."""
    cu = [int(c) for c in cu_query_lens]
    bt = np.asarray(block_tables, dtype=np.int64)
    Tq, Hq, d = q_bits.shape
    Hkv = k_cache.shape[2]
    out, spread = np.zeros((Tq, Hq, d)), np.zeros((Tq, Hq, d))
    rows = {}
    for s in range(len(cu) - 1):
        qlen, kv = cu[s + 1] - cu[s], int(kv_lens[s])
        if qlen == 0:
            continue
        prefix = 0 if prefix_lens is None else int(prefix_lens[s])
        every = np.arange(kv, dtype=np.int64)
        seen = [visible_with_prefix(kv, qlen, i, causal, window, prefix, sinks) for i in range(qlen)]
        if sinks:  # a page whose keys no query sees need not exist
            every = np.unique(np.concatenate(seen))
            seen = [np.searchsorted(every, t) for t in seen]
        for g in range(Hkv):
            K = gather_kv(k_cache, bt, s, every, g, block_size, kv_dtype, k_scale)
            V = gather_kv(v_cache, bt, s, every, g, block_size, kv_dtype, v_scale)
            if k_scales is not None:
                page = bt[s, every // block_size]
                K, V = K * k_scales[page, g][:, None], V * v_scales[page, g][:, None]
                if staged:
                    K, V = round_bf16(K), round_bf16(V)
            for h in range(Hq):
                if kv_head_of(h, Hq, Hkv) != g:
                    continue
                X = scale * (decode_bf16(q_bits[cu[s]:cu[s + 1], h, :]) @ K.T)
                for i in range(qlen):
                    t = seen[i]
                    x = shape_scores(X[i, t], (kv - qlen + i) - every[t], softcap,
                                     0.0 if slopes is None else float(slopes[h]))
                    e = np.exp(x - np.max(x))
                    p = e / np.sum(e)
                    out[cu[s] + i, h] = p @ V[t]
                    spread[cu[s] + i, h] = p @ np.abs(V[t])
                    if with_probs:
                        rows[(cu[s] + i, h)] = (t, p, V[t])
    return (out, spread, rows) if with_probs else (out, spread)
