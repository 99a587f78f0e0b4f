"""Sinks under a window: the oracle's mask, the schedule's tile lists against a
brute-force enumeration of the keys that each row sees, and refusals (no GPU)."""
import numpy as np
import pytest

import paged_kv_attention_unified_gb300 as ua
from oracle import scores as S


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_unified_gb300 import build
    build.build()


def test_mask_by_hand():
    seen = lambda **k: S.visible_with_prefix(10, 2, 1, True, 3, 0, **k).tolist()  # noqa: E731
    assert seen() == [7, 8, 9]
    assert seen(sinks=2) == [0, 1, 7, 8, 9]
    assert seen(sinks=8) == list(range(10))
    assert S.visible_with_prefix(10, 10, 1, True, 3, 0, sinks=4).tolist() == [0, 1]
    assert S.visible_with_prefix(10, 10, 2, False, 2, 0, sinks=1).tolist() == [0] + list(range(1, 10))
    assert S.visible_with_prefix(10, 10, 8, True, 1, 9, sinks=1).tolist() == [0, 8]


def test_oracle_reads_no_page_that_no_query_sees():
    q = np.zeros((2, 1, 32), dtype=np.uint16)
    cache = np.full((4, 16, 1, 32), 0x3F80, dtype=np.uint16)  # 1.0
    table = np.array([[0, -99, -99, 2, 3]])
    out, _ = S.paged_attention_shaped(q, cache, cache, [0, 2], [70], table, 16, 1.0, window=20, sinks=5)
    assert np.array_equal(out, np.ones_like(out))


CASES = [  # query lengths, kv lengths, window, sinks, causal, prefix
    ([1, 1, 1], [40, 500, 2000], 64, 4, 1, None),
    ([1, 3], [5000, 333], 100, 33, 1, None),
    ([1, 2], [3000, 1000], 16, 700, 1, None),
    ([200, 1, 77], [900, 1200, 77], 130, 4, 1, None),
    ([300], [2000], 1, 1, 1, None),
    ([300, 50], [2000, 700], 200, 129, 1, None),
    ([260, 9], [1500, 800], 200, 128, 1, [70, 790]),
    ([150, 1], [800, 640], 90, 10, 0, None),
    ([700], [700], 128, 16, 1, None),
    ([40], [40], 1000, 7, 1, None),
    ([5], [1000], 2 ** 31 - 1, 2 ** 31 - 1, 1, None),
    ([5], [1000], 10, 2 ** 31 - 1, 1, None),
]


def _read(t, step, window, sinks, ctx, qpk):
    """Positions a tile reads: its range without the whole steps that its rows pass over."""
    lo, hi = -(-sinks // step) * step, max(0, ctx + t["row0"] // qpk - window + 1) // step * step
    return {k for k in range(t["kv_lo"], t["kv_hi"]) if not (lo <= k < hi and lo < hi)}


@pytest.mark.parametrize("splits", [0, 1, 7, 128])
@pytest.mark.parametrize("case", CASES)
def test_tiles_hold_the_visible_keys_and_no_more(case, splits):
    ql, kv, window, sinks, causal, prefix = case
    hq, hkv, bs, qpk = 8, 2, 16, 4
    cu = np.concatenate([[0], np.cumsum(ql)]).tolist()
    info, pre, dec, groups = ua.ua_schedule(cu, kv, hq, hkv, 128, bs, 400, causal=causal, window=window,
                                            num_splits=splits, prefix_lens=prefix, sink_tokens=sinks)
    need, got, keys_read = {}, {}, 0
    for s, (n, k) in enumerate(zip(ql, kv)):
        for i in range(n):
            seen = S.visible_with_prefix(k, n, i, bool(causal), window, 0 if prefix is None else prefix[s], sinks)
            for h in range(hq):
                need[s, h // qpk, i * qpk + h % qpk] = set(seen.tolist())
    for t, step in [(t, 128) for t in pre] + [(t, 16) for t in dec]:
        ctx = kv[t["seq"]] - ql[t["seq"]]
        # pieces end and begin outside of what the rows pass over
        keys = _read(t, step, window, sinks, ctx, qpk)
        assert keys and t["kv_lo"] in keys and t["kv_hi"] - 1 in keys
        if step == 16:
            keys_read += len(keys) * t["nrows"]
        for r in range(t["row0"], t["row0"] + t["nrows"]):
            at = got.setdefault((t["seq"], t["kv_head"], r), set())
            assert not at & keys  # once each
            at |= keys
    assert got.keys() == need.keys()
    for key, seen in need.items():
        assert seen <= got[key]
    for row, keys in got.items():  # decode rows read what an 8-row block sees, in steps of 16
        if (ql[row[0]] * qpk) <= 32:
            first, last = row[2] // 8 * 8, min(row[2] // 8 * 8 + 7, ql[row[0]] * qpk - 1)
            block = set().union(*(need[row[0], row[1], r] for r in range(first, last + 1)))
            assert keys <= {k for b in block for k in range(b // 16 * 16, b // 16 * 16 + 16)}
    for g in groups:
        assert 2 <= g["nsplits"] <= ua.UA_MAX_SPLITS


def test_splits_share_the_keys_that_are_read():
    """One token after 131071 keys, window 4096, 4 sinks: the pieces are of one size."""
    _, _, dec, _ = ua.ua_schedule([0, 1], [131072], 8, 1, 128, 16, 8192, window=4096, sink_tokens=4,
                                  num_splits=4)
    sizes = [len(_read(t, 16, 4096, 4, 131071, 8)) for t in sorted(dec, key=lambda t: t["kv_lo"])]
    assert len(sizes) == 4 and sum(sizes) == 4096 + 16 and max(sizes) - min(sizes) <= 64


@pytest.mark.parametrize("d", [32, 96, 128, 160, 224, 256])
@pytest.mark.parametrize("dtype", [ua.UA_KV_BF16, ua.UA_KV_FP8_E4M3])
def test_prompts_have_a_prefill_kernel_at_every_head_dim(d, dtype):
    info, pre, dec, _ = ua.ua_schedule([0, 900], [2000], 8, 2, d, 16, 200, kv_dtype=dtype, window=300,
                                       sink_tokens=4, decode_rows_max=0)
    assert pre and not dec


def test_no_sinks_is_the_plain_window():
    args = ([0, 1, 301], [900, 700], 8, 2, 128, 16, 100)
    want = ua.ua_schedule(*args, window=100)
    assert ua.ua_schedule(*args, window=100, sink_tokens=0)[1:] == want[1:]
    plain = ua.ua_schedule(*args)
    assert ua.ua_schedule(*args, window=0, sink_tokens=9)[2:] == plain[2:]


def test_refusals():
    args = ([0, 1], [900], 8, 2, 128, 16, 100)
    for bad in (dict(window=100, sink_tokens=-1), dict(window=0, sink_tokens=-5),
                dict(window=100, sink_tokens=-2 ** 40), dict(window=100, sink_tokens=4, causal=2)):
        with pytest.raises(ua.UAError) as e:
            ua.ua_schedule(*args, **bad)
        assert e.value.status == ua.UA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ua.ua_schedule(*args, window=5, sink_tokens=4, causal=0, prefix_lens=[3])
    with pytest.raises(ValueError):
        ua.ua_schedule(*args, window=5, sink_tokens=4, prefix_lens=[3, 3])


@pytest.mark.parametrize("n,window,hkv,pieces", [
    (1, 256, 8, 1), (1, 496, 8, 4), (1, 1024, 8, 8), (1, 4096, 8, 16), (6, 1024, 8, 8), (8, 1024, 8, 4),
    (1, 1024, 64, 4), (100, 1024, 8, 1)])
def test_small_pieces_only_where_they_are_few(n, window, hkv, pieces):
    """The pieces of a tile: from 128 keys where they are few and fill one wave, else from 256."""
    _, _, dec, _ = ua.ua_schedule(list(range(n + 1)), [30000] * n, 64, hkv, 128, 16, 1875, window=window, sink_tokens=4)
    one = [t for t in dec if t["seq"] == 0 and t["kv_head"] == 0]
    assert len(one) == pieces
