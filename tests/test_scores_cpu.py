"""Shaped scores without a GPU: the oracle pinned, the scheduler's key ranges
under a prefix mask against a brute-force enumeration, and refusals."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_kv_attention_unified_gb300 as ua
import workloads as W
from oracle import scores as S


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_unified_gb300 import build
    build.build()


def _raw(case):
    r = case.raw()
    return (r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"], r["kv_lens"], r["block_tables"],
            case.block_size, case.scale)


def test_oracle_without_shape_is_the_plain_oracle():
    for window in (0, 20):
        case = W.random_small_case(5, head_dim=32, max_kv=120, window=window)
        exp, _ = oracle.paged_attention(*_raw(case), causal=case.causal, window=window)
        got, spread = S.paged_attention_shaped(*_raw(case), causal=case.causal, window=window)
        assert np.allclose(got, exp, atol=1e-12)
        assert np.all(spread >= np.abs(got) - 1e-12)


def test_oracle_against_dense_torch():
    """One dense sequence with every shape at once, by elementary torch operations."""
    case = W.make_case("dense", [20], [50], 4, 2, 32, 16, seed=3)
    cap, slopes, prefix, window = 3.0, [0.5, 0.25, 0.1, 0.0], 40, 33
    got, _ = S.paged_attention_shaped(*_raw(case), window=window, softcap=cap, slopes=slopes,
                                      prefix_lens=[prefix])
    k, v = (c[case.block_tables[0].long()].reshape(-1, 2, 32)[:50].double()
            for c in (case.k_cache, case.v_cache))
    pos, t = torch.arange(30, 50)[:, None], torch.arange(50)[None, :]
    seen = ((t <= pos) | (t < prefix)) & (t > pos - window)
    for h in range(4):
        x = case.q[:, h].double() @ k[:, h // 2].T * case.scale
        x = torch.tanh(x / cap) * cap - slopes[h] * (pos - t).abs().double()
        p = torch.softmax(x.masked_fill(~seen, -torch.inf), -1)
        assert np.allclose(got[:, h], (p @ v[:, h // 2]).numpy(), atol=1e-12)


def test_oracle_prefix_and_bias_by_hand():
    assert S.visible_with_prefix(6, 2, 0, True, 0, 0).tolist() == [0, 1, 2, 3, 4]
    assert S.visible_with_prefix(6, 6, 1, True, 0, 4).tolist() == [0, 1, 2, 3]
    assert S.visible_with_prefix(6, 6, 5, True, 3, 4).tolist() == [3, 4, 5]
    assert S.visible_with_prefix(6, 6, 1, True, 2, 100).tolist() == [0, 1, 2, 3, 4, 5]
    assert np.allclose(S.shape_scores([3.0, 0.0], np.array([2, -2]), 2.0, 0.5),
                       [2 * np.tanh(1.5) - 1.0, -1.0])


def _ranges(cu, kv, prefix, hq, hkv, d, window, decode_rows_max=-1, bs=16):
    info, pre, dec, grp = ua.ua_schedule(cu, kv, hq, hkv, d, bs, max(1, max(kv) // bs + 1),
                                         window=window, decode_rows_max=decode_rows_max,
                                         prefix_lens=prefix)
    qpk = hq // hkv
    covered = {}
    for t in pre + dec:
        for r in range(t["row0"], t["row0"] + t["nrows"]):
            covered.setdefault((t["seq"], t["kv_head"], r), []).append((t["kv_lo"], t["kv_hi"]))
    for s in range(len(kv)):
        ql = cu[s + 1] - cu[s]
        for g in range(hkv):
            for r in range(ql * qpk):
                pieces = sorted(covered.pop((s, g, r)))
                for (_, a), (b, _) in zip(pieces, pieces[1:]):
                    assert a == b
                vis = S.visible_with_prefix(kv[s], ql, r // qpk, True, window, prefix[s])
                assert pieces[0][0] <= vis.min() and vis.max() < pieces[-1][1] <= kv[s]
    assert not covered
    return info, pre, dec


@pytest.mark.parametrize("seed", range(12))
def test_schedule_covers_every_key_a_row_sees(seed):
    rng = np.random.default_rng(seed)
    n = int(rng.integers(1, 6))
    ql = rng.integers(0, 200, n)
    kv = ql + rng.integers(0, 400, n)
    prefix = rng.integers(0, 500, n)
    cu = [0] + np.cumsum(ql).tolist()
    _ranges(cu, kv.tolist(), prefix.tolist(), 8, 2, [64, 128, 192, 96][seed % 4],
            int(rng.choice([0, 50])), decode_rows_max=int(rng.choice([-1, 0])))


def test_schedule_reads_no_further_than_rows_see():
    # 300 tokens, prefix 200: tiles of whole tokens (qpk 4) end at the prefix or at their last row
    _, pre, _ = _ranges([0, 300], [300], [200], 4, 1, 128, 0)
    assert sorted(r for t in pre for r in range(t["row0"], t["row0"] + t["nrows"])) == list(range(1200))
    for t in pre:
        assert (t["kv_lo"], t["kv_hi"]) == (0, max(200, (t["row0"] + t["nrows"] - 1) // 4 + 1))
    assert {t["kv_hi"] for t in pre} > {200, 300}
    # prefix 0 is the causal schedule
    for f in ("kv_lo", "kv_hi", "row0"):
        a = [t[f] for t in ua.ua_schedule([0, 300], [300], 4, 1, 128, 16, 20, prefix_lens=[0])[1]]
        assert a == [t[f] for t in ua.ua_schedule([0, 300], [300], 4, 1, 128, 16, 20)[1]]


@pytest.mark.parametrize("d", [32, 64, 96, 128, 160, 192, 224, 256])
def test_prompts_with_a_prefix_have_a_prefill_kernel_at_every_head_dim(d):
    info, pre, dec = _ranges([0, 40, 41], [90, 300], [7, 0], 4, 2, d, 0, decode_rows_max=32)
    assert info.num_prefill_tiles > 0 and {t["seq"] for t in dec} == {1}
    # but none where no kernel takes the group size, or the block size
    assert _ranges([0, 40], [90], [7], 5, 1, d, 0, decode_rows_max=32)[0].num_prefill_tiles == 0
    assert _ranges([0, 40], [90], [7], 4, 2, d, 0, decode_rows_max=32, bs=48)[0].num_prefill_tiles == 0
    # by default only where the decode kernel would take longer, at head dims without a kernel of their own
    own = d in (64, 128, 192, 256)
    few, many = ([0, 40], [90], [7]), ([0, 900, 1900], [2500, 2500], [7, 7])
    assert (_ranges(*few, 4, 2, d, 0)[0].num_prefill_tiles > 0) == own
    assert _ranges(*many, 8, 4, d, 0)[0].num_prefill_tiles > 0
    assert (_ranges(*many, 8, 4, d, 3)[0].num_prefill_tiles > 0) >= own


def test_prefix_refusals():
    with pytest.raises(ua.UAError) as e:
        ua.ua_schedule([0, 4], [4], 4, 4, 64, 16, 1, prefix_lens=[-1])
    assert e.value.status == ua.UA_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ua.ua_schedule([0, 4], [4], 4, 4, 64, 16, 1, prefix_lens=[1, 2])
    with pytest.raises(ValueError):
        ua.ua_schedule([0, 4], [4], 4, 4, 64, 16, 1, causal=0, prefix_lens=[1])
    info = ua.ua_plan_info()
    i32 = lambda *v: (ctypes.c_int32 * len(v))(*v)  # noqa: E731
    assert ua.lib().ua_schedule_prefix(i32(0, 4), i32(4), None, 1, 4, 4, 64, 16, 1, 0, 0, 0, 0, -1,
                                       ctypes.byref(info), None, 0, None, 0, None, 0) == ua.UA_ERR_INVALID_ARG
    # an empty batch needs no prefix
    assert ua.lib().ua_schedule_prefix(None, None, None, 0, 4, 4, 64, 16, 1, 0, 0, 0, 0, -1,
                                       ctypes.byref(info), None, 0, None, 0, None, 0) == ua.UA_OK


def test_scores_need_a_plan():
    assert ua.lib().ua_plan_set_scores(None, 0.0, None) == ua.UA_ERR_INVALID_ARG


def test_a_prefix_of_any_length_reaches_the_last_key():
    args = ([0, 40], [90], 4, 2, 64, 16, 6)
    for far in (90, 2 ** 31 - 1, 2 ** 31 + 5, 2 ** 40):
        assert ua.ua_schedule(*args, prefix_lens=[far])[1:] == ua.ua_schedule(*args, prefix_lens=[90])[1:]


@pytest.mark.parametrize("d", [64, 128, 160, 192, 256])
def test_prefill_tiles_have_one_query_tile_where_that_fills_more_sms(d):
    """One query tile (128 rows) at the wide head dims, and for prompts alone
    that leave half of the SMs without a tile of two; two otherwise."""
    def rows(cu, kv):
        bounds = [cu, kv, 32, 8, d, 16, 700]
        pre = ua.ua_schedule(*bounds, prefix_lens=[0] * len(kv))[1]
        return max(t["nrows"] for t in pre)
    assert rows([0, 576], [576]) == 128                     # 9 tiles of 256 rows a head, 72 in all
    assert rows([0, 600], [600]) == (128 if d > 128 else 256)   # 80 of 152
    assert rows([0, 576, 577], [576, 10000]) == (128 if d > 128 else 256)  # a decode step beside it


def test_cap_polynomial_keeps_its_error_bound():
    """The kernels' odd polynomial for tanh, in binary32 as they evaluate it (each multiply-add rounded
    once), on |a| <= 1/2: 5.5e-7 by its fit, four roundings of at most 2^-24 each by Horner's steps,
    whose later terms are below a quarter of the first."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(ua.__file__), "csrc", "score_shape.cuh")).read()
    coef = [float(re.search(rf"\ba{i} = c \* (-?[0-9.]+)f", src).group(1)) for i in range(4)]
    f = np.float32
    a = np.linspace(-0.5, 0.5, 200001)
    a = a[np.abs(a) > 1e-6].astype(f)
    fma = lambda x, y, z: f(x.astype(np.float64) * y + z)  # noqa: E731
    sq = f(a * a)
    poly = fma(fma(fma(np.full_like(a, f(coef[3])), sq, f(coef[2])), sq, f(coef[1])), sq, f(coef[0]))
    got, exact = f(a * poly).astype(np.float64), np.tanh(a.astype(np.float64))
    assert np.max(np.abs(got / exact - 1)) <= 5.5e-7 + 4 * 2.0 ** -24
