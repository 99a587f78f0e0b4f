"""Attention over an e4m3 cache whose pages have value scales far apart, element by
element against the fp64 oracle: what a quiet page holds beside a loud one counts,
in the sum of the weights and in the elements that the loud page leaves at zero.

Bound of an element, of its own values alone (e_t: weights with the largest at 1):
  2^-8 |exact| + 1.01 sum_t (eps e_t + low) |v_t| / sum_t e_t + n 2^-127
eps: half a step of the weights' type (f16 in decode tiles 2^-11, bf16 in prefill
tiles 2^-8) and 2^-11 for the scores' errors; low: half a step of f16's subnormal
weights, 2^-25 (bf16 has binary32's range: 0). The sum's error is at most 2^-11
sum_t e_t, below 2^-8 |exact| / 8 with the bf16 output's own half step at 2^-9 at
most. 2^-127 a key: sums in binary32, in units of at most 2^22, round at 2^-149 of
those.
"""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import block_scales as B
from oracle import scores as S
from paged_kv_attention_unified_gb300 import torch_utils as tu

from _helpers import as_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


def _rows(case, ks, vs, staged, **shape):
    r = case.raw()
    return S.paged_attention_shaped(
        r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"], r["kv_lens"], r["block_tables"], case.block_size,
        case.scale, kv_dtype=W.FP8, causal=case.causal, window=case.window, k_scales=as_f64(ks), v_scales=as_f64(vs),
        staged=staged, with_probs=True, **shape)


def _forward(case, ks, vs, phi=None, **plan_args):
    b = tu.to_device(case)
    with tu.make_plan(b, **plan_args) as plan:
        plan.set_block_scales(ks.cuda(), vs.cuda())
        if phi is not None:
            plan.set_unified_max(phi)
        out = torch.full(b.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        tu.forward(plan, b, out)
        assert plan.last_device_error() == 0
        return as_f64(out), plan.info.num_prefill_tiles > 0


def _check(case, ks, vs, skip=(), phi=None, sinks=0, **plan_args):
    got, staged = _forward(case, ks, vs, phi, sink_tokens=sinks, **plan_args)
    _compare(case, got, staged, ks, vs, skip, sinks=sinks)


def _compare(case, got, staged, ks, vs, skip=(), **shape):
    """skip: tokens whose rows hold anything."""
    exp, _, rows = _rows(case, ks, vs, staged, **shape)
    eps, low = (2.0 ** -8 + 2.0 ** -11, 0.0) if staged else (2.0 ** -10, 2.0 ** -25)
    for (tok, h), (t, p, v) in rows.items():
        if tok in skip:
            continue
        e = p / p.max()
        tol = 1.01 * ((eps * e + low) @ np.abs(v)) / e.sum() + len(t) * 2.0 ** -127
        err = np.abs(got[tok, h] - exp[tok, h])
        assert np.all(err <= 2.0 ** -8 * np.abs(exp[tok, h]) + tol), (
            tok, h, err.max(), np.nanmax(err / (2.0 ** -8 * np.abs(exp[tok, h]) + tol + 1e-300)))


def _case(name, ql, kv, d, hq=4, hkv=2, bs=16, seed=0, **args):
    return W.make_case(name, ql, kv, hq, hkv, d, bs, kv_dtype=W.FP8, seed=seed, **args)


def _scales(case, v=2.0 ** -6):
    return tuple(torch.full((case.num_blocks, case.num_kv_heads), x) for x in (2.0 ** -7, v))


def _codes(case):
    return case.v_cache.view(torch.uint8)


@pytest.mark.parametrize("rows", [0, 10 ** 6])
@pytest.mark.parametrize("loud", [2.0 ** 10, 2.0 ** 26, 2.0 ** 27, 2.0 ** 30, 2.0 ** 60, 2.0 ** 100])
@pytest.mark.parametrize("zeros_first", [True, False])
def test_a_page_of_zeros_halves_the_weights(zeros_first, loud, rows):
    """Equal scores: a page of zeros under the least scale, as the append leaves it, has as much of the
    weight as a loud page (and each warp's page, each split piece's, has its own)."""
    for ql, kv, splits in (([1], [32], 0), ([2], [128], 0), ([1], [640], 3), ([40], [160], 0)):
        case = _case("zeros", ql, kv, 128, seed=1)
        case.k_cache[:] = case.k_cache[0, 0, 0]
        ks, vs = _scales(case)
        pages = case.block_tables[0, :kv[0] // 16].long()
        half = pages[:len(pages) // 2] if zeros_first else pages[len(pages) // 2:]
        vs[pages] = loud
        vs[half] = B.LEAST
        _codes(case)[half] = 0
        _check(case, ks, vs, decode_rows_max=rows, num_splits=splits)


@pytest.mark.parametrize("rows", [0, 10 ** 6])
@pytest.mark.parametrize("ratio", [4, 12, 18, 20, 24, 26, 60, 120, 190])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_loud_page_that_is_loud_in_half_of_the_dims(d, ratio, rows):
    """Its other dims are zeros: there the row's elements are the quiet pages'."""
    for at in (0, 3, 7):
        case = _case("half", [1, 3, 33], [128, 600, 133], d, seed=d + ratio)
        ks, vs = _scales(case, 2.0 ** min(100 - ratio, -6))
        for s in range(3):
            page = int(case.block_tables[s, at])
            vs[page] = 2.0 ** (min(100 - ratio, -6) + ratio)
            _codes(case)[page, :, :, : d // 2] = 0
        _check(case, ks, vs, decode_rows_max=rows)


@pytest.mark.parametrize("spread", [3, 10, 40, 100])
@pytest.mark.parametrize("d,hq,hkv,bs", [(32, 4, 2, 16), (64, 8, 2, 64), (96, 4, 1, 16), (128, 16, 2, 16),
                                         (128, 4, 2, 128), (160, 4, 2, 32), (192, 4, 2, 16), (224, 4, 4, 16),
                                         (256, 8, 2, 16)])
def test_every_page_has_its_own_scale_and_its_own_zeros(d, hq, hkv, bs, spread):
    case = _case("own", [1, 1, 2, 1], [900, 17, 333, 2000], d, hq, hkv, bs, seed=d + spread)
    g = torch.Generator().manual_seed(spread)
    ks, vs = _scales(case)
    vs = torch.exp2(((torch.rand(vs.shape, generator=g) * 2 - 1) * spread).round())
    zero = torch.rand(case.num_blocks, 1, hkv, d, generator=g) < 0.7
    _codes(case).masked_fill_(zero, 0)
    _check(case, ks, vs, decode_rows_max=10 ** 6)
    _check(case, ks, vs, decode_rows_max=10 ** 6, num_splits=5)
    _check(case, ks, vs * 0.75, decode_rows_max=10 ** 6, phi=0.0)  # (not powers of two)


def test_under_a_window_with_sinks():
    case = _case("sinks", [1, 2], [900, 2000], 128, seed=5, window=300)
    ks, vs = _scales(case)
    g = torch.Generator().manual_seed(5)
    vs = torch.exp2(((torch.rand(vs.shape, generator=g) * 2 - 1) * 60).round())
    _codes(case).masked_fill_(torch.rand(case.num_blocks, 1, 2, 128, generator=g) < 0.7, 0)
    _check(case, ks, vs, decode_rows_max=10 ** 6, sinks=20)


@pytest.mark.parametrize("ratio", [0.5, 1, 2, 8, 16, 64, 256, 4096])
def test_scales_that_rise_and_fall_from_page_to_page(ratio):
    """Ordinary spreads: the same relative precision on both sides of each of them."""
    case = _case("wave", [1] * 4, [16, 33, 700, 1500], 128, 8, 2, seed=6)
    ks, vs = _scales(case)
    for s in range(4):
        for i, page in enumerate(case.block_tables[s].tolist()):
            vs[page] = 2.0 ** -6 * ratio ** (i % 3)
    _check(case, ks, vs)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 0.0, -1.0, 1e-40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_block_without_a_usable_scale_spoils_only_the_rows_that_see_it(d, bad):
    """It lies in the tiles of rows that do not: behind their positions, or before their window."""
    for ql, kv, window, page, skip, rows in (
            (3, 33, 0, 2, (2,), 10 ** 6), (2, 49, 17, 1, (0,), 10 ** 6), (16, 700, 0, 43, range(4, 16), 10 ** 6),
            (200, 257, 0, 16, (199,), 0), (150, 256, 91, 0, (), 0), (150, 256, 92, 0, (0,), 0),
            (150, 256, 92, 0, (0,), 10 ** 6)):
        case = _case("bad", [ql], [kv], d, seed=d + kv, window=window)
        ks, vs = _scales(case)
        block = int(case.block_tables[0, page])
        for which in ((0,), (1,), (0, 1)):
            x = [ks.clone(), vs.clone()]
            for i in which:
                x[i][block] = bad
            got, staged = _forward(case, *x, decode_rows_max=rows)
            _compare(case, got, staged, ks, vs, skip)
