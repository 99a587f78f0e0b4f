"""Distance biases of any finite slope against the fp64 oracle: steep ones, whose
products with a distance leave the range or the precision of binary32, and
negative ones over long contexts, whose largest scores carry the largest bias.

The bound is that of tests/test_gpu_scores.py: it grants the scores' arithmetic
2^-10 of a weight, so that a bias may not cost the scores their precision.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
from paged_kv_attention_unified_gb300 import torch_utils as tu

from _helpers import as_f64
from test_gpu_scores import _bound, _check, _expected, _plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


HUGE = float(np.finfo(np.float32).max)
STEEP = {"steep": [1e4, 1e7, 1e12, HUGE], "negative": [-1e3, -1e5, -1e12, -HUGE], "mild_negative": [-0.5, -3.0, -30.0, 2.0]}
KERNELS = [(64, W.BF16), (96, W.BF16), (128, W.BF16), (128, W.FP8), (192, W.BF16), (256, W.BF16)]


@pytest.mark.parametrize("slopes", STEEP)
@pytest.mark.parametrize("cap", [0.0, 15.0])
@pytest.mark.parametrize("d,dtype", KERNELS)
def test_prompts(d, dtype, cap, slopes):
    case = W.make_case(f"slope_{slopes}_{d}", [150, 40], [700, 300], 4, 2, d, 16, kv_dtype=dtype, seed=50)
    info = _check(case, cap=cap, slopes=STEEP[slopes], decode_rows_max=0)
    assert info.num_prefill_tiles > 0 and info.num_decode_tiles == 0


@pytest.mark.parametrize("slopes", STEEP)
@pytest.mark.parametrize("d,dtype", [(64, W.BF16), (128, W.FP8), (224, W.BF16)])
def test_decode(d, dtype, slopes):
    case = W.make_case(f"dslope_{slopes}_{d}", [1, 2, 3], [1, 900, 333], 4, 1, d, 16, kv_dtype=dtype, seed=51)
    _check(case, slopes=STEEP[slopes], decode_rows_max=10 ** 6)
    _check(case, slopes=STEEP[slopes], decode_rows_max=10 ** 6, num_splits=7)


@pytest.mark.parametrize("slopes", STEEP)
@pytest.mark.parametrize("d", [64, 192])
@pytest.mark.parametrize("kind", ["window", "prefix", "open"])
def test_masks(kind, d, slopes):
    """The farthest visible key is the window's first, one of the prefix, or at either end."""
    case = W.make_case(f"mslope_{kind}_{d}", [1, 150, 60], [401, 350, 120], 4, 2, d, 16, seed=52,
                       window=100 if kind == "window" else 0, causal=kind != "open")
    _check(case, slopes=STEEP[slopes], prefix=[300, 340, 0] if kind == "prefix" else None)


@pytest.mark.parametrize("slopes", STEEP)
@pytest.mark.parametrize("d,rows_max", [(64, 0), (128, 0), (256, 0), (128, 100)])
def test_long_contexts(d, rows_max, slopes):
    """Far tiles' references are huge numbers that the nearer keys then leave behind, or the other way round."""
    case = W.make_case(f"lslope_{slopes}_{d}", [3, 20], [30011, 5000], 4, 4, d, 16, seed=53)
    _check(case, slopes=STEEP[slopes], decode_rows_max=rows_max)


@pytest.mark.parametrize("slopes", STEEP)
def test_fp8_products(slopes):
    """One key has all of the weight, or few: e4m3 weights against a reference that the bias cannot
    push away. Queries that are exact e4m3 values under their row's scale."""
    case = W.make_case(f"f8slope_{slopes}", [200, 140], [260, 3000], 4, 2, 128, 16, kv_dtype=W.FP8, seed=54)
    q = (torch.randn(case.q.shape, generator=torch.Generator().manual_seed(5)).clamp(-1.75, 1.75) * 256)
    q = (q.to(torch.float8_e4m3fn).float() / 256).to(torch.bfloat16)
    q[..., 0] = 1.75
    case.q.copy_(q)
    exp, _, rows = _expected(case, rows=True, slopes=STEEP[slopes])
    b = tu.to_device(case)
    with _plan(b, decode_rows_max=0, slopes=STEEP[slopes]) as plan:
        ua.ua_plan_set_fp8_products(plan.handle, True)
        got = as_f64(tu.forward(plan, b))
        assert plan.last_device_error() == 0
    for (tok, h), (_, p, v) in rows.items():
        e = p / p.max()  # half a step of 2^-4, or 2^-10 below 2^-6
        tol = (np.maximum(2.0 ** -4 * e, 2.0 ** -10) + 2.0 ** -10 * e) @ np.abs(v) / e.sum()
        assert np.all(np.abs(got[tok, h] - exp[tok, h]) <= tol + 2.0 ** -8 * (np.abs(exp[tok, h]) + tol))


def test_unified_max():
    case = W.make_case("uslope", [1, 2], [900, 333], 4, 2, 128, 16, seed=55)
    b = tu.to_device(case)
    for slopes in STEEP.values():
        exp, spread = _expected(case, slopes=slopes)
        with _plan(b, slopes=slopes) as plan:
            plan.set_unified_max(0.0)
            got = as_f64(tu.forward(plan, b))
        assert np.all(np.abs(got - exp) <= _bound(case, exp, spread))
