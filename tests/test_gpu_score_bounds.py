"""Prompts over an e4m3 cache against the bound of 16-bit floating weights, with
no absolute term: their staged keys meet bf16 weights, which keep their relative
precision below a reference that a rising distance bias has put up to 48 log2
units (and the slack of 8) above the row's maximum. A weight leaves bf16's
normal range only at 2^-126 of the reference, 2^-70 of the row's largest or
less, and kv_len of those are below 2^-50 of it.

Per output element, with A = sum_t p_t |v_t|: A (2^-8 + 2^-10) for the weights'
rounding and the scores' arithmetic, 2^-8 |out| for the output's, and kv_len
2^-70 max |v|.
"""
import numpy as np
import pytest
import torch

import workloads as W
from paged_kv_attention_unified_gb300 import torch_utils as tu

from _helpers import as_f64
from test_gpu_scores import SHAPES, _expected, _plan, _shape

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


@pytest.mark.parametrize("slopes", [None, [0.9, 0.06, 0.01, 3.0]])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 96, 128, 192, 256])
def test_staged_prompts(d, shape, slopes):
    case = W.make_case(f"bound_{shape}_{d}", [150, 70, 200], [1200, 333, 200], 4, 2, d, 16, kv_dtype=W.FP8, seed=60)
    kw = _shape(shape, case)
    if slopes is not None:
        kw["slopes"] = slopes
    b = tu.to_device(case)
    with _plan(b, decode_rows_max=0, **kw) as plan:
        assert plan.info.num_prefill_tiles > 0 and plan.info.num_decode_tiles == 0
        got = as_f64(tu.forward(plan, b))
        assert plan.last_device_error() == 0
    exp, spread = _expected(case, **kw)
    tol = 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * (1 + 2.0 ** -8) * spread
    tol += 1200 * 2.0 ** -70 * 448.0 * case.v_scale
    assert np.all(np.abs(got - exp) <= tol)


@pytest.mark.parametrize("splits", [1, 6])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,dtype", [(128, W.BF16), (128, W.FP8), (64, W.BF16)])
def test_a_call_repeats_itself_bit_for_bit(d, dtype, shape, splits):
    """Neither the order of the split pieces nor that of the tiles enters the result."""
    case = W.make_case(f"again_{shape}_{d}", [1, 2, 150, 1], [3000, 900, 400, 77], 8, 2, d, 16, kv_dtype=dtype, seed=61)
    b = tu.to_device(case)
    with _plan(b, num_splits=splits, **_shape(shape, case)) as plan:
        first = tu.forward(plan, b)
        for _ in range(10):
            assert torch.equal(tu.forward(plan, b).view(torch.int16), first.view(torch.int16))
