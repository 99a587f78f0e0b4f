"""GPU parity of shaped scores (cap, distance bias, prefix mask) against the
fp64 oracle, in every kernel that applies them, and their refusals.

Error bound of one output element, with p_t the softmax weights and A = sum_t
p_t |v_t|: the weights are rounded to bf16 (2^-8 of each; f16 for decode over
an e4m3 cache, less), the denominator sums them unrounded, and the score
arithmetic (binary32 dot products of up to 256 terms, the cap's few 2^-24 of at
most 50, exp2) changes a weight by less than 2^-10 of itself. So A (2^-8 +
2^-10) before the output rounding of 2^-8 |out|. f16 weights below 2^-14 have
an absolute error of 2^-25, against a denominator of at least 1 (every kernel's
reference lies at or below the row's maximum): kv_len 2^-25 max |v| more.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
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


def _slopes(hq):
    return [2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]


def _plan(b, prefix=None, cap=0.0, slopes=None, num_splits=0, decode_rows_max=-1, stream=None):
    plan = ua.Plan(b.cu_host, b.kv_host, b.num_q_heads, b.num_kv_heads, b.head_dim, b.block_size,
                   int(b.block_tables.shape[1]), kv_dtype=b.kv_dtype, causal=b.causal,
                   window=b.window, num_splits=num_splits, decode_rows_max=decode_rows_max,
                   prefix_lens=prefix, stream=stream)
    plan.set_scores(cap, None if slopes is None else torch.tensor(slopes, device="cuda"))
    return plan


def _expected(case, prefix=None, cap=0.0, slopes=None, rows=False):
    r = case.raw()
    return S.paged_attention_shaped(r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"],
                                    r["kv_lens"], r["block_tables"], case.block_size, case.scale,
                                    kv_dtype=case.kv_dtype, k_scale=case.k_scale,
                                    v_scale=case.v_scale, causal=case.causal, window=case.window,
                                    softcap=cap, slopes=slopes, prefix_lens=prefix, with_probs=rows)


def _bound(case, exp, spread):
    vmax = 10.0 if case.kv_dtype == W.BF16 else 448.0 * case.v_scale
    tail = 0.0 if case.kv_dtype == W.BF16 else max(case.kv_lens.tolist() or [0]) * 2.0 ** -25 * vmax
    return 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * (1 + 2.0 ** -8) * spread + tail + 1e-30


def _check(case, prefix=None, cap=0.0, slopes=None, **plan_args):
    b = tu.to_device(case)
    with _plan(b, prefix, cap, slopes, **plan_args) as plan:
        info = plan.info
        out = torch.full(b.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        tu.forward(plan, b, out)
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0
    exp, spread = _expected(case, prefix, cap, slopes)
    got = as_f64(out)
    assert np.all(np.isfinite(got))
    excess = np.abs(got - exp) - _bound(case, exp, spread)
    assert excess.max(initial=-1.0) <= 0, f"{case.name}: {excess.max()} over the bound"
    return info


SHAPES = {  # cap, bias, prefix
    "cap": (30.0, False, False), "bias": (0.0, True, False), "prefix": (0.0, False, True),
    "cap_bias": (5.0, True, False), "all": (20.0, True, True),
}


def _shape(name, case, seed=0):
    cap, bias, prefix = SHAPES[name]
    rng = np.random.default_rng(seed)
    return dict(cap=cap, slopes=_slopes(case.num_q_heads) if bias else None,
                prefix=[int(rng.integers(0, kv + 20)) for kv in case.kv_lens.tolist()]
                if prefix else None)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,dtype,hq,hkv,bs", [
    (128, W.BF16, 8, 2, 16), (128, W.FP8, 16, 2, 32), (64, W.BF16, 4, 4, 16), (64, W.FP8, 8, 1, 16),
    (32, W.BF16, 5, 1, 64), (96, W.BF16, 6, 2, 16), (160, W.FP8, 4, 2, 16), (192, W.BF16, 4, 2, 16),
    (224, W.BF16, 4, 4, 16), (256, W.FP8, 8, 4, 128), (256, W.BF16, 3, 1, 16)])
def test_decode(shape, d, dtype, hq, hkv, bs):
    """Short queries in the decode kernel: odd lengths, one key, unused page slots poisoned."""
    case = W.make_case(f"dec_{shape}_{d}_{dtype}", [1, 1, 3, 1, 2], [1, 17, 40, 333, 700], hq, hkv, d,
                       bs, kv_dtype=dtype, seed=d, poison=True)
    info = _check(case, **_shape(shape, case), decode_rows_max=10 ** 6)
    assert info.num_prefill_tiles == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [W.BF16, W.FP8])
def test_decode_splits(shape, dtype):
    case = W.make_case(f"spl_{shape}", [1, 2], [900, 2001], 8, 2, 128, 16, kv_dtype=dtype, seed=7)
    info = _check(case, **_shape(shape, case), num_splits=9)
    assert info.num_combine_groups > 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,dtype,hq,hkv,bs", [
    (128, W.BF16, 8, 2, 16), (128, W.BF16, 2, 2, 128), (128, W.FP8, 8, 2, 16), (64, W.BF16, 4, 4, 32),
    (64, W.FP8, 4, 1, 16), (192, W.BF16, 4, 2, 16), (192, W.FP8, 2, 2, 16), (256, W.BF16, 4, 1, 64),
    (256, W.BF16, 2, 2, 128)])
def test_prefill(shape, d, dtype, hq, hkv, bs):
    case = W.make_case(f"pre_{shape}_{d}_{dtype}", [65, 200, 131, 300], [65, 257, 600, 301], hq, hkv, d,
                       bs, kv_dtype=dtype, seed=d + 1, poison=True)
    info = _check(case, **_shape(shape, case), decode_rows_max=0)
    assert info.num_decode_tiles == 0


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_window_beside_the_shapes(shape, d):
    case = W.make_case(f"win_{shape}_{d}", [1, 150, 2, 90], [400, 350, 129, 90], 4, 2, d, 16, seed=21,
                       window=100)
    info = _check(case, **_shape(shape, case))
    assert info.num_prefill_tiles > 0 and info.num_decode_tiles > 0


@pytest.mark.parametrize("shape", ["cap", "bias", "cap_bias"])
@pytest.mark.parametrize("d,dtype", [(128, W.BF16), (128, W.FP8), (192, W.BF16)])
def test_without_causal_mask_the_bias_falls_both_ways(shape, d, dtype):
    case = W.make_case(f"nc_{shape}_{d}", [1, 140, 5], [70, 300, 33], 4, 2, d, 16, kv_dtype=dtype,
                       seed=22, causal=False)
    _check(case, **_shape(shape, case))


def test_group_size_that_no_prefill_kernel_takes():
    case = W.make_case("qpk5", [80, 3], [300, 40], 10, 2, 128, 16, seed=23)
    info = _check(case, **_shape("all", case))
    assert info.num_prefill_tiles == 0


@pytest.mark.parametrize("scale", [-0.09, 3.0, 0.0, 1e30])
@pytest.mark.parametrize("d", [64, 128, 192])
def test_scales_of_either_sign_and_saturated_caps(scale, d):
    """Scores far above the cap (and a huge scale) saturate at +-cap. Queries and keys are 0 or
    +-1: their products are exact, so a score is exactly 0 or far from it."""
    case = W.make_case(f"sat_{d}", [1, 70], [90, 120], 4, 2, d, 16, seed=24, scale=scale)
    for t in (case.q, case.k_cache):
        t.copy_(t.sign())
    _check(case, cap=2.0)


def test_large_and_small_caps():
    case = W.make_case("caps", [1, 90], [200, 300], 4, 2, 128, 16, seed=25)
    for cap in (ua.UA_MIN_SOFTCAP, 0.5, 1000.0):
        _check(case, cap=cap)


def test_bias_over_a_long_context():
    """Far keys underflow to weight zero and split pieces of nothing but those weigh nothing."""
    case = W.make_case("far", [1, 1], [20011, 9000], 4, 1, 64, 16, seed=26)
    _check(case, slopes=[0.9, 0.3, 0.01, 0.0], num_splits=16)


@pytest.mark.parametrize("phi", [0.0, 3.0, -50.0])
def test_unified_max_over_shaped_scores(phi):
    case = W.make_case("phi", [1, 1, 2], [300, 1000, 40], 8, 2, 128, 16, seed=27)
    b = tu.to_device(case)
    kw = _shape("all", case)
    exp, spread = _expected(case, **kw)
    with _plan(b, **kw) as plan:
        plan.set_unified_max(phi)
        got = as_f64(tu.forward(plan, b))
    assert np.all(np.abs(got - exp) <= _bound(case, exp, spread))


@pytest.mark.parametrize("shape", SHAPES)
def test_fp8_products(shape):
    """e4m3 products: queries that are exact e4m3 values under their row's scale (the largest
    1.75 = 448 / 256), so that only the weights' rounding is left: half a step of 2^-4, or 2^-10
    below 2^-6, of weights relative to a reference at or below the row's maximum."""
    case = W.make_case(f"f8p_{shape}", [200, 140], [260, 500], 4, 2, 128, 16, kv_dtype=W.FP8, seed=28)
    q = (torch.randn(case.q.shape, generator=torch.Generator().manual_seed(5)).clamp(-1.75, 1.75) * 256)
    q = (q.to(torch.float8_e4m3fn).float() / 256).to(torch.bfloat16)
    q[..., 0] = 1.75
    case.q.copy_(q)
    kw = _shape(shape, case)
    exp, _, rows = _expected(case, rows=True, **kw)
    b = tu.to_device(case)
    with _plan(b, decode_rows_max=0, **kw) as plan:
        ua.ua_plan_set_fp8_products(plan.handle, True)
        got = as_f64(tu.forward(plan, b))
        assert plan.last_device_error() == 0
    for (tok, h), (_, p, v) in rows.items():
        e = p / p.max()
        tol = (np.maximum(2.0 ** -4 * e, 2.0 ** -10) + 2.0 ** -10 * e) @ np.abs(v) / e.sum()
        assert np.all(np.abs(got[tok, h] - exp[tok, h]) <= tol + 2.0 ** -8 * (np.abs(exp[tok, h]) + tol))


def test_plain_scores_come_back_bit_for_bit():
    case = W.make_case("back", [1, 100, 2], [200, 300, 40], 8, 2, 128, 16, seed=29)
    b = tu.to_device(case)
    with _plan(b) as never, _plan(b, cap=10.0, slopes=_slopes(8)) as plan:
        want = tu.forward(never, b)
        shaped = tu.forward(plan, b)
        plan.set_scores()
        got = tu.forward(plan, b)
        assert not torch.equal(shaped, want)
        assert torch.equal(got, want)


def test_plans_of_different_shapes_on_two_streams():
    case = W.make_case("streams", [1, 300, 1], [2000, 600, 77], 8, 2, 128, 16, seed=30)
    b = tu.to_device(case)
    wants, plans, outs = [], [], []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for name, st in zip(("cap", "all"), streams):
        kw = _shape(name, case)
        wants.append(_expected(case, **kw))
        plans.append(_plan(b, stream=st, **kw))
        outs.append(b.new_out())
    torch.cuda.synchronize()
    for _ in range(5):
        for plan, st, out in zip(plans, streams, outs):
            tu.forward(plan, b, out, stream=st)
    torch.cuda.synchronize()
    for (exp, spread), out, plan in zip(wants, outs, plans):
        assert np.all(np.abs(as_f64(out) - exp) <= _bound(case, exp, spread))
        plan.close()


def test_captured_forward_replays_on_new_values():
    case = W.make_case("graph", [1, 200, 1], [300, 260, 77], 8, 2, 128, 16, seed=31)
    b = tu.to_device(case)
    kw = _shape("all", case)
    with _plan(b, **kw) as plan:
        out = tu.forward(plan, b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tu.forward(plan, b, out)
        case.q.copy_(case.q.flip(0))
        b.q.copy_(case.q)
        out.fill_(float("nan"))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        exp, spread = _expected(case, **kw)
        assert np.all(np.abs(as_f64(out) - exp) <= _bound(case, exp, spread))


def test_rows_behind_the_last_sequence_stay():
    case = W.make_case("behind", [3, 0, 70], [40, 0, 90], 4, 2, 64, 16, seed=32)
    b = tu.to_device(case)
    room = torch.full((case.q.shape[0] + 5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    with _plan(b, **_shape("all", case)) as plan:
        tu.forward(plan, b, room[:-5])
        torch.cuda.synchronize()
    assert torch.all(room[-5:] == 7.0)


def test_bad_page_under_a_shape_is_reported():
    case = W.make_case("badpage", [1, 100], [300, 200], 4, 2, 128, 16, seed=33)
    b = tu.to_device(case)
    b.block_tables[0, 3] = -5
    b.block_tables[1, 2] = b.num_blocks
    with _plan(b, **_shape("all", case)) as plan:
        tu.forward(plan, b)
        assert plan.last_device_error() == ua.UA_ERR_BOUNDS


@pytest.mark.parametrize("cap", [-1.0, float("nan"), float("inf"), 5000.0, 1e-4])
def test_caps_outside_their_range_are_refused(cap):
    case = W.make_case("ref", [1], [20], 4, 2, 64, 16)
    b = tu.to_device(case)
    with _plan(b, cap=8.0) as plan:
        want = tu.forward(plan, b)
        with pytest.raises(ua.UAError) as e:
            plan.set_scores(cap)
        assert e.value.status == ua.UA_ERR_INVALID_ARG
        assert torch.equal(tu.forward(plan, b), want)  # the refused call changed nothing


def test_slopes_that_are_no_device_floats_are_refused():
    case = W.make_case("ref2", [1], [20], 4, 2, 64, 16)
    b = tu.to_device(case)
    with _plan(b) as plan:
        for slopes in (torch.zeros(4), torch.zeros(4).pin_memory()):
            with pytest.raises(ua.UAError) as e:
                plan.set_scores(0.0, slopes)
            assert e.value.status == ua.UA_ERR_INVALID_ARG
        with pytest.raises(ua.UAError):
            ua.ua_plan_set_scores(plan.handle, 0.0, torch.zeros(8, device="cuda").data_ptr() + 2)
        for slopes in (torch.zeros(4, device="cuda", dtype=torch.bfloat16),
                       torch.zeros(3, device="cuda"), torch.zeros(8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                plan.set_scores(0.0, slopes)
        tu.forward(plan, b)
        assert plan.last_device_error() == 0


@pytest.mark.parametrize("d,dtype", [(64, W.BF16), (128, W.BF16), (128, W.FP8), (192, W.BF16)])
@pytest.mark.parametrize("cap", [0.0, 15.0])
def test_steep_negative_and_zero_slopes(d, dtype, cap):
    """Slopes that move the reference in every key tile, that favour far keys, and none."""
    case = W.make_case(f"steep_{d}", [150, 1, 40], [700, 900, 300], 4, 2, d, 16, kv_dtype=dtype, seed=34)
    _check(case, cap=cap, slopes=[5.0, -0.02, 0.0, 0.3])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [64, 128, 256])
def test_whatever_unused_slots_hold(shape, d):
    """Slots past the last key hold infinities and the type's largest values: of no consequence,
    neither to the result nor to which way a key tile's scores are taken."""
    case = W.make_case(f"junk_{shape}_{d}", [90, 1, 3], [333, 45, 100], 4, 2, d, 64, seed=35)
    case.q.abs_()
    bs = case.block_size
    for cache in (case.k_cache, case.v_cache):
        for s, kv in enumerate(case.kv_lens.tolist()):
            last = int(case.block_tables[s, (kv - 1) // bs])
            cache[last, kv % bs:] = float("inf")
            cache[last, kv % bs::2] = torch.finfo(torch.bfloat16).max
    _check(case, **_shape(shape, case))


def test_scores_on_both_sides_of_half_the_cap():
    """Some key tiles of a prompt exceed half the cap, others do not, on either side of zero."""
    for d in (64, 128, 256):
        case = W.make_case(f"mix_{d}", [300], [700], 4, 2, d, 16, seed=36)
        case.k_cache[int(case.block_tables[0, 9])] *= 8      # keys 144 .. 159
        case.k_cache[int(case.block_tables[0, 30])] *= -20   # keys 480 .. 495
        _check(case, cap=6.0)
        _check(case, cap=6.0, slopes=[0.05, 0.01, 0.0, 0.2])


def test_one_plan_changes_its_scores_between_forwards():
    case = W.make_case("changes", [1, 130], [200, 400], 4, 2, 128, 16, seed=37)
    b = tu.to_device(case)
    with _plan(b) as plan:
        for cap, slopes in ((0.0, None), (9.0, None), (0.0, _slopes(4)), (9.0, _slopes(4)), (0.0, None)):
            plan.set_scores(cap, None if slopes is None else torch.tensor(slopes, device="cuda"))
            exp, spread = _expected(case, cap=cap, slopes=slopes)
            assert np.all(np.abs(as_f64(tu.forward(plan, b)) - exp) <= _bound(case, exp, spread))


@pytest.mark.parametrize("dtype", [W.BF16, W.FP8])
def test_a_prompt_in_chunks_sees_its_prefix_as_it_comes(dtype):
    """The prefix reaches as far as the keys do; a chunk behind it is causal."""
    full = W.make_case("chunks", [400], [400], 4, 2, 128, 16, kv_dtype=dtype, seed=38)
    for begin, end in ((0, 150), (150, 151), (151, 400)):
        case = W.make_case("chunk", [end - begin], [end], 4, 2, 128, 16, kv_dtype=dtype, seed=38,
                           num_blocks=full.num_blocks)
        case.q.copy_(full.q[begin:end])
        _check(case, prefix=[220])


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,dtype,hq,hkv,bs", [
    (32, W.BF16, 4, 2, 16), (32, W.FP8, 8, 2, 32), (96, W.BF16, 4, 1, 16), (96, W.FP8, 2, 2, 128),
    (160, W.BF16, 4, 2, 64), (160, W.FP8, 4, 4, 16), (224, W.BF16, 2, 1, 16), (224, W.FP8, 8, 4, 32)])
def test_prompts_at_the_other_head_dims(shape, d, dtype, hq, hkv, bs):
    """Shaped scores have a prefill kernel at every head dim (operands padded with zeros), beside
    decoding sequences; unused slots poisoned."""
    case = W.make_case(f"pad_{shape}_{d}_{dtype}", [200, 1, 131, 2], [257, 300, 600, 40], hq, hkv, d, bs,
                       kv_dtype=dtype, seed=d + 2, poison=True)
    info = _check(case, **_shape(shape, case), decode_rows_max=32)
    assert info.num_prefill_tiles > 0 and info.num_decode_tiles > 0


def test_plans_at_the_other_head_dims_switch_with_their_scores():
    """The lists, the settings, the errors and the timing of a plan follow its scores."""
    case = W.make_case("switch", [150, 1], [200, 90], 4, 2, 96, 16, seed=39)
    b = tu.to_device(case)
    with _plan(b, decode_rows_max=32) as never, _plan(b, decode_rows_max=32) as plan:
        want = tu.forward(never, b)
        assert plan.info.num_prefill_tiles == 0
        for _ in range(2):
            plan.set_scores(12.0)
            assert plan.info.num_prefill_tiles > 0
            ua.ua_plan_set_prefill_ctas(plan.handle, 1)
            plan.set_unified_max(0.0)
            exp, spread = _expected(case, cap=12.0)
            assert np.all(np.abs(as_f64(tu.forward(plan, b)) - exp) <= _bound(case, exp, spread))
            plan.set_scores()
            plan.set_unified_max(None)
            assert plan.info.num_prefill_tiles == 0
            assert torch.equal(tu.forward(plan, b), want)
        plan.set_scores(12.0)
        ua.ua_plan_set_profiling(plan.handle, True)
        tu.forward(plan, b)
        times = ua.ua_plan_kernel_times(plan.handle)
        assert times["prefill"][1] == 1 and times["decode"][1] == 1
        b.block_tables[0, 2] = b.num_blocks + 7
        tu.forward(plan, b)
        assert plan.last_device_error() == ua.UA_ERR_BOUNDS
        assert plan.last_device_error() == 0


@pytest.mark.parametrize("hkv,d,ql,kv", [
    (20, 128, [70, 40], [300, 90]),      # rows of several load rounds, few pages: sixteen blocks each
    (40, 64, [60] * 20, [700] * 20),     # the same, 120 pages: one block each
    (1, 64, [300, 50], [301, 1000])])    # rows of four lanes
def test_staging_of_e4m3_pages(hkv, d, ql, kv):
    """Prompts over an e4m3 cache at every way of sharing a staging page between blocks; pages and
    sequences end inside them, unused slots are poisoned."""
    case = W.make_case(f"stage_{hkv}_{d}", ql, kv, hkv, hkv, d, 32, kv_dtype=W.FP8, seed=40, poison=True)
    info = _check(case, cap=20.0, decode_rows_max=0)
    assert info.num_prefill_tiles > 0
    b = tu.to_device(case)
    b.block_tables[0, 1] = -3
    with _plan(b, cap=20.0, decode_rows_max=0) as plan:
        tu.forward(plan, b)
        assert plan.last_device_error() == ua.UA_ERR_BOUNDS


@pytest.mark.parametrize("d,dtype", [(96, W.BF16), (160, W.FP8)])
def test_captured_shaped_and_plain_forwards_of_one_plan(d, dtype):
    """Graphs of a plan's plain and shaped forwards, replayed in turn: each keeps the scores, lists
    and workspace it was captured with."""
    case = W.make_case(f"cap_{d}", [150, 1, 33], [200, 900, 64], 4, 2, d, 16, kv_dtype=dtype, seed=41)
    b = tu.to_device(case)
    slopes = torch.tensor(_slopes(4), device="cuda")
    with _plan(b, decode_rows_max=32) as plan:
        graphs, outs = [], []
        for cap, sl in ((0.0, None), (9.0, None), (9.0, slopes)):
            plan.set_scores(cap, sl)
            out = torch.empty_like(b.q)
            tu.forward(plan, b, out)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                tu.forward(plan, b, out, stream=torch.cuda.current_stream())
            graphs.append(g)
            outs.append(out)
        plan.set_scores()
        for i in (2, 0, 1, 2, 1, 0):
            outs[i].fill_(float("nan"))
            graphs[i].replay()
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0
    for out, (cap, sl) in zip(outs, ((0.0, None), (9.0, None), (9.0, _slopes(4)))):
        exp, spread = _expected(case, cap=cap, slopes=sl)
        assert np.all(np.abs(as_f64(out) - exp) <= _bound(case, exp, spread))
