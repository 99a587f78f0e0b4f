"""Plans at the head dims whose shaped prompts run in a padded prefill kernel:
what such a plan costs before its scores are shaped, and when they are."""
import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
from oracle import scores as S
from paged_kv_attention_unified_gb300 import torch_utils as tu

from _helpers import as_f64

pytestmark = pytest.mark.gpu

GIB = 1 << 30


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


def _free():
    torch.cuda.synchronize()
    return torch.cuda.mem_get_info()[0]


def _long_prompts(num_seqs, kv_len):
    """Sequences of 40 new tokens, 8 heads of 96 over an e4m3 cache: a staging copy takes 3 KiB a key."""
    return ua.Plan([40 * i for i in range(num_seqs + 1)], [kv_len] * num_seqs, 8, 8, 96, 16, kv_len // 16,
                   kv_dtype=ua.UA_KV_FP8_E4M3)


def test_a_plain_plan_has_no_staging_copy():
    """24 x 131072 keys: 9 GiB of staging, of which earlier plans can have left 1 GiB in the pool
    (it may hold more until a synchronisation trims it)."""
    torch.zeros(1, device="cuda")
    before = _free()
    with _long_prompts(24, 131072) as plan:
        assert plan.info.num_prefill_tiles == 0
        assert before - _free() < GIB
        plan.set_scores(30.0)
        assert plan.info.num_prefill_tiles > 0
        assert before - _free() > 7 * GIB


def test_a_plan_outlives_scores_that_memory_is_wanting_for():
    """A staging copy larger than the GPU: the call is refused, the plan stays plain, and nothing
    of the failure is left for later calls."""
    with _long_prompts(1, 2 ** 27) as plan:  # 384 GiB
        lists = plan.info.num_decode_tiles
        for _ in range(2):
            with pytest.raises(ua.UAError) as e:
                plan.set_scores(30.0)
            assert e.value.status == ua.UA_ERR_CUDA
            assert (plan.info.num_prefill_tiles, plan.info.num_decode_tiles) == (0, lists)
        plan.set_scores()
        case = W.make_case("after", [1, 40], [90, 40], 4, 2, 64, 16, seed=1)
        b = tu.to_device(case)
        with tu.make_plan(b) as other:
            tu.forward(other, b)
            assert other.last_device_error() == 0
        assert plan.last_device_error() == 0


def _within(got, case, **shape):
    """The bound of tests/test_gpu_scores.py over a bf16 cache."""
    r = case.raw()
    exp, spread = S.paged_attention_shaped(r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"],
                                           r["kv_lens"], r["block_tables"], case.block_size, case.scale,
                                           causal=case.causal, window=case.window, **shape)
    tol = 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * (1 + 2.0 ** -8) * spread + 1e-30
    return bool(np.all(np.abs(as_f64(got) - exp) <= tol))


def _case(seed=2):
    return W.make_case("twin", [150, 1, 70], [200, 900, 400], 4, 2, 96, 16, seed=seed)


def test_settings_made_before_the_scores_hold_for_them():
    case = _case()
    b = tu.to_device(case)
    with tu.make_plan(b, decode_rows_max=32) as plan:
        plan.set_unified_max(0.0)
        ua.ua_plan_set_prefill_ctas(plan.handle, 1)
        ua.ua_plan_set_profiling(plan.handle, True)
        plan.set_scores(12.0)
        assert plan.info.num_prefill_tiles > 0
        out = tu.forward(plan, b)
        times = ua.ua_plan_kernel_times(plan.handle)
        assert times["prefill"][1] == 1 and times["decode"][1] == 1
        assert _within(out, case, softcap=12.0)
        assert plan.last_device_error() == 0


def test_profiling_from_before_the_first_shaped_forward():
    """Enabled after the scores are shaped: the spans are reset before the kernels write them."""
    b = tu.to_device(_case(8))
    for _ in range(10):
        with tu.make_plan(b, decode_rows_max=32) as plan:
            plan.set_scores(12.0)
            ua.ua_plan_set_profiling(plan.handle, True)
            tu.forward(plan, b)
            times = ua.ua_plan_kernel_times(plan.handle)
            for kind in ("prefill", "decode"):
                assert times[kind][1] == 1 and 0 < times[kind][0] < 1000, times


def test_scores_shaped_while_the_gpu_is_busy_and_used_on_another_stream():
    """The second schedule's lists are there before a forward on any stream reads them."""
    case = _case(3)
    b = tu.to_device(case)
    made, used = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with tu.make_plan(b, decode_rows_max=32, stream=made) as plan:
            used.wait_stream(made)
            with torch.cuda.stream(made):
                torch.cuda._sleep(20_000_000)
            plan.set_scores(9.0)
            out = b.new_out()
            tu.forward(plan, b, out, stream=used)
            tu.forward(plan, b, out, stream=used)
            used.synchronize()
            assert _within(out, case, softcap=9.0)
            assert plan.last_device_error() == 0


@pytest.mark.parametrize("forward_before", [False, True])
def test_scores_shaped_while_a_stream_is_captured(forward_before):
    """The second schedule is made outside the capture; the graph that was being captured runs it."""
    case = _case(4)
    b = tu.to_device(case)
    side = torch.cuda.Stream()
    with tu.make_plan(b, decode_rows_max=32, stream=side) as plan:
        out = b.new_out()
        if forward_before:
            tu.forward(plan, b, out, stream=side)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            plan.set_scores(9.0)
            tu.forward(plan, b, out, stream=side)
        out.fill_(float("nan"))
        for _ in range(2):
            graph.replay()
        torch.cuda.synchronize()
        assert _within(out, case, softcap=9.0)
        assert plan.last_device_error() == 0


def test_a_plan_is_destroyed_right_after_its_scores_are_shaped():
    b = tu.to_device(_case(5))
    for _ in range(20):
        plan = tu.make_plan(b, decode_rows_max=32)
        plan.set_scores(9.0)
        plan.close()
    torch.cuda.synchronize()


@pytest.mark.parametrize("through", ["plan", "current", "helper", "closed"])
def test_slopes_given_back_while_a_forward_on_another_stream_reads_them(through):
    """The plan gives the slopes' memory back when its scores change (or it ends); a forward that is
    still to run on another stream has them all the same."""
    case = W.make_case("held", [1, 120], [300, 200], 4, 2, 128, 16, seed=6)
    b = tu.to_device(case)
    values, side = [0.5, 0.25, 0.1, 0.0], torch.cuda.Stream()
    out = b.new_out()
    torch.cuda.synchronize()
    with tu.make_plan(b) as plan:
        slopes = torch.tensor(values, device="cuda")
        at = slopes.data_ptr()
        plan.set_scores(0.0, slopes)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(50_000_000)
        if through == "helper":
            tu.forward(plan, b, out, stream=side)
        else:
            with torch.cuda.stream(side if through == "current" else None):
                plan.forward(b.q, b.k_cache, b.v_cache, out, b.cu_query_lens, b.kv_lens, b.block_tables,
                             b.num_blocks, b.max_q, b.max_kv, b.scale,
                             stream=None if through == "current" else side)
        del slopes
        if through == "closed":
            plan.close()
            del plan
        else:
            plan.set_scores()
        others = [torch.full((4,), 100.0, device="cuda") for _ in range(50)]
        torch.cuda.synchronize()
    assert _within(out, case, slopes=values)
    assert at and len(others) == 50


def test_biased_forwards_on_every_kind_of_stream():
    """None, the default stream, torch streams and raw handles, once and again, and captured."""
    case = W.make_case("kinds", [1, 120], [300, 200], 4, 2, 128, 16, seed=7)
    b = tu.to_device(case)
    values, side = [0.5, 0.25, 0.1, 0.0], torch.cuda.Stream()
    with tu.make_plan(b) as plan:
        plan.set_scores(0.0, torch.tensor(values, device="cuda"))
        torch.cuda.synchronize()
        for stream in (None, torch.cuda.default_stream(), side, side.cuda_stream, 0,
                       type("Handle", (), {"cuda_stream": side.cuda_stream})(), torch.cuda.ExternalStream(side.cuda_stream)) * 2:
            out = b.new_out()
            torch.cuda.synchronize()
            tu.forward(plan, b, out, stream=stream)
            torch.cuda.synchronize()
            assert _within(out, case, slopes=values)
        slopes = torch.tensor(values, device="cuda")
        plan.set_scores(0.0, slopes)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            tu.forward(plan, b, out)
        plan.set_scores()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert _within(out, case, slopes=values)
