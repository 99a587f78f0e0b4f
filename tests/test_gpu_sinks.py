"""GPU parity of windowed attention with sinks against the fp64 oracle, in every
kernel, with every other mask and score shape, and over sessions whose unseen
pages have been given back. Bounds: tests/test_gpu_scores.py."""
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


def _plan(b, sinks, cap=0.0, slopes=None, prefix=None, **args):
    plan = tu.make_plan(b, prefix_lens=prefix, sink_tokens=sinks, **args)
    plan.set_scores(cap, None if slopes is None else torch.tensor(slopes, device="cuda"))
    return plan


def _expected(case, sinks, cap=0.0, slopes=None, prefix=None):
    r = case.raw()
    return S.paged_attention_shaped(r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"], r["kv_lens"],
                                    r["block_tables"], case.block_size, case.scale, kv_dtype=case.kv_dtype,
                                    k_scale=case.k_scale, v_scale=case.v_scale, causal=case.causal,
                                    window=case.window, softcap=cap, slopes=slopes, prefix_lens=prefix,
                                    sinks=sinks)


def _bound(case, exp, spread):
    vmax = 10.0 if case.kv_dtype == W.BF16 else 448.0 * case.v_scale
    tail = 0.0 if case.kv_dtype == W.BF16 else max(case.kv_lens.tolist()) * 2.0 ** -25 * vmax
    return 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * (1 + 2.0 ** -8) * spread + tail + 1e-30


def _give_back(case, sinks):
    """Entries of pages that hold only unseen keys point nowhere, and the pages hold NaN."""
    bs = case.block_size
    for s, (n, kv) in enumerate(zip(case.query_lens, case.kv_lens.tolist())):
        for page in range(-(-kv // bs)):
            if page * bs >= sinks and (page + 1) * bs <= kv - n - case.window + 1:
                blk = int(case.block_tables[s, page])
                case.block_tables[s, page] = -1 - page
                for cache in (case.k_cache, case.v_cache):
                    cache.view(torch.uint8)[blk] = 0x7F if case.kv_dtype == W.FP8 else 0xFF


def _check(case, sinks, gone=True, setup=None, shape=None, **plan_args):
    if gone:
        _give_back(case, sinks)
    shape = shape or {}
    b = tu.to_device(case)
    with _plan(b, sinks, **shape, **plan_args) as plan:
        info = plan.info
        out = torch.full(b.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        tu.forward(plan, b, out)
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0
    exp, spread = _expected(case, sinks, **shape)
    got = as_f64(out)
    assert np.all(np.isfinite(got))
    excess = np.abs(got - exp) - _bound(case, exp, spread)
    assert excess.max() <= 0, f"{case.name}: {excess.max()} over the bound"
    return info


DIMS = [(128, W.BF16, 8, 2, 16), (128, W.FP8, 16, 2, 32), (64, W.BF16, 4, 4, 16), (64, W.FP8, 8, 1, 16),
        (32, W.BF16, 5, 1, 64), (96, W.BF16, 6, 2, 16), (160, W.FP8, 4, 2, 16), (192, W.BF16, 4, 2, 16),
        (224, W.BF16, 4, 4, 16), (256, W.FP8, 8, 4, 128), (256, W.BF16, 4, 1, 16)]


@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 1), (40, 90), (300, 16), (128, 129)])
@pytest.mark.parametrize("d,dtype,hq,hkv,bs", DIMS)
def test_decode(d, dtype, hq, hkv, bs, window, sinks):
    case = W.make_case(f"dec_{d}_{dtype}", [1, 1, 3, 1, 2], [1, 17, 40, 333, 1700], hq, hkv, d, bs,
                       kv_dtype=dtype, seed=d, poison=True, window=window)
    info = _check(case, sinks, decode_rows_max=10 ** 6)
    assert info.num_prefill_tiles == 0


@pytest.mark.parametrize("dtype", [W.BF16, W.FP8])
@pytest.mark.parametrize("window,sinks,splits", [(700, 4, 9), (33, 500, 128), (1000, 48, 2)])
def test_decode_splits(dtype, window, sinks, splits):
    case = W.make_case("spl", [1, 2], [1900, 2001], 8, 2, 128, 16, kv_dtype=dtype, seed=7, window=window)
    info = _check(case, sinks, num_splits=splits)
    assert info.num_combine_groups > 0


@pytest.mark.parametrize("window,sinks", [(100, 4), (1, 1), (60, 200), (130, 128), (33, 129), (400, 64)])
@pytest.mark.parametrize("d,dtype,hq,hkv,bs", [
    (128, W.BF16, 8, 2, 16), (128, W.BF16, 2, 2, 128), (128, W.FP8, 8, 2, 16), (64, W.BF16, 4, 4, 32),
    (96, W.FP8, 4, 1, 16), (192, W.BF16, 4, 2, 16), (192, W.FP8, 2, 2, 64), (256, W.BF16, 4, 1, 64),
    (256, W.BF16, 2, 2, 128), (224, W.BF16, 2, 1, 16)])
def test_prefill(d, dtype, hq, hkv, bs, window, sinks):
    case = W.make_case(f"pre_{d}_{dtype}", [65, 200, 131, 300], [65, 257, 1100, 801], hq, hkv, d, bs,
                       kv_dtype=dtype, seed=d + 1, poison=True, window=window)
    info = _check(case, sinks, decode_rows_max=0)
    assert info.num_decode_tiles == 0


SHAPES = {"cap": dict(cap=20.0), "bias": dict(slopes=[0.25, 0.06, -0.02, 0.0]),
          "prefix": dict(prefix=[0, 200, 900, 30]),
          "all": dict(cap=10.0, slopes=[0.25, 0.06, 0.01, 0.002], prefix=[3, 500, 0, 90])}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d,dtype", [(64, W.BF16), (128, W.BF16), (128, W.FP8), (96, W.BF16), (256, W.BF16)])
def test_beside_the_score_shapes(shape, d, dtype):
    case = W.make_case(f"shape_{shape}_{d}", [1, 150, 2, 90], [400, 750, 1029, 90], 4, 2, d, 16, seed=21,
                       kv_dtype=dtype, window=100)
    info = _check(case, 20, shape=SHAPES[shape], decode_rows_max=32)
    assert info.num_prefill_tiles > 0 and info.num_decode_tiles > 0


@pytest.mark.parametrize("d", [64, 128, 192])
def test_without_causal_mask(d):
    case = W.make_case(f"nc_{d}", [1, 140, 5], [370, 700, 33], 4, 2, d, 16, seed=22, causal=False, window=50)
    _check(case, 10)


def test_group_size_that_no_prefill_kernel_takes():
    case = W.make_case("qpk5", [80, 3], [900, 340], 10, 2, 128, 16, seed=23, window=120)
    assert _check(case, 5).num_prefill_tiles == 0


@pytest.mark.parametrize("sinks", [10 ** 6, 2 ** 40])
def test_more_sinks_than_keys_is_no_window(sinks):
    case = W.make_case("many", [1, 100], [300, 500], 4, 2, 128, 16, seed=24, window=10)
    _check(case, sinks, gone=False)


def test_sinks_that_draw_all_attention():
    """Scores of the first keys tower over the window's: what is left of those underflows."""
    case = W.make_case("draw", [1, 80, 3], [900, 700, 50], 4, 2, 128, 16, seed=25, window=64)
    case.q.abs_()
    for s in range(3):
        case.k_cache[int(case.block_tables[s, 0]), :4] = 8.0
    _check(case, 4)


def test_session_that_gives_its_pages_back():
    """Token after token and chunk after chunk over one table whose middle empties."""
    case = W.make_case("session", [1, 1, 200], [3000, 1025, 2500], 8, 2, 128, 16, seed=26, window=256, poison=True)
    b0 = tu.to_device(case)
    with _plan(b0, 4) as plan:
        want = tu.forward(plan, b0)
        assert plan.last_device_error() == 0
    _give_back(case, 4)
    b = tu.to_device(case)
    with _plan(b, 4) as plan:
        got = tu.forward(plan, b)
        assert plan.last_device_error() == 0
    assert torch.equal(got, want) and torch.all(got.isfinite())


def test_missing_pages_that_are_seen_are_reported():
    for page in (0, 2990 // 16):
        case = W.make_case("badpage", [1], [3000], 8, 2, 128, 16, seed=27, window=64)
        case.block_tables[0, page] = -5
        b = tu.to_device(case)
        with _plan(b, 4) as plan:
            tu.forward(plan, b)
            assert plan.last_device_error() == ua.UA_ERR_BOUNDS


def test_fp8_products():
    """Against the same plan with staged products: both round, within the sum of their bounds
    (tests/test_gpu_scores.py test_fp8_products)."""
    case = W.make_case("f8p", [200, 140], [1260, 500], 4, 2, 128, 16, kv_dtype=W.FP8, seed=28, window=150)
    q = (torch.randn(case.q.shape, generator=torch.Generator().manual_seed(5)).clamp(-1.75, 1.75) * 256)
    q = (q.to(torch.float8_e4m3fn).float() / 256).to(torch.bfloat16)
    q[..., 0] = 1.75
    case.q.copy_(q)
    _give_back(case, 9)
    r, b = case.raw(), tu.to_device(case)
    exp, _, rows = S.paged_attention_shaped(
        r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"], r["kv_lens"], r["block_tables"], 16, case.scale,
        kv_dtype=W.FP8, k_scale=case.k_scale, v_scale=case.v_scale, window=150, sinks=9, with_probs=True)
    with _plan(b, 9, decode_rows_max=0) as plan:
        ua.ua_plan_set_fp8_products(plan.handle, True)
        got = as_f64(tu.forward(plan, b))
        assert plan.last_device_error() == 0
    for (tok, h), (_, p, v) in rows.items():
        e = p / p.max()
        tol = (np.maximum(2.0 ** -4 * e, 2.0 ** -10) + 2.0 ** -10 * e) @ np.abs(v) / e.sum()
        assert np.all(np.abs(got[tok, h] - exp[tok, h]) <= tol + 2.0 ** -8 * (np.abs(exp[tok, h]) + tol))


def test_captured_forward_and_unified_max():
    case = W.make_case("graph", [1, 200, 1], [1300, 460, 77], 8, 2, 128, 16, seed=31, window=90)
    b = tu.to_device(case)
    with _plan(b, 7) as plan:
        plan.set_unified_max(1.0)
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
        exp, spread = _expected(case, 7)
        assert np.all(np.abs(as_f64(out) - exp) <= _bound(case, exp, spread))


def test_window_without_sinks_is_unchanged():
    case = W.make_case("plain", [1, 100], [900, 600], 8, 2, 128, 16, seed=32, window=100)
    b = tu.to_device(case)
    with tu.make_plan(b) as plain, tu.make_plan(b, sink_tokens=0) as none:
        assert torch.equal(tu.forward(plain, b), tu.forward(none, b))


def test_refusals():
    case = W.make_case("ref", [1], [20], 4, 2, 64, 16, window=4)
    b = tu.to_device(case)
    for sinks in (-1, -2 ** 40):
        with pytest.raises(ua.UAError) as e:
            tu.make_plan(b, sink_tokens=sinks)
        assert e.value.status == ua.UA_ERR_INVALID_ARG
    b.causal = 0
    with pytest.raises(ValueError):
        tu.make_plan(b, sink_tokens=4, prefix_lens=[3])


@pytest.mark.parametrize("dtype", [W.BF16, W.FP8])
@pytest.mark.parametrize("splits", [1, 3, 7])
def test_gather_takes_the_keys_that_the_decode_kernel_reads(splits, dtype):
    """Over pages given back: no row of theirs, no error, every other row bit for bit."""
    window, sinks, elt = 100, 20, 1 if dtype == W.FP8 else 2
    case = W.make_case("gather", [1, 3, 9, 1], [900, 640, 433, 60], 8, 2, 128, 16, kv_dtype=dtype, seed=33, window=window)
    _give_back(case, sinks)
    b = tu.to_device(case)
    with _plan(b, sinks, num_splits=splits, decode_rows_max=10 ** 6) as plan:
        _, _, dec, _ = ua.ua_schedule(b.cu_host, b.kv_host, 8, 2, 128, 16, int(b.block_tables.shape[1]),
                                      kv_dtype=b.kv_dtype, window=window, num_splits=splits,
                                      num_sms=plan.info.num_sms, decode_rows_max=10 ** 6, sink_tokens=sinks)
        want = []
        for t in dec:
            n, kv = case.query_lens[t["seq"]], int(case.kv_lens[t["seq"]])
            first = kv - n + t["row0"] // 4  # position of the tile's first row
            unseen = lambda key: sinks <= key <= first - window  # noqa: E731
            for key in range(t["kv_lo"], t["kv_hi"]):
                step = key // 16 * 16
                if not (unseen(step) and unseen(step + 15)):
                    want.append((int(case.block_tables[t["seq"], key // 16]), key % 16, t["kv_head"]))
        ranges = sum(t["kv_hi"] - t["kv_lo"] for t in dec)
        assert splits == 7 or len(want) < ranges  # (seven pieces end and start at the gap)
        assert min(page for page, _, _ in want) >= 0
        ko, vo = (torch.zeros((len(want) + 1, 128 * elt), dtype=torch.uint8, device="cuda") for _ in range(2))
        ua.ua_gather_kv_debug(plan.handle, b.k_cache, b.v_cache, b.kv_lens, b.block_tables, b.num_blocks, ko, vo,
                              len(want))
        assert plan.last_device_error() == 0
        with pytest.raises(ua.UAError):
            ua.ua_gather_kv_debug(plan.handle, b.k_cache, b.v_cache, b.kv_lens, b.block_tables, b.num_blocks, ko, vo,
                                  len(want) - 1)
    page, slot, head = (torch.tensor(x) for x in zip(*want))
    for got, cache in ((ko, case.k_cache), (vo, case.v_cache)):
        raw = cache.contiguous().view(torch.uint8).reshape(case.num_blocks, 16, 2, 128 * elt)
        assert torch.equal(got.cpu()[:-1], raw[page, slot, head]) and not got[-1].any()
