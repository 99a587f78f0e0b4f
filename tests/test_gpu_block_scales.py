"""GPU parity of an e4m3 cache with block scales: the appends that write codes and
scales, and attention over it, against the fp64 oracle; refusals.

A code is right when it is at most half a step (2^-4 of the value, 2^-10 below the
smallest normal) from the exact quotient, with the error of a rotated element
(tests/test_gpu_rope.py) and 2^-23 of the quotient more. Attention: the bound of
tests/test_gpu_scores.py, where prefills read keys and values as the staged copy
rounds them (the oracle's too). Decode weights carry their page's value scale: a
weight below 2^-14 of the reference has an absolute error of 2^-25, of codes up to
448, against a denominator of at least 1 / (the largest value scale).
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
from oracle import attention as A
from oracle import block_scales as B
from oracle import rope as R
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


# ---------------------------------------------------------------- appends

class Step:
    def __init__(self, ql, kv, hq, hkv, d, bs, seed=0, power=True, loud=1.0):
        self.case = W.make_case(f"fill_{d}_{bs}", ql, kv, hq, hkv, d, bs, kv_dtype=W.FP8, seed=seed)
        self.b = tu.to_device(self.case)
        g = torch.Generator().manual_seed(seed + 1)
        rows = torch.randn(sum(ql), hq + 2 * hkv, d, generator=g)
        rows *= torch.exp2(2 * torch.randn(sum(ql), hq + 2 * hkv, 1, generator=g)) * loud
        rows = rows.to(torch.bfloat16).cuda()
        self.q, self.k, self.v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        size = torch.exp2(3 * torch.randn(2, self.b.num_blocks, hkv, generator=g)) / 448
        if power:
            size = torch.exp2(size.log2().ceil())
        self.scales = [x.contiguous().cuda() for x in size]
        self.before = self.values(), [as_f64(x) for x in self.scales]

    def values(self):
        return [as_f64(x.view(torch.float8_e4m3fn).float()) for x in (self.b.k_cache, self.b.v_cache)]

    def plan(self, **args):
        plan = tu.make_plan(self.b, **args)
        plan.set_block_scales(*self.scales)
        return plan

    def append(self, plan, **args):
        b = self.b
        plan.append_kv(self.k.contiguous(), self.v.contiguous(), b.k_cache, b.v_cache, b.block_tables,
                       b.num_blocks, **args)

    def rope_append(self, plan, rope, positions=None, **args):
        b, out = self.b, torch.empty(self.q.shape, dtype=torch.bfloat16, device="cuda")
        plan.rope_append_kv(rope, self.q, self.k, self.v, out, b.k_cache, b.v_cache, b.block_tables, b.num_blocks,
                            positions=positions, **args)
        return out

    def check(self, k, v, k_slack=None, skip=()):
        """k, v: the exact elements; k_slack: their error (absolute)."""
        c = self.case
        for got, scales, old, old_scales, x, slack in zip(
                self.values(), self.scales, *self.before, (k, v), (k_slack, None)):
            want, want_scales = B.append(x, old, old_scales, c.cu_query_lens.tolist(), c.kv_lens.tolist(),
                                         c.block_tables.numpy(), c.block_size, skip)
            assert np.array_equal(as_f64(scales), want_scales, equal_nan=True)
            new = np.zeros(got.shape[:2], dtype=bool)
            more = np.zeros(got.shape)
            for s, (n, kv) in enumerate(zip(c.query_lens, c.kv_lens.tolist())):
                if s in skip:
                    continue
                pos = np.arange(kv - n, kv)
                page = c.block_tables.numpy()[s, pos // c.block_size]
                new[page, pos % c.block_size] = True
                if slack is not None:
                    cu = int(c.cu_query_lens[s])
                    more[page, pos % c.block_size] = slack[cu:cu + n] / want_scales[page][..., None]
            assert np.array_equal(got[~new], want[~new], equal_nan=True)
            exp, more = want[new], more[new]
            tol = np.maximum(2.0 ** -4 * np.abs(exp), 2.0 ** -10) + more * 1.1 + 2.0 ** -23 * np.abs(exp)
            assert np.all(np.abs(got[new] - np.clip(exp, -448, 448)) <= tol)


SIZES = [  # d, hq, hkv, bs
    (128, 8, 2, 16), (128, 8, 8, 64), (64, 4, 1, 16), (32, 2, 2, 16), (96, 6, 3, 32), (160, 4, 2, 16),
    (192, 5, 5, 16), (224, 2, 1, 48), (256, 4, 4, 128), (256, 2, 1, 16), (32, 1, 1, 256), (128, 16, 16, 128)]


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("d,hq,hkv,bs", SIZES)
def test_append(d, hq, hkv, bs, power):
    s = Step([1, 9, 0, 17, 1, 300, 33, 2], [1, 40, 5, 17, 700, 300, 170, 258], hq, hkv, d, bs, seed=d + bs, power=power)
    with s.plan() as plan:
        s.append(plan)
        assert plan.last_device_error() == 0
        s.check(as_f64(s.k), as_f64(s.v))
        was = s.b.k_cache.clone(), s.b.v_cache.clone(), s.scales[0].clone(), s.scales[1].clone()
        s.append(plan)  # the same step again changes nothing
        torch.cuda.synchronize()
        for x, y in zip(was, (s.b.k_cache, s.b.v_cache, *s.scales)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("share", [1.0, 0.5, 0.37])
@pytest.mark.parametrize("d,hq,hkv,bs", SIZES)
def test_rope_append(d, hq, hkv, bs, share, interleaved):
    s = Step([1, 9, 0, 17, 1, 300, 33, 2], [1, 40, 5, 17, 700, 300, 170, 258], hq, hkv, d, bs, seed=d + bs + 7)
    w = R.frequencies(2 * int(d * share / 2), 10000.0)[0]
    pos = np.concatenate([np.arange(b - a, b) for a, b in zip(s.case.query_lens, s.case.kv_lens.tolist())])
    with s.plan() as plan, ua.Rope(w, interleaved, 1.25) as rope:
        out = s.rope_append(plan, rope)
        assert plan.last_device_error() == 0
    slack = lambda x: 2.5e-6 * 1.25 * R.pair_size(as_f64(x), 2 * len(w), interleaved)  # noqa: E731
    exp = R.rotate(as_f64(s.q), pos, w, interleaved, 1.25)
    assert np.all(np.abs(as_f64(out) - exp) <= 2.0 ** -8 * np.abs(exp) + 1.01 * slack(s.q))
    s.check(R.rotate(as_f64(s.k), pos, w, interleaved, 1.25), as_f64(s.v), slack(s.k))


def test_rope_append_with_axes():
    s = Step([5, 40], [50, 40], 6, 2, 96, 16, seed=3)
    w, pair_axes = R.frequencies(96, 10000.0)[0], [i % 3 for i in range(48)]
    pos = np.random.default_rng(4).integers(0, 5000, size=(3, 45))
    with s.plan() as plan, ua.Rope(w, axes=pair_axes) as rope:
        out = s.rope_append(plan, rope, torch.from_numpy(pos).to(torch.int32).cuda())
    slack = lambda x: 2.5e-6 * R.pair_size(as_f64(x), 96, False)  # noqa: E731
    exp = R.rotate(as_f64(s.q), pos, w, False, 1.0, pair_axes)
    assert np.all(np.abs(as_f64(out) - exp) <= 2.0 ** -8 * np.abs(exp) + 1.01 * slack(s.q))
    s.check(R.rotate(as_f64(s.k), pos, w, False, 1.0, pair_axes), as_f64(s.v), slack(s.k))


def test_scales_at_their_borders():
    """Largest magnitudes of exactly 448 times a power of two, one bf16 step above, zeros, infinities,
    NaN, the smallest and the largest numbers, and pages that never had a scale."""
    s = Step([20, 1, 1, 1, 1], [20, 40, 40, 40, 40], 2, 2, 64, 16, seed=5)
    for x in (s.k, s.v):
        x.copy_(x.sign())
        x[:16, 0, 3], x[:16, 1, 3] = 448.0, 450.0
        x[16:20, 0], x[16:20, 1] = 0.0, 2.0 ** -120
        x[20, 0, 5], x[20, 1, 5] = float("inf"), -float("inf")
        x[21, 0, 7] = float("nan")
        x[22, :, 1], x[23, :, 1] = 3e38, 2.0 ** -126
    for x in s.scales:
        pages = [int(s.case.block_tables[i, 2]) for i in range(1, 5)]
        x[pages[0]], x[pages[1]], x[pages[2]], x[pages[3]] = 0.5, 0.0, 3.0, float("inf")
    s.before = s.values(), [as_f64(x) for x in s.scales]
    with s.plan() as plan:
        s.append(plan)
        assert plan.last_device_error() == 0
    k, v = as_f64(s.k), as_f64(s.v)
    got = s.values()
    assert np.all(np.isnan(got[0][int(s.case.block_tables[2, 2]), 7, 0, 7]))
    for name, x in (("k", k), ("v", v)):
        x[21, 0, 7] = 0.0
        cache = getattr(s.b, name + "_cache").view(torch.uint8)
        cache[int(s.case.block_tables[2, 2]), 7, 0, 7] = 0  # (seen above)
    s.check(k, v)


@pytest.mark.parametrize("bs", [16, 64])
def test_step_by_step_equals_the_rule_step_by_step(bs):
    """One token a step, from an empty cache: scales grow on the way, earlier codes follow."""
    s = Step([1], [40], 2, 2, 64, bs, seed=6)
    for x in s.scales:
        x.zero_()
    rows = (torch.randn(2, 40, 2, 64) * torch.exp2(torch.arange(40) / 4.0)[:, None, None]).to(torch.bfloat16).cuda()
    for n in range(1, 41):
        s.before = s.values(), [as_f64(x) for x in s.scales]
        s.case.kv_lens[0] = s.b.kv_host[0] = n
        s.k, s.v = rows[0, n - 1:n], rows[1, n - 1:n]
        with s.plan() as plan:
            s.append(plan)
            s.check(as_f64(s.k), as_f64(s.v))


@pytest.mark.parametrize("rope", [False, True])
def test_pages_out_of_range_are_reported_and_nothing_is_written(rope):
    s = Step([20, 3], [50, 20], 4, 2, 64, 16, seed=8)
    for bad in (-1, s.b.num_blocks, 2 ** 31 - 1):
        s.b.block_tables[0, 2:] = bad
        s.b.block_tables[0, 1] = -7
        with s.plan() as plan, ua.Rope(R.frequencies(64, 10000.0)[0]) as r:
            out = s.rope_append(plan, r) if rope else s.append(plan)
            assert plan.last_device_error() == ua.UA_ERR_BOUNDS
        if rope:
            assert torch.all(out.isfinite())
    pos = np.concatenate([np.arange(30, 50), np.arange(17, 20)])
    w = R.frequencies(64, 10000.0)[0]
    if rope:
        s.check(R.rotate(as_f64(s.k), pos, w, False), as_f64(s.v), 2.5e-6 * R.pair_size(as_f64(s.k), 64, False),
                skip=(0,))
    else:
        s.check(as_f64(s.k), as_f64(s.v), skip=(0,))


def test_captured_appends_and_forward_replay_on_another_stream():
    s = Step([3, 70], [20, 90], 8, 2, 128, 16, seed=9)
    w = R.frequencies(128, 10000.0)[0]
    side = torch.cuda.Stream()
    with s.plan() as plan, ua.Rope(w) as rope:
        s.rope_append(plan, rope)
        tu.forward(plan, s.b)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = s.rope_append(plan, rope)
            s.b.q.copy_(q)
            out = tu.forward(plan, s.b)
        # another step's rows and an older cache
        for name, x in zip(("k_cache", "v_cache"), s.before[0]):
            getattr(s.b, name).view(torch.float8_e4m3fn).copy_(torch.from_numpy(x).to(torch.float8_e4m3fn))
        for x, y in zip(s.scales, s.before[1]):
            x.copy_(torch.from_numpy(y))
        s.k.copy_(s.k.flip(0))
        s.v.copy_(s.v.flip(0))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        pos = np.concatenate([np.arange(17, 20), np.arange(20, 90)])
        s.check(R.rotate(as_f64(s.k), pos, w, False), as_f64(s.v), 2.5e-6 * R.pair_size(as_f64(s.k), 128, False))
        want = tu.forward(plan, s.b)
        assert torch.equal(out, want)


# ---------------------------------------------------------------- attention

def _scales(case, seed, power, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.exp2(spread * torch.randn(2, case.num_blocks, case.num_kv_heads, generator=g)) / 128
    if power:
        x = torch.exp2(x.log2().round())
    x[0] *= 0.5
    return x[0].contiguous(), x[1].contiguous()


def _expected(case, ks, vs, cap=0.0, slopes=None, prefix=None, sinks=0, staged=False):
    r = case.raw()
    return S.paged_attention_shaped(
        r["q"], r["k_cache"], r["v_cache"], r["cu_query_lens"], r["kv_lens"], r["block_tables"], case.block_size,
        case.scale, kv_dtype=W.FP8, causal=case.causal, window=case.window, softcap=cap, slopes=slopes,
        prefix_lens=prefix, sinks=sinks, k_scales=as_f64(ks), v_scales=as_f64(vs), staged=staged)


def _check(case, power=True, spread=2.0, seed=50, phi=None, setup=None, stream=None, shape=None, **plan_args):
    shape = dict(shape or {})
    ks, vs = _scales(case, seed, power, spread)
    b = tu.to_device(case)
    with tu.make_plan(b, prefix_lens=shape.get("prefix"), sink_tokens=shape.get("sinks", 0), **plan_args) as plan:
        if shape.get("cap") or shape.get("slopes"):
            plan.set_scores(shape.get("cap", 0.0), None if shape.get("slopes") is None else
                            torch.tensor(shape["slopes"], device="cuda"))
        plan.set_block_scales(ks.cuda(), vs.cuda())
        if phi is not None:
            plan.set_unified_max(phi)
        info = plan.info
        out = torch.full(b.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
        tu.forward(plan, b, out)
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0
    exp, spread = _expected(case, ks, vs, **shape, staged=info.num_prefill_tiles > 0)
    got = as_f64(out)
    assert np.all(np.isfinite(got))
    tail = max(case.kv_lens.tolist()) * 2.0 ** -25 * 448.0 * float(vs.max())
    bound = 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * (1 + 2.0 ** -8) * spread + tail + 1e-30
    assert (np.abs(got - exp) - bound).max() <= 0
    return info


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("d,hq,hkv,bs", [
    (128, 16, 2, 16), (128, 4, 4, 128), (64, 8, 1, 16), (32, 5, 1, 64), (96, 6, 2, 16), (160, 4, 2, 16),
    (192, 4, 2, 32), (224, 4, 4, 16), (256, 8, 4, 16)])
def test_decode(d, hq, hkv, bs, power):
    case = W.make_case(f"dec_{d}", [1, 1, 3, 1, 2], [1, 17, 40, 333, 2500], hq, hkv, d, bs, kv_dtype=W.FP8, seed=d,
                       poison=True)
    info = _check(case, power, decode_rows_max=10 ** 6)
    assert info.num_prefill_tiles == 0


@pytest.mark.parametrize("splits", [2, 9, 100])
def test_decode_splits(splits):
    case = W.make_case("spl", [1, 2], [1900, 2001], 8, 2, 128, 16, kv_dtype=W.FP8, seed=7)
    assert _check(case, False, num_splits=splits).num_combine_groups > 0


@pytest.mark.parametrize("power", [True, False])
@pytest.mark.parametrize("d,hq,hkv,bs", [
    (128, 8, 2, 16), (128, 2, 2, 128), (64, 4, 4, 32), (192, 2, 2, 16), (256, 4, 1, 64)])
def test_prefill(d, hq, hkv, bs, power):
    case = W.make_case(f"pre_{d}", [65, 200, 131, 300], [65, 257, 600, 301], hq, hkv, d, bs, kv_dtype=W.FP8,
                       seed=d + 1, poison=True)
    info = _check(case, power, decode_rows_max=0)
    assert info.num_decode_tiles == 0


SHAPES = {"cap": dict(cap=20.0), "bias": dict(slopes=[0.25, 0.06, -0.02, 0.0]), "prefix": dict(prefix=[9, 333]),
          "sinks": dict(sinks=20), "all": dict(cap=10.0, slopes=[0.25, 0.06, 0.01, 0.002], prefix=[30, 400], sinks=5)}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("d", [32, 96, 128, 256])
@pytest.mark.parametrize("ql,rows", [([1, 3], 32), ([150, 201], 0)])
def test_beside_the_score_shapes(shape, d, ql, rows):
    """Prompts at head dims that only shaped scores have a prefill kernel for among them."""
    case = W.make_case(f"shape_{shape}_{d}", ql, [400, 750], 4, 2, d, 16, kv_dtype=W.FP8, seed=21,
                       window=100 if shape in ("sinks", "all") else 0)
    info = _check(case, shape=SHAPES[shape], decode_rows_max=rows)
    assert (info.num_prefill_tiles > 0) == (rows == 0)


@pytest.mark.parametrize("spread", [0.0, 6.0, 12.0])
def test_scales_far_apart(spread):
    """Value scales that differ by many powers of two from page to page: every row is as exact as
    its own pages allow (the bound of the weights alone is not enough for those; the value of a row
    that sees one page is)."""
    case = W.make_case("apart", [1] * 6, [16, 32, 160, 900, 1600, 333], 4, 2, 128, 16, kv_dtype=W.FP8, seed=33)
    _check(case, False, spread=spread)
    _check(case, True, spread=spread, num_splits=3)


@pytest.mark.parametrize("first", [True, False])
def test_a_page_of_zeros_beside_loud_ones(first):
    """Values of zero under the least scale, where most of the attention goes."""
    case = W.make_case("zeros", [1, 1], [48, 320], 4, 2, 64, 16, kv_dtype=W.FP8, seed=34)
    ks, vs = (torch.full((case.num_blocks, 2), 1 / 64) for _ in range(2))
    for s in range(2):
        page = int(case.block_tables[s, 0 if first else 2])
        case.v_cache.view(torch.uint8)[page] = 0
        vs[page] = B.LEAST
    b = tu.to_device(case)
    exp, spread = _expected(case, ks, vs)
    with tu.make_plan(b) as plan:
        plan.set_block_scales(ks.cuda(), vs.cuda())
        got = as_f64(tu.forward(plan, b))
    assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * 1.01 * spread
                  + 320 * 2.0 ** -25 * 7.0)


@pytest.mark.parametrize("phi", [0.0, 3.0, -50.0])
def test_unified_max(phi):
    case = W.make_case("phi", [1, 1, 2], [300, 1000, 40], 8, 2, 128, 16, kv_dtype=W.FP8, seed=27)
    _check(case, False, phi=phi)


def test_mixed_batch_and_no_causal_mask():
    case = W.make_case("mixed", [1, 200, 2, 1], [900, 260, 40, 3000], 8, 2, 128, 16, kv_dtype=W.FP8, seed=35)
    info = _check(case)  # powers of two: the staged copy is exact
    assert info.num_prefill_tiles > 0 and info.num_decode_tiles > 0
    case = W.make_case("nc", [1, 140, 5], [70, 300, 33], 4, 2, 64, 16, kv_dtype=W.FP8, seed=36, causal=False)
    _check(case)


def test_equal_scales_are_one_scale_a_tensor():
    """Powers of two, the same for every block: as the tensor's scale (another order of roundings)."""
    case = W.make_case("same", [1, 130, 3], [900, 260, 40], 8, 2, 128, 16, kv_dtype=W.FP8, seed=37)
    b = tu.to_device(case)
    b.k_scale, b.v_scale = 2.0 ** -7, 2.0 ** -6
    one = lambda x: torch.full((b.num_blocks, 2), x, device="cuda")  # noqa: E731
    with tu.make_plan(b) as plan:
        want = tu.forward(plan, b)
        plan.set_block_scales(one(2.0 ** -7), one(2.0 ** -6))
        b.k_scale, b.v_scale = float("nan"), 0.0  # ignored
        got = tu.forward(plan, b)
        assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -6, atol=1e-4)
        plan.set_block_scales()
        b.k_scale, b.v_scale = 2.0 ** -7, 2.0 ** -6
        assert torch.equal(tu.forward(plan, b), want)


def test_whatever_unseen_scales_hold():
    case = W.make_case("unseen", [1, 90], [100, 333], 4, 2, 128, 16, kv_dtype=W.FP8, seed=38, num_blocks=64)
    ks, vs = _scales(case, 1, True)
    used = set()
    for s, kv in enumerate(case.kv_lens.tolist()):
        used |= {int(x) for x in case.block_tables[s, :-(-kv // 16)]}
    exp, spread = _expected(case, ks, vs)
    for blk in set(range(64)) - used:
        ks[blk], vs[blk] = float("nan"), float("inf")
    b = tu.to_device(case)
    with tu.make_plan(b) as plan:
        plan.set_block_scales(ks.cuda(), vs.cuda())
        got = as_f64(tu.forward(plan, b))
    vmax = 448.0 * max(float(vs[x].max()) for x in used)
    assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + (2.0 ** -8 + 2.0 ** -10) * 1.01 * spread
                  + 333 * 2.0 ** -25 * vmax)


def test_a_session_from_empty_pages():
    """Prompts, then tokens one at a time: rope append and attention with sinks, every step against
    the oracle on what the cache holds."""
    hq, hkv, d, bs, window, sinks = 8, 2, 128, 16, 40, 4
    case = W.make_case("session", [100, 1, 37], [100, 1, 37], hq, hkv, d, bs, kv_dtype=W.FP8, seed=39,
                       extra_table_cols=1, window=window)
    blocks = 3 * 8
    case.block_tables = torch.randperm(blocks).to(torch.int32).view(3, 8).contiguous()
    case.k_cache = torch.zeros(blocks, bs, hkv, d).to(torch.float8_e4m3fn)
    case.v_cache = case.k_cache.clone()
    b = tu.to_device(case)
    ks, vs = tu.new_block_scales(b)
    w, pair_axes = R.frequencies(d, 10000.0)[0], [i % 3 for i in range(d // 2)]
    g = torch.Generator().manual_seed(40)
    lens = [0, 0, 0]
    with ua.Rope(w, axes=pair_axes) as rope:
        for ql in ([100, 1, 37], [1, 1, 1], [1, 9, 1], [1, 1, 20]):
            lens = [a + n for a, n in zip(lens, ql)]
            rows = torch.randn(sum(ql), hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
            cu = [0, ql[0], ql[0] + ql[1], sum(ql)]
            b.q, b.cu_host, b.kv_host = torch.empty_like(rows[:, :hq].contiguous()), cu, lens
            b.cu_query_lens, b.kv_lens = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (cu, lens))
            pos = torch.randint(0, 3000, (3, sum(ql)), generator=g).to(torch.int32).cuda()
            with tu.make_plan(b, sink_tokens=sinks) as plan:
                plan.set_block_scales(ks, vs)
                tu.rope_append_kv(plan, b, rope, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], pos)
                got = tu.forward(plan, b)
                assert plan.last_device_error() == 0
            bits = lambda t: t.cpu().view(torch.int16).numpy().view(np.uint16)  # noqa: E731
            exp, spread = S.paged_attention_shaped(
                bits(b.q), b.k_cache.cpu().numpy(), b.v_cache.cpu().numpy(), cu, lens, b.block_tables.cpu().numpy(),
                bs, case.scale, kv_dtype=W.FP8, window=window, sinks=sinks, k_scales=as_f64(ks), v_scales=as_f64(vs))
            tail = max(lens) * 2.0 ** -25 * 448.0 * float(vs.max())
            assert np.all(np.abs(as_f64(got) - exp) <= 2.0 ** -8 * np.abs(exp) + 1.26 * 2.0 ** -8 * spread + tail)
            # what was appended: one rounding of the keys, no block's codes beyond its scale
            key = R.rotate(as_f64(rows[:, hq:hq + hkv]), pos.cpu().numpy(), w, False, 1.0, pair_axes)
            at = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, ql)])
            seq = np.repeat(np.arange(3), ql)
            page = b.block_tables.cpu().numpy()[seq, at // bs]
            held = A.decode_e4m3(b.k_cache.cpu().numpy())[page, at % bs] * as_f64(ks)[page][..., None]
            assert np.all(np.abs(held - key) <= np.maximum(2.0 ** -4 * np.abs(key),
                                                           2.0 ** -10 * as_f64(ks)[page][..., None]) + 1e-5)


# ---------------------------------------------------------------- refusals

def test_refusals():
    case = W.make_case("ref", [2], [40], 4, 2, 128, 16, kv_dtype=W.FP8, seed=41)
    b = tu.to_device(case)
    good = lambda: torch.ones(b.num_blocks, 2, device="cuda")  # noqa: E731
    ks, vs = good(), good()
    with tu.make_plan(b) as plan:
        want = tu.forward(plan, b)
        for x in (ks[:1], ks.double(), ks.T.contiguous(), ks.repeat(1, 2)[:, ::2], ks.flatten()):
            with pytest.raises(ValueError):
                plan.set_block_scales(x, vs)
        with pytest.raises(ValueError):
            plan.set_block_scales(ks)
        both = torch.ones(b.num_blocks + 1, 2, device="cuda")
        for x, y, status in ((ks.cpu(), vs.cpu(), None), (ks, ks, ua.UA_ERR_INVALID_ARG),
                             (both[:-1], both[1:], ua.UA_ERR_INVALID_ARG),
                             (ks.cpu().pin_memory(), vs, ua.UA_ERR_INVALID_ARG)):
            with pytest.raises(ua.UAError) as e:
                plan.set_block_scales(x, y)
            assert status is None or e.value.status == status
        for n in (0, -1, 2 ** 31 - 1):
            with pytest.raises(ua.UAError) as e:
                ua.ua_plan_set_block_scales(plan.handle, ks, vs, n)
            assert e.value.status == ua.UA_ERR_INVALID_ARG
        for x, y in ((ks, None), (None, vs), (ks.data_ptr() + 2, vs)):
            with pytest.raises(ua.UAError):
                ua.ua_plan_set_block_scales(plan.handle, x, y, b.num_blocks)
        assert torch.equal(tu.forward(plan, b), want)  # nothing was set
        # another number of blocks than the call's
        plan.set_block_scales(torch.ones(b.num_blocks + 1, 2, device="cuda"), torch.ones(b.num_blocks + 1, 2, device="cuda"))
        rows = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda")
        with ua.Rope([0.5] * 64) as rope:
            for call in (lambda: tu.forward(plan, b),
                         lambda: tu.append_kv(plan, b, rows[:, :2].contiguous(), rows[:, 2:4].contiguous()),
                         lambda: tu.rope_append_kv(plan, b, rope, rows[:, :4], rows[:, 4:6], rows[:, 6:])):
                with pytest.raises(ua.UAError) as e:
                    call()
                assert e.value.status == ua.UA_ERR_INVALID_ARG
        # fp8 products and block scales exclude one another
        with pytest.raises(ua.UAError) as e:
            ua.ua_plan_set_fp8_products(plan.handle, True)
        assert e.value.status == ua.UA_ERR_UNSUPPORTED
        plan.set_block_scales()
        ua.ua_plan_set_fp8_products(plan.handle, True)
        with pytest.raises(ua.UAError) as e:
            plan.set_block_scales(ks, vs)
        assert e.value.status == ua.UA_ERR_UNSUPPORTED
    case = W.make_case("ref16", [2], [20], 4, 2, 128, 16)
    with tu.make_plan(tu.to_device(case)) as plan:
        with pytest.raises(ua.UAError) as e:
            plan.set_block_scales(ks, vs)
        assert e.value.status == ua.UA_ERR_UNSUPPORTED


def test_scales_live_until_the_streams_are_done():
    case = W.make_case("life", [1, 1], [3000, 5000], 8, 2, 128, 16, kv_dtype=W.FP8, seed=42)
    b = tu.to_device(case)
    ks, vs = _scales(case, 2, True)
    side = torch.cuda.Stream()
    with tu.make_plan(b) as plan:
        plan.set_block_scales(ks.cuda(), vs.cuda())
        want = tu.forward(plan, b)
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
            got = tu.forward(plan, b, stream=side)
        plan.set_block_scales()
        junk = [torch.full((b.num_blocks, 2), 1e30, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk


def test_pages_beyond_32_bits():
    """Pages whose first element lies past 2^32: appended to and read as the first ones are."""
    hkv, d, bs, need = 2, 128, 16, 5
    blocks = 2 ** 32 // (bs * hkv * d) + 64
    k_cache, v_cache = (torch.zeros(blocks, bs, hkv, d, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(blocks, hkv, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(43)
    q, k, v = (torch.randn(77, h, d, generator=g).to(torch.bfloat16).cuda() for h in (4, hkv, hkv))
    cu, kv = torch.tensor([0, 77], dtype=torch.int32, device="cuda"), torch.tensor([77], dtype=torch.int32, device="cuda")
    outs = {}
    for rows in (0, 10 ** 6):  # decode_rows_max: in the prefill kernel over a staged copy, in the decode kernel
        for last in (False, True):
            pages = torch.arange(need, dtype=torch.int32, device="cuda")
            table = (blocks - 1 - pages if last else pages)[None].contiguous()
            out = torch.empty_like(q)
            with ua.Plan([0, 77], [77], 4, hkv, d, bs, need, kv_dtype=ua.UA_KV_FP8_E4M3, decode_rows_max=rows) as plan:
                plan.set_block_scales(ks, vs)
                plan.append_kv(k, v, k_cache, v_cache, table, blocks)
                plan.forward(q, k_cache, v_cache, out, cu, kv, table, blocks, 77, 77, d ** -0.5)
                assert plan.last_device_error() == 0
            outs[rows, last] = out
        assert torch.equal(outs[rows, False], outs[rows, True])
    for cache, scales in ((k_cache, ks), (v_cache, vs)):
        assert torch.equal(cache[:need], cache[-need:].flip(0)) and torch.equal(scales[:need], scales[-need:].flip(0))
        assert int(cache[:need].count_nonzero()) > 0 and torch.all(scales[need:-need] == 0)


def test_two_plans_on_two_streams_fill_one_cache():
    """Sequences of the same cache, appended to and read by two plans at once."""
    s = Step([150, 3, 90, 40], [150, 60, 200, 41], 8, 2, 128, 16, seed=44)
    b, c = s.b, s.case
    whole = [t.clone() for t in (b.k_cache, b.v_cache, *s.scales)]
    with s.plan() as plan:
        s.append(plan)
        torch.cuda.synchronize()
        want = [t.clone() for t in (b.k_cache, b.v_cache, *s.scales)]
    for t, w in zip((b.k_cache, b.v_cache, *s.scales), whole):
        t.copy_(w)
    torch.cuda.synchronize()
    streams, plans = [torch.cuda.Stream(), torch.cuda.Stream()], []
    cu, kv = c.cu_query_lens.tolist(), c.kv_lens.tolist()
    for st, (i, j) in zip(streams, ((0, 2), (2, 4))):
        plan = ua.Plan([x - cu[i] for x in cu[i:j + 1]], kv[i:j], 8, 2, 128, 16, b.block_tables.shape[1],
                       kv_dtype=ua.UA_KV_FP8_E4M3, stream=st)
        plan.set_block_scales(*s.scales)
        plans.append((plan, s.k[cu[i]:cu[j]].contiguous(), s.v[cu[i]:cu[j]].contiguous(), b.block_tables[i:j].contiguous()))
    torch.cuda.synchronize()
    for _ in range(3):
        for st, (plan, k, v, table) in zip(streams, plans):
            plan.append_kv(k, v, b.k_cache, b.v_cache, table, b.num_blocks, stream=st)
    torch.cuda.synchronize()
    for t, w in zip((b.k_cache, b.v_cache, *s.scales), want):
        assert torch.equal(t, w)
    for plan, *_ in plans:
        assert plan.last_device_error() == 0
        plan.close()


@pytest.mark.parametrize("rows", [0, 10 ** 6])
def test_sinks_over_pages_given_back(rows):
    """Pages that no query sees are gone, their scales hold anything."""
    case = W.make_case("gone", [3, 70], [900, 640], 8, 2, 128, 16, kv_dtype=W.FP8, seed=45, window=100)
    ks, vs = _scales(case, 3, True)
    exp, spread = _expected(case, ks, vs, sinks=20, staged=rows == 0)
    for s, (n, kv) in enumerate(zip(case.query_lens, case.kv_lens.tolist())):
        for page in range(2, (kv - n - 100 + 1) // 16):
            blk = int(case.block_tables[s, page])
            case.block_tables[s, page] = -1
            ks[blk], vs[blk] = float("nan"), 0.0
            case.k_cache.view(torch.uint8)[blk] = case.v_cache.view(torch.uint8)[blk] = 0x7F
    b = tu.to_device(case)
    with tu.make_plan(b, sink_tokens=20, decode_rows_max=rows) as plan:
        plan.set_block_scales(ks.cuda(), vs.cuda())
        got = as_f64(tu.forward(plan, b))
        assert plan.last_device_error() == 0
    tail = 900 * 2.0 ** -25 * 448.0 * float(vs.nan_to_num(0.0).max())
    assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + 1.26 * 2.0 ** -8 * spread + tail)


@pytest.mark.parametrize("scales_first", [True, False])
def test_scales_and_shaped_scores_in_either_order(scales_first):
    """Prompts at a head dim whose shaped scores have a schedule of their own."""
    case = W.make_case("order", [200, 150], [400, 750], 4, 2, 96, 16, kv_dtype=W.FP8, seed=46)
    ks, vs = _scales(case, 4, True)
    b = tu.to_device(case)
    with tu.make_plan(b, decode_rows_max=0) as plan:
        calls = [lambda: plan.set_block_scales(ks.cuda(), vs.cuda()), lambda: plan.set_scores(15.0)]
        for call in calls if scales_first else calls[::-1]:
            call()
        assert plan.info.num_prefill_tiles > 0
        got = as_f64(tu.forward(plan, b))
        exp, spread = _expected(case, ks, vs, cap=15.0, staged=True)
        assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + 1.26 * 2.0 ** -8 * spread + 1e-30)
        plan.set_scores()  # plain again: in the decode kernel
        assert plan.info.num_prefill_tiles == 0
        got = as_f64(tu.forward(plan, b))
        exp, spread = _expected(case, ks, vs)
        tail = 750 * 2.0 ** -25 * 448.0 * float(vs.max())
        assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + 1.26 * 2.0 ** -8 * spread + tail)
        assert plan.last_device_error() == 0


def test_plan_without_tokens():
    b = tu.to_device(W.make_case("none", [0, 0], [20, 0], 4, 2, 64, 16, kv_dtype=W.FP8))
    ks, vs = tu.new_block_scales(b)
    with tu.make_plan(b, sink_tokens=3) as plan, ua.Rope([0.5] * 32, axes=[0, 1] * 16) as rope:
        plan.set_block_scales(ks, vs)
        rows = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device="cuda")
        plan.rope_append_kv(rope, rows[:, :4], rows[:, 4:6], rows[:, 6:], rows[:, :4].contiguous(), b.k_cache, b.v_cache,
                            b.block_tables, b.num_blocks, positions=torch.zeros(2, 0, dtype=torch.int32, device="cuda"))
        plan.append_kv(rows[:, :2], rows[:, 2:4], b.k_cache, b.v_cache, b.block_tables, b.num_blocks)
        tu.forward(plan, b)
        assert plan.last_device_error() == 0


@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("d,hkv,bs", [(128, 8, 16), (64, 1, 64), (96, 2, 32), (256, 2, 16)])
def test_a_token_a_sequence(d, hkv, bs, rope):
    """Steps whose tiles are those of the plain append."""
    kv = [1, 16, 17, 40, 0, 65, 129, 700]
    s = Step([1, 1, 1, 1, 0, 1, 1, 1], kv, 2 * hkv, hkv, d, bs, seed=d + 11)
    with s.plan() as plan, ua.Rope(R.frequencies(d, 10000.0)[0]) as r:
        s.rope_append(plan, r) if rope else s.append(plan)
        assert plan.last_device_error() == 0
    if not rope:
        return s.check(as_f64(s.k), as_f64(s.v))
    pos = np.array([x - 1 for x in kv if x])
    s.check(R.rotate(as_f64(s.k), pos, R.frequencies(d, 10000.0)[0], False), as_f64(s.v),
            2.5e-6 * R.pair_size(as_f64(s.k), d, False))
