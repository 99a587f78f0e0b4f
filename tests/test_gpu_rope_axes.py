"""GPU parity of rotary append with positions of several axes, and its refusals.
Bounds: tests/test_gpu_rope.py."""
import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
from oracle import rope as R
from paged_kv_attention_unified_gb300 import torch_utils as tu

from _helpers import as_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


class Step:
    def __init__(self, ql, kv, hq, hkv, d, bs, dtype=W.BF16, seed=0):
        self.case = W.make_case(f"axes_{d}_{bs}_{dtype}", ql, kv, hq, hkv, d, bs, kv_dtype=dtype, seed=seed)
        self.b = tu.to_device(self.case)
        self.b.k_scale, self.b.v_scale = (0.02, 0.015) if dtype == W.FP8 else (1.0, 1.0)
        g = torch.Generator().manual_seed(seed + 1)
        rows = torch.randn(sum(ql), hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        self.slot_pos = np.concatenate([np.arange(b - a, b) for a, b in zip(ql, kv)]).astype(np.int64)
        self.seq = np.repeat(np.arange(len(ql)), ql)

    def run(self, plan, rope, positions=None, stream=None):
        b = self.b
        out = torch.empty(self.q.shape, dtype=torch.bfloat16, device="cuda")
        plan.rope_append_kv(rope, self.q, self.k, self.v, out, b.k_cache, b.v_cache, b.block_tables, b.num_blocks,
                            positions=positions, k_scale=b.k_scale, v_scale=b.v_scale, stream=stream)
        return out

    def check(self, out, w, interleaved, pair_axes, positions, amplitude=1.0):
        def near(x, got, scale=None):
            exp = R.rotate(as_f64(x), positions, w, interleaved, amplitude, pair_axes)
            slack = 2.5e-6 * abs(amplitude) * R.pair_size(as_f64(x), 2 * len(w), interleaved)
            if scale is None:
                tol = 2.0 ** -8 * np.abs(exp) + 1.01 * slack
            else:
                exp, slack = np.clip(exp / scale, -448, 448), slack / scale
                tol = np.maximum(2.0 ** -4 * np.abs(exp), 2.0 ** -10) + 1.1 * slack + 2.0 ** -23 * np.abs(exp)
            assert np.all(np.abs(got - exp) <= tol)
        near(self.q, as_f64(out))
        bs = self.case.block_size
        page, slot = self.case.block_tables.numpy()[self.seq, self.slot_pos // bs], self.slot_pos % bs
        if self.case.kv_dtype == W.FP8:
            near(self.k, as_f64(self.b.k_cache.view(torch.float8_e4m3fn).float())[page, slot], self.b.k_scale)
        else:
            near(self.k, as_f64(self.b.k_cache)[page, slot])
            assert torch.equal(self.b.v_cache[page, slot], self.v)


def _places(tokens, axes, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(-100, 100000, size=(axes, tokens))


GRID = [  # rot, d, hq, hkv, bs, dtype, axes
    (128, 128, 8, 2, 16, W.BF16, 3), (128, 128, 4, 4, 32, W.FP8, 3), (64, 128, 5, 1, 16, W.BF16, 2),
    (96, 96, 6, 2, 16, W.FP8, 4), (20, 96, 4, 2, 16, W.BF16, 3), (6, 32, 4, 4, 16, W.FP8, 3),
    (90, 160, 4, 1, 32, W.BF16, 3), (254, 256, 2, 2, 16, W.FP8, 4), (256, 256, 4, 1, 128, W.BF16, 2)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("order", ["runs", "turns", "last"])
@pytest.mark.parametrize("rot,d,hq,hkv,bs,dtype,axes", GRID)
def test_positions_of_each_axis(rot, d, hq, hkv, bs, dtype, axes, order, interleaved):
    s = Step([1, 9, 0, 17, 1, 30], [1, 40, 5, 17, 700, 90], hq, hkv, d, bs, dtype, seed=rot + d)
    n = rot // 2
    w = R.frequencies(rot, 10000.0)[0]
    pair_axes = {"runs": [min(axes - 1, i * axes // n) for i in range(n)], "turns": [i % axes for i in range(n)],
                 "last": [axes - 1] * n}[order]
    pos = _places(58, max(pair_axes) + 1, rot)
    with tu.make_plan(s.b) as plan, ua.Rope(w, interleaved, 1.25, axes=pair_axes) as rope:
        out = s.run(plan, rope, torch.from_numpy(pos).to(torch.int32).cuda())
        assert plan.last_device_error() == 0
    s.check(out, w, interleaved, pair_axes, pos, 1.25)


def test_rows_of_positions_apart_and_more_tokens_than_the_plans():
    s = Step([3, 4], [20, 9], 4, 2, 64, 16, seed=1)
    w, pair_axes = R.frequencies(64, 10000.0)[0], [0, 1, 2, 1] * 8
    pos = _places(7, 3, 5)
    room = torch.full((3, 50), 999999, dtype=torch.int32, device="cuda")
    room[:, 2:9] = torch.from_numpy(pos)
    more = torch.zeros(5, *s.q.shape[1:], dtype=torch.bfloat16, device="cuda")
    with tu.make_plan(s.b) as plan, ua.Rope(w, axes=pair_axes) as rope:
        out = s.run(plan, rope, room[:, 2:9])
        s.check(out, w, False, pair_axes, pos)
        s.q, s.k, s.v = (torch.cat([x, more[:, :x.shape[1]]]) for x in (s.q, s.k, s.v))
        again = s.run(plan, rope, room[:, 2:14])
        assert torch.equal(again[:7], out)
        # positions of the plan's tokens alone do not go with q's twelve
        with pytest.raises(ValueError):
            s.run(plan, rope, room[:, 2:9])


def test_without_positions_every_axis_is_at_the_slot():
    s = Step([1, 40], [333, 90], 4, 2, 128, 16, seed=2)
    w, pair_axes = R.frequencies(128, 10000.0)[0], [i % 3 for i in range(64)]
    with tu.make_plan(s.b) as plan, ua.Rope(w) as one, ua.Rope(w, axes=pair_axes) as three:
        want = s.run(plan, one)
        cache = s.b.k_cache.clone()
        s.b.k_cache.zero_()
        assert torch.equal(s.run(plan, three), want)
        # text: the same position on every axis
        pos = torch.from_numpy(s.slot_pos).to(torch.int32).cuda()
        assert torch.equal(s.run(plan, three, pos.repeat(3, 1)), want)
        assert torch.equal(s.run(plan, one, pos[None]), want)
        assert torch.equal(s.b.k_cache[s.case.block_tables.numpy()[s.seq, s.slot_pos // 16], s.slot_pos % 16],
                           cache[s.case.block_tables.numpy()[s.seq, s.slot_pos // 16], s.slot_pos % 16])


def test_captured_step_takes_new_positions():
    s = Step([2, 30], [50, 30], 4, 2, 128, 16, seed=3)
    w, pair_axes = R.frequencies(128, 10000.0)[0], [i * 3 // 64 for i in range(64)]
    pos = torch.from_numpy(_places(32, 3, 6)).to(torch.int32).cuda()
    with tu.make_plan(s.b) as plan, ua.Rope(w, axes=pair_axes) as rope:
        s.run(plan, rope, pos)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = s.run(plan, rope, pos)
        pos.copy_(torch.from_numpy(_places(32, 3, 7)))
        graph.replay()
        torch.cuda.synchronize()
        s.check(out, w, False, pair_axes, pos.cpu().numpy())


def test_refusals():
    s = Step([3], [20], 4, 2, 64, 16, seed=4)
    w = R.frequencies(64, 10000.0)[0]
    pos = torch.zeros(3, 3, dtype=torch.int32, device="cuda")
    with tu.make_plan(s.b) as plan, ua.Rope(w, axes=[0, 1] * 16) as rope, ua.Rope(w) as one:
        before = s.b.k_cache.clone()
        for bad in (pos, pos[:2, :2], pos[:2].float(), pos[:2].cpu(), pos.T[:2], pos[:1].expand(2, 3),
                    pos[:2, None]):
            with pytest.raises(ValueError):
                s.run(plan, rope, bad)
        with pytest.raises(ua.UAError) as e:  # one row says nothing of the second axis
            s.run(plan, rope, pos[0])
        assert e.value.status == ua.UA_ERR_INVALID_ARG
        with pytest.raises(ValueError):
            s.run(plan, one, pos[:2])
        lib, b, p = ua.lib(), s.b, lambda t: t.data_ptr()  # noqa: E731
        out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
        args = lambda stride, at: (plan.handle, rope.handle, p(s.q), s.q.stride(0), p(s.k), s.k.stride(0),  # noqa: E731
                                   p(s.v), s.v.stride(0), p(out), p(b.k_cache), p(b.v_cache), p(b.block_tables),
                                   b.num_blocks, at, stride, 1.0, 1.0, 0)
        assert lib.ua_rope_append_kv_axes(*args(2, p(pos))) == ua.UA_ERR_INVALID_ARG
        assert lib.ua_rope_append_kv_axes(*args(3, p(pos) + 2)) == ua.UA_ERR_INVALID_ARG
        assert torch.equal(s.b.k_cache, before)
        assert lib.ua_rope_append_kv_axes(*args(3, p(pos))) == ua.UA_OK
        assert lib.ua_rope_append_kv_axes(*args(0, None)) == ua.UA_OK
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0


@pytest.mark.parametrize("axes", [None, [0] * 32])
def test_one_axis_has_no_row_distance(axes):
    """The distance of the rows of positions plays no part where there is one row."""
    s = Step([3, 20], [20, 20], 4, 2, 64, 16, seed=8)
    w = R.frequencies(64, 10000.0)[0]
    pos = torch.from_numpy(_places(23, 1, 9)).to(torch.int32).cuda()
    with tu.make_plan(s.b) as plan, ua.Rope(w, axes=axes) as rope:
        want = s.run(plan, rope, pos[0])
        cache = s.b.k_cache.clone()
        lib, b, p = ua.lib(), s.b, lambda t: t.data_ptr()  # noqa: E731
        for stride in (0, -1, 22, 2 ** 62, -2 ** 63):
            s.b.k_cache.zero_()
            out = torch.zeros_like(want)
            assert lib.ua_rope_append_kv_axes(
                plan.handle, rope.handle, p(s.q), s.q.stride(0), p(s.k), s.k.stride(0), p(s.v), s.v.stride(0), p(out),
                p(b.k_cache), p(b.v_cache), p(b.block_tables), b.num_blocks, p(pos), stride, 1.0, 1.0,
                torch.cuda.current_stream().cuda_stream) == ua.UA_OK
            rows = s.case.block_tables.numpy()[s.seq, s.slot_pos // 16], s.slot_pos % 16
            assert torch.equal(out, want) and torch.equal(b.k_cache[rows], cache[rows])
        assert plan.last_device_error() == 0
