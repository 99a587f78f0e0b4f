"""GPU parity of rotary append against the fp64 oracle, its refusals, and the
chain it is part of: rotary append, then attention with shaped scores.

Error bound of a rotated element y of the pair (a, b): cos and sin carry the
angle's error (2^-22 turns: 1.5e-6) and the sine function's (2 units of
2^-24), the two products and their sum three roundings of 2^-24, all of them
times at most m (|a| + |b|): 2.5e-6 m (|a| + |b|); then half a step of the
type: 2^-8 |y| for bf16; 2^-4 |y / s|, or 2^-10 below the smallest normal, for
the e4m3 code of y / s (whose quotient adds 2^-24).
"""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua
import workloads as W
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


def _freqs(rot, base=10000.0):
    return R.frequencies(rot, base)[0]


class Step:
    """A batch with its new rows, and what the step must leave behind."""

    def __init__(self, ql, kv, hq, hkv, d, bs, dtype=W.BF16, seed=0, fused=False):
        self.case = W.make_case(f"rope_{d}_{bs}_{dtype}", ql, kv, hq, hkv, d, bs, kv_dtype=dtype, seed=seed)
        self.b = tu.to_device(self.case)
        T = sum(ql)
        g = torch.Generator().manual_seed(seed + 1)
        rows = torch.randn(T, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
        self.q, self.k, self.v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:]
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        self.slot_pos = np.concatenate([np.arange(b - a, b) for a, b in zip(ql, kv)] or [[]]).astype(np.int64)
        self.seq = np.repeat(np.arange(len(ql)), ql)
        self.before = self.caches()
        self.b.k_scale, self.b.v_scale = (0.02, 0.015) if dtype == W.FP8 else (1.0, 1.0)

    def caches(self):
        c = [self.b.k_cache, self.b.v_cache]
        if self.case.kv_dtype == W.FP8:
            c = [x.view(torch.float8_e4m3fn) for x in c]
        return [as_f64(x.float()) for x in c]

    def run(self, plan, rope, q_out=None, positions=None, stream=None):
        q_out = torch.empty(self.q.shape, dtype=torch.bfloat16, device="cuda") if q_out is None else q_out
        b = self.b
        plan.rope_append_kv(rope, self.q, self.k, self.v, q_out, b.k_cache, b.v_cache, b.block_tables,
                            b.num_blocks, positions=positions, k_scale=b.k_scale, v_scale=b.v_scale,
                            stream=stream)
        return q_out

    def check(self, q_in, q_out, w, interleaved, amplitude=1.0, positions=None, skip=()):
        pos = self.slot_pos if positions is None else positions
        turn = lambda x: R.rotate(as_f64(x), pos, w, interleaved, amplitude)  # noqa: E731
        slack = lambda x: 2.5e-6 * abs(amplitude) * R.pair_size(as_f64(x), 2 * len(w), interleaved)  # noqa: E731
        exp = turn(q_in)
        assert np.all(np.abs(as_f64(q_out) - exp) <= 2.0 ** -8 * np.abs(exp) + 1.01 * slack(q_in))
        bs, bt = self.case.block_size, self.case.block_tables.numpy()
        keep = np.array([i for i in range(len(pos)) if self.seq[i] not in skip], dtype=np.int64)
        page = bt[self.seq[keep], self.slot_pos[keep] // bs]
        slot = self.slot_pos[keep] % bs
        for got, old, x, exp, tol, scale in zip(
                self.caches(), self.before, (self.k, self.v), (turn(self.k), as_f64(self.v)),
                (slack(self.k), 0.0 * as_f64(self.v)), (self.b.k_scale, self.b.v_scale)):
            exp, tol = exp[keep], tol[keep]
            if self.case.kv_dtype == W.FP8:
                exp, tol = np.clip(exp / scale, -448, 448), tol / scale
                tol = np.maximum(2.0 ** -4 * np.abs(exp), 2.0 ** -10) + 1.1 * tol + 2.0 ** -23 * np.abs(exp)
            else:
                tol = 2.0 ** -8 * np.abs(exp) + 1.01 * tol
            assert np.all(np.abs(got[page, slot] - exp) <= tol)
            rest = np.ones(got.shape[:2], dtype=bool)
            rest[page, slot] = False
            assert np.array_equal(got[rest], old[rest], equal_nan=True)


GRID = [  # rot, d, hq, hkv, bs, dtype
    (128, 128, 8, 2, 16, W.BF16), (128, 128, 4, 4, 32, W.FP8), (64, 128, 5, 1, 16, W.BF16),
    (64, 64, 8, 8, 64, W.FP8), (32, 32, 3, 1, 16, W.BF16), (96, 96, 6, 2, 16, W.FP8),
    (2, 64, 2, 1, 16, W.BF16), (20, 96, 4, 2, 16, W.BF16), (6, 32, 4, 4, 16, W.FP8),
    (90, 160, 4, 1, 32, W.BF16), (160, 160, 2, 2, 16, W.BF16), (192, 192, 3, 3, 16, W.BF16),
    (224, 224, 2, 1, 16, W.FP8), (254, 256, 2, 2, 16, W.FP8), (256, 256, 4, 1, 128, W.BF16),
    (16, 256, 1, 1, 16, W.BF16), (48, 224, 40, 8, 16, W.BF16)]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d,hq,hkv,bs,dtype", GRID)
def test_rope_append(rot, d, hq, hkv, bs, dtype, interleaved):
    s = Step([1, 9, 0, 17, 1, 30], [1, 40, 5, 17, 700, 90], hq, hkv, d, bs, dtype, seed=rot + d)
    w = _freqs(rot)
    with tu.make_plan(s.b) as plan, ua.Rope(w, interleaved) as rope:
        out = s.run(plan, rope)
        assert plan.last_device_error() == 0
    s.check(s.q, out, w, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [64, 44])
def test_strided_rows_positions_and_amplitude(rot, interleaved):
    s = Step([5, 1, 33], [50, 77, 33], 6, 2, 96, 16, seed=3, fused=True)
    pos = np.array([0, -1, 5, 10 ** 6 + 1, 131071] + [2 ** 24] + list(range(-3, 30)), dtype=np.int64)
    w = [2 * math.pi] + _freqs(rot, 500000.0)[:-2] + [-0.25]
    with tu.make_plan(s.b) as plan, ua.Rope(w, interleaved, amplitude=1.25) as rope:
        out = s.run(plan, rope, positions=torch.from_numpy(pos).to(torch.int32).cuda())
    s.check(s.q, out, w, interleaved, 1.25, pos)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (128, True), (36, False), (36, True)])
def test_in_place(rot, interleaved):
    s = Step([64, 1, 7], [64, 900, 8], 16, 4, 128, 16, seed=4)
    q_in = s.q.clone()
    with tu.make_plan(s.b) as plan, ua.Rope(_freqs(rot), interleaved) as rope:
        out = s.run(plan, rope, q_out=s.q)
    assert out.data_ptr() == s.q.data_ptr()
    s.check(q_in, out, _freqs(rot), interleaved)


def test_pairs_of_infinities_and_nan_stay_in_their_pair():
    s = Step([2], [2], 2, 2, 64, 16, seed=5)
    s.q[0, 0, 3] = float("inf")
    s.k[0, 1, 40] = float("nan")
    with tu.make_plan(s.b) as plan, ua.Rope(_freqs(32)) as rope:  # elements from 32 on pass unchanged
        out = s.run(plan, rope)
    bad = ~torch.isfinite(out.float())
    assert bad[0, 0, 3] and set(torch.nonzero(bad[0, 0]).flatten().tolist()) <= {3, 19}
    assert int(bad.sum()) <= 2
    bad = ~torch.isfinite(s.b.k_cache[int(s.case.block_tables[0, 0]), :2].float())
    assert torch.nonzero(bad).tolist() == [[0, 1, 40]]


def test_saturation_and_nan_of_e4m3_codes():
    s = Step([1], [1], 1, 1, 32, 16, W.FP8, seed=6)
    s.k[0, 0, 0], s.k[0, 0, 1], s.k[0, 0, 31] = 1e4, float("nan"), -1e4
    with tu.make_plan(s.b) as plan, ua.Rope([0.0]) as rope:  # no turn
        s.run(plan, rope)
    got = s.caches()[0][int(s.case.block_tables[0, 0]), 0, 0]
    # the pair (0, 1) of the half layout holds the NaN: it stays in its place
    assert np.isnan(got[1]) and got[31] == -448.0
    assert got[0] == 448.0 or np.isnan(got[0])  # 1e4 * 1 - nan * 0


def test_bad_page_is_reported_and_the_query_still_turned():
    s = Step([4, 4], [20, 36], 4, 4, 64, 16, seed=7)
    s.b.block_tables[1, 35 // 16] = 10 ** 6
    w = _freqs(64)
    with tu.make_plan(s.b) as plan, ua.Rope(w) as rope:
        out = s.run(plan, rope)
        assert plan.last_device_error() == ua.UA_ERR_BOUNDS
    s.check(s.q, out, w, False, skip=(1,))


def test_captured_append_replays_on_new_rows_after_the_rope_is_gone():
    s = Step([1] * 20, [30 + 7 * i for i in range(20)], 8, 2, 128, 16, W.FP8, seed=8)
    w = _freqs(128)
    plan, rope = tu.make_plan(s.b), ua.Rope(w)
    out = s.run(plan, rope)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(plan, rope, q_out=out)
    rope.close()
    for t in (s.q, s.k, s.v):
        t.neg_()
    graph.replay()
    torch.cuda.synchronize()
    s.check(s.q, out, w, False)
    plan.close()


def test_another_stream_and_rows_behind_the_last_sequence():
    s = Step([3, 2], [10, 40], 4, 2, 64, 16, seed=9)
    room = torch.full((9, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with tu.make_plan(s.b, stream=side) as plan, ua.Rope(_freqs(64)) as rope:
        s.run(plan, rope, q_out=room[:5], stream=side)
        torch.cuda.synchronize()
    s.check(s.q, room[:5], _freqs(64), False)
    assert torch.all(room[5:] == 5.0)


def test_empty_batch_does_nothing():
    s = Step([0, 0], [5, 0], 2, 1, 64, 16, seed=10)
    with tu.make_plan(s.b) as plan, ua.Rope(_freqs(64)) as rope:
        s.run(plan, rope)
        assert plan.last_device_error() == 0
    for got, old in zip(s.caches(), s.before):
        assert np.array_equal(got, old, equal_nan=True)


def test_refusals():
    s = Step([4], [20], 4, 2, 64, 16, seed=11)
    b, out = s.b, torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    args = dict(q=s.q, k_new=s.k, v_new=s.v, q_out=out, k_cache=b.k_cache, v_cache=b.v_cache,
                block_tables=b.block_tables, num_blocks=b.num_blocks)
    shifted = torch.empty(4 * 4 * 64 + 8, dtype=torch.bfloat16, device="cuda")
    wide = torch.empty(4, 8, 64, dtype=torch.bfloat16, device="cuda")  # q and q_out share its rows
    one = torch.empty(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    with tu.make_plan(b) as plan, ua.Rope(_freqs(64)) as rope, ua.Rope(_freqs(96)) as wider:
        def refused(exc, rope=rope, **kw):
            with pytest.raises(exc) as e:
                plan.rope_append_kv(rope, **{**args, **kw})
            if exc is ua.UAError:
                assert e.value.status == ua.UA_ERR_INVALID_ARG
        refused(ua.UAError, rope=wider)                                  # wider than the head
        refused(ua.UAError, num_blocks=0)
        refused(ua.UAError, q=shifted[4:4 + 1024].view(4, 4, 64))        # misaligned
        refused(ua.UAError, q=shifted[8:8 + 1024].view(4, 4, 64), q_out=shifted[:1024].view(4, 4, 64))
        refused(ua.UAError, q=wide[:, :4], q_out=wide.view(-1)[:1024].view(4, 4, 64))  # strided in place
        refused(ua.UAError, k_new=out[:, :2], q_out=out)                 # q_out over the new keys
        refused(ua.UAError, q=one, q_out=torch.empty_like(one))          # rows too short
        refused(ValueError, q=one)                                       # q_out of another shape
        refused(ValueError, q=s.q.transpose(1, 2))
        refused(ValueError, q=s.q[..., ::2])
        refused(ValueError, q=s.q.float())
        refused(ValueError, positions=torch.zeros(4, dtype=torch.int64, device="cuda"))
        refused(ValueError, positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
        refused(ValueError, k_new=s.k[:3])
        refused(ValueError, q_out=wide[:, :4])
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0
    for got, old in zip(s.caches(), s.before):
        assert np.array_equal(got, old, equal_nan=True)
    s = Step([1], [5], 2, 1, 64, 16, W.FP8, seed=12)
    with tu.make_plan(s.b) as plan, ua.Rope(_freqs(64)) as rope:
        for ks in (0.0, float("nan"), float("inf")):
            s.b.k_scale = ks
            with pytest.raises(ua.UAError) as e:
                s.run(plan, rope)
            assert e.value.status == ua.UA_ERR_INVALID_ARG


@pytest.mark.parametrize("d,dtype", [(128, W.BF16), (128, W.FP8), (96, W.BF16), (256, W.BF16)])
def test_a_layer_step_by_step(d, dtype):
    """What a serving loop does: a prompt in two chunks, then single tokens, each step rotary
    append and attention with a cap and a prefix over the cache that the steps before filled."""
    hq, hkv, bs, cap, prefix = 4, 2, 16, 20.0, 30
    lens = [40, 33, 1, 1]
    total = sum(lens)
    blocks = -(-total // bs) + 2
    g = torch.Generator().manual_seed(13)
    rows = torch.randn(total, hq + 2 * hkv, d, generator=g).to(torch.bfloat16).cuda()
    fp8 = dtype == W.FP8
    ks, vs = (0.02, 0.02) if fp8 else (1.0, 1.0)
    kc, vc = (torch.zeros(blocks, bs, hkv, d, device="cuda").to(
        torch.float8_e4m3fn if fp8 else torch.bfloat16) for _ in range(2))
    table = torch.randperm(blocks, generator=g)[:-(-total // bs)].to(torch.int32).view(1, -1).cuda()
    w, done = _freqs(d // 2), 0
    with ua.Rope(w, interleaved=True) as rope:
        for n in lens:
            new = rows[done:done + n]
            done += n
            q_out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q_out)
            dev = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
            with ua.Plan([0, n], [done], hq, hkv, d, bs, table.shape[1],
                         kv_dtype=ua.UA_KV_FP8_E4M3 if fp8 else ua.UA_KV_BF16, prefix_lens=[prefix]) as plan:
                plan.set_scores(softcap=cap)
                plan.rope_append_kv(rope, new[:, :hq], new[:, hq:hq + hkv], new[:, hq + hkv:], q_out, kc, vc,
                                    table, blocks, k_scale=ks, v_scale=vs)
                plan.forward(q_out, kc, vc, out, dev(0, n), dev(done), table, blocks, n, done, d ** -0.5,
                             k_scale=ks, v_scale=vs)
                assert plan.last_device_error() == 0
            # the whole chain from the unrotated rows; keys and values as the cache holds them
            pos = np.arange(done)
            turn = lambda x, p: R.rotate(as_f64(x), p, w, True)  # noqa: E731
            page, slot = table[0, torch.arange(done, device="cuda") // bs].long(), torch.arange(done, device="cuda") % bs
            held = [as_f64(c[page, slot].float()) * s for c, s in ((kc, ks), (vc, vs))]
            exp_k = turn(rows[:done, hq:hq + hkv], pos)
            step = 2.0 ** -4 if fp8 else 2.0 ** -8
            assert np.all(np.abs(held[0] - exp_k) <= step * np.abs(exp_k) + 2.0 ** -10 * ks + 1e-4)
            q = as_f64(q_out)
            assert np.all(np.abs(q - turn(new[:, :hq], pos[done - n:])) <= 2.0 ** -8 * np.abs(q) * 1.01 + 1e-4)
            for i in range(n):
                t = S.visible_with_prefix(done, n, i, True, 0, prefix)
                for h in range(hq):
                    x = S.shape_scores(held[0][t, h // 2] @ q[i, h] * d ** -0.5, done - n + i - t, cap, 0.0)
                    p = np.exp(x - x.max())
                    p /= p.sum()
                    v = held[1][t, h // 2]
                    exp, spread = p @ v, p @ np.abs(v)
                    tol = 2.0 ** -8 * np.abs(exp) + 1.01 * (2.0 ** -8 + 2.0 ** -10) * spread + 1e-4 * fp8
                    assert np.all(np.abs(as_f64(out[i, h]) - exp) <= tol)


def test_torch_helpers_turn_in_place_and_append():
    s = Step([3, 1, 40], [60, 33, 40], 8, 2, 128, 16, W.FP8, seed=14)
    q_in = s.b.q.copy_(s.q).clone()
    with tu.make_plan(s.b, prefix_lens=[10, 0, 5]) as plan, ua.Rope(_freqs(96)) as rope:
        tu.rope_append_kv(plan, s.b, rope, s.b.q, s.k, s.v)
        assert plan.last_device_error() == 0
    s.check(q_in, s.b.q, _freqs(96), False)


@pytest.mark.parametrize("nrows", range(1, 9))
def test_every_number_of_tokens_in_a_tile(nrows):
    """The warps of a tile share its tokens: 1, 2, 3 .. 8 of them, and a tile more."""
    s = Step([nrows, 8 + nrows], [nrows, 50 + nrows], 5, 1, 64, 16, seed=20 + nrows)
    for interleaved in (False, True):
        with tu.make_plan(s.b) as plan, ua.Rope(_freqs(64), interleaved) as rope:
            out = s.run(plan, rope)
            assert plan.last_device_error() == 0
        s.check(s.q, out, _freqs(64), interleaved)


def test_a_cache_behind_2_31_elements():
    """Slots whose element offset passes 32 bits."""
    hkv, d, bs, blocks = 16, 256, 256, 2100  # 2.2e9 elements a cache
    kc, vc = (torch.zeros(blocks, bs, hkv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(15)
    rows = torch.randn(2, 2 * hkv + 16, d, generator=g).to(torch.bfloat16).cuda()
    q, k, v = rows[:, :16].contiguous(), rows[:, 16:16 + hkv], rows[:, 16 + hkv:]
    table = torch.tensor([[blocks - 1]], dtype=torch.int32, device="cuda")
    w, out = _freqs(256), torch.empty(2, 16, d, dtype=torch.bfloat16, device="cuda")
    with ua.Plan([0, 2], [200], 16, hkv, d, bs, 1) as plan, ua.Rope(w) as rope:
        plan.rope_append_kv(rope, q, k, v, out, kc, vc, table, blocks)
        assert plan.last_device_error() == 0
    exp = R.rotate(as_f64(k), [198, 199], w, False)
    got = as_f64(kc[blocks - 1, 198:200])
    assert np.all(np.abs(got - exp) <= 2.0 ** -8 * np.abs(exp) + 2.5e-6 * R.pair_size(as_f64(k), 256, False))
    assert torch.equal(vc[blocks - 1, 198:200], v)
    assert int(kc[:blocks - 1].count_nonzero()) == 0


def test_tensors_of_another_device_or_of_fewer_tokens_are_refused():
    s = Step([4], [20], 4, 2, 64, 16, seed=12)
    b, out = s.b, torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda")
    args = dict(q=s.q, k_new=s.k, v_new=s.v, q_out=out, k_cache=b.k_cache, v_cache=b.v_cache,
                block_tables=b.block_tables, num_blocks=b.num_blocks,
                positions=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with tu.make_plan(b) as plan, ua.Rope(_freqs(64)) as rope:
        for name in ("q", "k_new", "v_new", "q_out", "positions"):
            with pytest.raises(ValueError):
                plan.rope_append_kv(rope, **{**args, name: args[name].cpu()})
        short = {k: args[k][:3] for k in ("q", "k_new", "v_new", "q_out", "positions")}
        with pytest.raises(ValueError):
            plan.rope_append_kv(rope, **{**args, **short})
        for got, old in zip(s.caches(), s.before):
            assert np.array_equal(got, old, equal_nan=True)
        plan.rope_append_kv(rope, **args)  # and as they were, they are taken
        assert plan.last_device_error() == 0


def test_a_plan_and_an_append_before_torch_has_touched_the_gpu():
    """The stream is found without torch's CUDA state being set up by anyone."""
    import subprocess
    import sys
    code = """
import paged_kv_attention_unified_gb300 as ua
plan = ua.Plan([0, 2], [200], 4, 2, 64, 256, 1)
import torch
q = torch.randn(2, 4, 64, dtype=torch.bfloat16, device="cuda")
kv = torch.randn(2, 2, 64, dtype=torch.bfloat16, device="cuda")
cache = torch.zeros(2, 1, 256, 2, 64, dtype=torch.bfloat16, device="cuda")
out = torch.empty_like(q)
table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
plan.rope_append_kv(ua.Rope([1.0]), q, kv, kv, out, cache[0], cache[1], table, 1)
assert torch.equal(cache[1, 0, 198:200], kv) and plan.last_device_error() == 0
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300,
                       cwd=__import__("os").path.dirname(__import__("os").path.dirname(__file__)))
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,d", [(2, 32), (36, 64), (90, 96), (64, 96), (102, 224)])
def test_infinities_stay_in_their_pair_and_zeros_keep_their_sign(rot, d, interleaved):
    s = Step([3, 9], [3, 40], 6, 2, d, 16, seed=13)
    q = s.q.clone()
    q[:, :, rot:] = torch.tensor([-0.0, 0.0, 1.5, -float("inf")], device="cuda").repeat(d)[:d - rot].bfloat16()
    pair = min(3, rot // 2 - 1)
    a, b = (2 * pair, 2 * pair + 1) if interleaved else (pair, pair + rot // 2)
    q[::2, :, b] = float("inf")
    s.q = q
    with tu.make_plan(s.b) as plan, ua.Rope(_freqs(rot), interleaved) as rope:
        out = s.run(plan, rope)
    assert torch.equal(out[:, :, rot:].contiguous().view(torch.int16), q[:, :, rot:].contiguous().view(torch.int16))
    rest = [e for e in range(rot) if e not in (a, b)]
    assert torch.isfinite(out[:, :, rest].float()).all()
    assert not torch.isfinite(out[::2, :, [a, b]].float()).all(-1).any()


@pytest.mark.parametrize("k_scale,v_scale", [
    (1.0, 0.015), (0.0071, 3.3), (448.0, -0.37), (2.0 ** -126, 2.0 ** 127), (1.9999999, 2.0 ** -20),
    (3e38, 1.2e-38), (1.0000001, 7e-5)])
def test_e4m3_codes_of_every_bf16_value_are_those_of_the_plain_append(k_scale, v_scale):
    """Values that pass unrotated: every bf16 number, infinities and NaN too."""
    n = 512
    values = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    rows = values.view(n, 2, 64)
    keys = torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    keys[:, :, 2:] = rows[:, :, 2:]                        # the first two elements turn
    q = torch.zeros(n, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    caches = torch.zeros(4, 4, 128, 2, 64, dtype=torch.uint8, device="cuda")
    with ua.Plan([0, n], [n], 2, 2, 64, 128, 4, kv_dtype=ua.UA_KV_FP8_E4M3) as plan, \
            ua.Rope([0.5], interleaved=True) as rope:
        plan.rope_append_kv(rope, q, keys, rows, torch.empty_like(q), caches[0], caches[1], table, 4,
                            k_scale=k_scale, v_scale=v_scale)
        plan.append_kv(keys, rows, caches[2], caches[3], table, 4, k_scale, v_scale)
        assert plan.last_device_error() == 0
    assert torch.equal(caches[1], caches[3])
    assert torch.equal(caches[0][..., 2:], caches[2][..., 2:])
    assert not (caches[0][..., :2] & 127).any()  # a turned zero is a zero of either sign


@pytest.mark.parametrize("scale", [0.0, float("inf"), float("nan"), 1e-39])
def test_scales_that_are_not_normal_numbers_are_refused(scale):
    s = Step([4], [20], 4, 2, 64, 16, W.FP8, seed=14)
    for name in ("k_scale", "v_scale"):
        s.b.k_scale, s.b.v_scale = 1.0, 1.0
        setattr(s.b, name, scale)
        with tu.make_plan(s.b) as plan, ua.Rope(_freqs(64)) as rope:
            with pytest.raises(ua.UAError) as e:
                s.run(plan, rope)
            assert e.value.status == ua.UA_ERR_INVALID_ARG
