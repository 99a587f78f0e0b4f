"""Rotary positions without a GPU: the oracle against worked values, the host
entry points (frequencies, ropes) against the oracle, and their refusals."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_attention_unified_gb300 as ua
from oracle import rope as R


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_unified_gb300 import build
    build.build()


def test_oracle_quarter_turn_by_hand():
    # a quarter turn per position: (a, b) -> (-b, a) -> (-a, -b)
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    got = R.rotate(np.repeat(x, 2, 0), [1, 2], [math.pi / 2, math.pi / 2], interleaved=False)
    assert np.allclose(got[0, 0], [-3, -4, 1, 2, 5, 6], atol=1e-15)
    assert np.allclose(got[1, 0], [-1, -2, -3, -4, 5, 6], atol=1e-15)
    got = R.rotate(x, [1], [math.pi / 2, math.pi / 2], interleaved=True, amplitude=2.0)
    assert np.allclose(got[0, 0], [-4, 2, -8, 6, 5, 6], atol=1e-15)


def test_oracle_scores_depend_on_distance_only():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 32))
    w, _ = R.frequencies(32, 10000.0)
    for interleaved in (False, True):
        dots = [float(np.sum(R.rotate(q, [p + 7], w, interleaved) * R.rotate(k, [p], w, interleaved)))
                for p in (0, 3, 1000)]
        assert max(dots) - min(dots) < 1e-10


KINDS = [("plain", ua.UA_ROPE_PLAIN, {}), ("linear", ua.UA_ROPE_LINEAR, dict(factor=4.0)),
         ("ntk", ua.UA_ROPE_NTK, dict(factor=8.0)),
         ("bands", ua.UA_ROPE_BANDS, dict(factor=8.0, length=8192.0, low=1.0, high=4.0)),
         ("yarn", ua.UA_ROPE_YARN, dict(factor=16.0, length=4096.0, low=1.0, high=32.0))]


@pytest.mark.parametrize("rot", [4, 20, 64, 128, 256])
@pytest.mark.parametrize("kind,code,args", KINDS)
def test_frequencies(rot, kind, code, args):
    exp, amp = R.frequencies(rot, 500000.0, kind, **args)
    kw = {"original_max_position" if k == "length" else k: v for k, v in args.items()}
    got, m = ua.ua_rope_frequencies(rot, 500000.0, code, **kw)
    assert len(got) == rot // 2
    # pow against exp(log): a few units of 2^-53 times the logarithm (at most 14)
    assert np.allclose(got, exp, rtol=1e-13, atol=0)
    assert m == np.float32(amp)


@pytest.mark.parametrize("bad", [
    dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(rotary_dim=-2),
    dict(base=1.0), dict(base=0.5), dict(base=float("nan")), dict(base=float("inf")),
    dict(scaling=5), dict(scaling=-1),
    dict(scaling=ua.UA_ROPE_LINEAR, factor=0.5), dict(scaling=ua.UA_ROPE_LINEAR, factor=float("nan")),
    dict(scaling=ua.UA_ROPE_NTK, factor=2.0, rotary_dim=2),
    dict(scaling=ua.UA_ROPE_BANDS, factor=2.0),                                   # no length
    dict(scaling=ua.UA_ROPE_BANDS, factor=2.0, original_max_position=100.0, low=4.0, high=4.0),
    dict(scaling=ua.UA_ROPE_YARN, factor=2.0, original_max_position=100.0, low=0.0, high=4.0),
    dict(scaling=ua.UA_ROPE_YARN, factor=float("inf"), original_max_position=100.0),
])
def test_frequencies_refuse(bad):
    with pytest.raises(ua.UAError) as e:
        ua.ua_rope_frequencies(**{"rotary_dim": 64, **bad})
    assert e.value.status == ua.UA_ERR_INVALID_ARG


@pytest.mark.parametrize("w,amp", [([], 1.0), ([0.1] * 129, 1.0), ([float("nan")], 1.0),
                                   ([float("inf")], 1.0), ([6.3], 1.0), ([-6.3], 1.0),
                                   ([0.1], float("nan")), ([0.1], float("inf"))])
def test_ropes_refuse(w, amp):
    with pytest.raises(ua.UAError) as e:
        ua.Rope(w, amplitude=amp)
    assert e.value.status == ua.UA_ERR_INVALID_ARG


def test_ropes_need_a_known_layout():
    h, w = ctypes.c_void_p(), (ctypes.c_double * 1)(0.5)
    assert ua.lib().ua_rope_create(ctypes.byref(h), 2, 2, w, 1.0) == ua.UA_ERR_INVALID_ARG
    assert ua.lib().ua_rope_create(ctypes.byref(h), 2, 0, None, 1.0) == ua.UA_ERR_INVALID_ARG
    assert ua.lib().ua_rope_create(None, 2, 0, w, 1.0) == ua.UA_ERR_INVALID_ARG
    assert h.value is None


def test_ropes_are_made_and_closed():
    with_neg = ua.Rope([2 * math.pi, -0.5, 0.0], interleaved=True, amplitude=-1.5)
    assert with_neg.handle
    with_neg.close()
    with_neg.close()
    assert with_neg.handle is None
    assert ua.Rope.scaled(64, scaling=ua.UA_ROPE_YARN, factor=4.0, original_max_position=4096.0,
                          high=32.0).handle
    assert ua.lib().ua_rope_destroy(None) == ua.UA_OK


def test_append_without_plan_or_rope_is_refused():
    r = ua.Rope([0.5])
    for plan, rope in ((None, r.handle), (None, None)):
        assert ua.lib().ua_rope_append_kv(plan, rope, 16, 64, 16, 64, 16, 64, 16, 16, 16, 16, 1, None,
                                          1.0, 1.0, None) == ua.UA_ERR_INVALID_ARG


def test_host_tensors_are_refused():
    import torch
    q, kv = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cache, table = torch.zeros(1, 16, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        ua.ua_rope_append_kv(None, None, q, kv, kv, torch.empty_like(q), cache, cache, table, 1)


def _kernel_angle(p, w):
    """The rotation kernel's angle arithmetic in binary32 (fma as binary64
    products of binary32 values, exact there), in turns."""
    f = np.float32
    turns = w / (2 * math.pi)
    hi = f(turns)
    lo = f(turns - float(hi))
    p1, p0 = f((p >> 12) * 4096), f(p & 4095)
    t1, t0 = f(p1 * hi), f(p0 * hi)
    e1 = f(float(p1) * float(hi) - float(t1))
    e0 = f(float(p0) * float(hi) - float(t0))
    low = f(f(float(p1) * float(lo) + float(e1)) + f(float(p0) * float(lo) + float(e0)))
    r = f(f(t1 - np.rint(t1)) + f(t0 - np.rint(t0)))
    return f(f(r - np.rint(r)) + low)


def test_angle_arithmetic_keeps_its_error_bound():
    rng = np.random.default_rng(1)
    worst = 0.0
    for _ in range(4000):
        p = int(rng.integers(-2 ** 24, 2 ** 24 + 1))
        w = float(10.0 ** rng.uniform(-7, math.log10(2 * math.pi)))
        # the exact turn count's fraction, from integers: w / 2 pi = num / den
        num, den = (w / (2 * math.pi)).as_integer_ratio()
        frac = (p * num % den) / den
        d = (float(_kernel_angle(p, w)) - frac) % 1.0
        worst = max(worst, min(d, 1.0 - d))
    assert worst < 2.0 ** -22, worst
