"""Block scales of an e4m3 cache: the oracle's rule by hand and by properties, and
the refusals that need no GPU."""
import ctypes

import numpy as np
import pytest

import paged_kv_attention_unified_gb300 as ua
from oracle import block_scales as B
from oracle.fp8_products import round_e4m3


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_unified_gb300 import build
    build.build()


@pytest.mark.parametrize("amax,want", [
    (448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (224.5, 1.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
    (1.7578125, 2.0 ** -7), (0.0, 2.0 ** -100), (2.0 ** -130, 2.0 ** -100), (3e38, 2.0 ** 100)])
def test_scale_of_a_new_block(amax, want):
    assert B.next_scale(amax, 123.0, 0) == (want, 0)
    assert B.next_scale(amax, float("nan"), 3) == (want, 0)  # no scale to keep
    assert B.next_scale(amax, 0.0, 3) == (want, 0)


@pytest.mark.parametrize("amax,old,want", [
    (0.0, 0.5, (0.5, 0)), (224.0, 0.5, (0.5, 0)), (225.0, 0.5, (1.0, 1)), (448.0 * 6, 1.0, (8.0, 3)),
    (2.0 ** -126, 2.0 ** -100, (2.0 ** -100, 0)), (100.0, 0.25, (0.25, 0)), (112.5, 0.25, (0.5, 1))])
def test_scale_of_a_block_with_earlier_tokens(amax, old, want):
    assert B.next_scale(amax, old, 5) == want


def test_upper_limit_holds_for_grown_scales():
    scale, n = B.next_scale(3e38, 3.0, 1)
    assert scale <= 2.0 ** 100 < 2 * scale and scale == 3.0 * 2.0 ** n


def test_append_by_hand():
    codes = np.zeros((2, 16, 1, 2))
    codes[1, :2, 0] = [[448.0, 3.0], [-1.0, 2.0 ** -9]]
    scales = np.array([[7.0], [0.5]])
    x = np.array([[[900.0, 1.0]], [[2.0, -4.0]]])
    got, s = B.append(x, codes, scales, [0, 2], [4], np.array([[1]]), 16)
    assert s[1, 0] == 4.0 and s[0, 0] == 7.0  # 900 / 448 > 2: three doublings
    assert got[1, 0, 0].tolist() == [56.0, 0.375] and got[1, 1, 0].tolist() == [-0.125, 0.0]
    assert got[1, 2, 0].tolist() == [225.0, 0.25] and got[1, 3, 0].tolist() == [0.5, -1.0]


def test_earlier_codes_keep_their_values_but_for_subnormals():
    rng = np.random.default_rng(0)
    codes = round_e4m3(rng.normal(size=(1, 16, 2, 32)) * 40)
    x = rng.normal(size=(3, 2, 32)) * 300
    got, s = B.append(x, codes, np.ones((1, 2)), [0, 3], [12], np.array([[0]]), 16)
    was, now = codes[0, :9], got[0, :9] * s[0][:, None]
    assert s.max() > 1 and np.all((was == now) | (np.abs(was) < 2.0 ** -6 * s[0][:, None]))
    assert np.array_equal(got[0, 12:], codes[0, 12:])


def test_refusals_without_a_plan():
    lib, some = ua.lib(), ctypes.c_void_p(64)
    assert lib.ua_plan_set_block_scales(None, some, some, 4) == ua.UA_ERR_INVALID_ARG
    assert lib.ua_plan_set_block_scales(None, None, None, 0) == ua.UA_ERR_INVALID_ARG
    assert lib.ua_rope_get_axes(None, ctypes.byref(ctypes.c_int32())) == ua.UA_ERR_INVALID_ARG


def test_axes_of_a_rope():
    w = [0.5 ** i for i in range(8)]
    with ua.Rope(w) as one, ua.Rope(w, axes=[0] * 8) as same, ua.Rope(w, axes=[0, 1, 2, 3] * 2) as four, \
            ua.Rope.scaled(16, axes=[2] * 8) as third:
        assert [ua.ua_rope_get_axes(r.handle) for r in (one, same, four, third)] == [1, 1, 4, 3]
    for axes in ([0] * 7, [0] * 9, []):
        with pytest.raises(ValueError):
            ua.Rope(w, axes=axes)
    for axes in ([-1] + [0] * 7, [4] + [0] * 7, [2 ** 40] * 8, [-2 ** 40] * 8):
        with pytest.raises(ua.UAError) as e:
            ua.Rope(w, axes=axes)
        assert e.value.status == ua.UA_ERR_INVALID_ARG
    lib, h = ua.lib(), ctypes.c_void_p(7)
    freq, ax = (ctypes.c_double * 8)(*w), (ctypes.c_int32 * 8)()
    for args in ((16, 0, freq, 1.0, 0, ax), (16, 0, freq, 1.0, 5, ax), (16, 0, freq, 1.0, 2, None),
                 (16, 0, None, 1.0, 2, ax), (15, 0, freq, 1.0, 2, ax), (258, 0, freq, 1.0, 2, ax),
                 (16, 2, freq, 1.0, 2, ax), (16, 0, freq, float("nan"), 2, ax)):
        assert lib.ua_rope_create_axes(ctypes.byref(h), *args) == ua.UA_ERR_INVALID_ARG and not h.value
    assert lib.ua_rope_create_axes(None, 16, 0, freq, 1.0, 2, ax) == ua.UA_ERR_INVALID_ARG
