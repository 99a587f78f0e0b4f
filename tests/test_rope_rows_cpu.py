"""The rows of a rotary append, checked on the host before any launch: tensors
that stand in for device memory, and a library that records the call."""
import ctypes

import pytest
import torch

import paged_kv_attention_unified_gb300 as ua

T, HQ, HKV, D = 3, 8, 2, 64


class OnDevice(torch.Tensor):
    """A host tensor that says it is on device 0."""

    def get_device(self):
        return 0

    is_cuda = property(lambda self: True)


class Library:
    """Stands in for the library: takes every append, and knows one plan."""

    def __init__(self):
        self.appends = []

    def ua_rope_append_kv(self, *args):
        self.appends.append(args)
        return ua.UA_OK

    def ua_plan_get_batch(self, plan, tokens, hq, hkv, d):
        for ref, value in zip((tokens, hq, hkv, d), (T, HQ, HKV, D)):
            ref._obj.value = value
        return ua.UA_OK

    def ua_status_string(self, status):
        return b"refused"


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(ua, "lib", lambda: fake)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(ua, "_stream_handle", lambda stream: 0)
    return fake


def _plan():
    plan = ua.Plan.__new__(ua.Plan)
    plan.handle, plan.num_tokens = None, T
    plan.num_q_heads, plan.num_kv_heads, plan.head_dim = HQ, HKV, D
    return plan


def _rows(heads, d=D, tokens=T):
    return torch.zeros(tokens, heads, d, dtype=torch.bfloat16).as_subclass(OnDevice)


def _through(entry, q, k, v, q_out, positions=None):
    cache = torch.zeros(1, 16, HKV, D, dtype=torch.bfloat16)
    rest = (q, k, v, q_out, cache, cache, torch.zeros(1, 1, dtype=torch.int32), 1, positions)
    if entry == "plan":
        _plan().rope_append_kv(16, *rest)
    else:
        ua.ua_rope_append_kv(16, 16, *rest)


ENTRIES = ["plan", "handle"]


@pytest.mark.parametrize("entry", ENTRIES)
def test_rows_of_the_plans_heads_are_taken(library, entry):
    fused = _rows(HQ + 2 * HKV)
    _through(entry, fused[:, :HQ], fused[:, HQ:HQ + HKV], fused[:, HQ + HKV:], _rows(HQ))
    _through(entry, _rows(HQ), _rows(HKV), _rows(HKV), _rows(HQ))
    more = T + 2  # rows behind the plan's last token
    _through(entry, _rows(HQ, tokens=more), _rows(HKV, tokens=more), _rows(HKV, tokens=more),
             _rows(HQ, tokens=more))
    assert len(library.appends) == 3


@pytest.mark.parametrize("entry", ENTRIES)
@pytest.mark.parametrize("hq,hk,hv,d", [
    (HQ - 1, HKV, HKV, D), (HQ + 1, HKV, HKV, D), (1, HKV, HKV, D),      # q (and q_out, of its shape)
    (HQ, HKV - 1, HKV, D), (HQ, HKV + 1, HKV, D),                        # k_new
    (HQ, HKV, HKV - 1, D), (HQ, HKV, HKV + 1, D),                        # v_new
    (HQ, HKV, HKV, D // 2), (HQ, HKV, HKV, 2 * D)])                      # the head
def test_other_heads_inside_wide_rows_are_refused(library, entry, hq, hk, hv, d):
    """Views into a fused projection's rows, whose distance covers the plan's
    heads: q_out would be written past its end, or a neighbour's columns taken
    for keys and values."""
    wide = _rows(3 * (HQ + 2 * HKV), d)
    q, k, v = wide[:, :hq], wide[:, 20:20 + hk], wide[:, 30:30 + hv]
    with pytest.raises(ua.UAError) as e:
        _through(entry, q, k, v, _rows(hq, d))
    assert e.value.status == ua.UA_ERR_INVALID_ARG
    assert library.appends == []


def test_fewer_tokens_than_the_handles_plan_are_refused(library):
    short = dict(tokens=T - 1)
    with pytest.raises(ua.UAError) as e:
        _through("handle", _rows(HQ, **short), _rows(HKV, **short), _rows(HKV, **short), _rows(HQ, **short))
    assert e.value.status == ua.UA_ERR_INVALID_ARG
    assert library.appends == []


def test_a_null_plan_has_no_batch():
    from paged_kv_attention_unified_gb300 import build
    build.build()
    n, a, b, d = ctypes.c_int64(), ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    refs = [ctypes.byref(x) for x in (n, a, b, d)]
    assert ua.lib().ua_plan_get_batch(None, *refs) == ua.UA_ERR_INVALID_ARG


def test_one_head_may_have_any_distance():
    """[tokens, 1, d] as a transpose of [1, tokens, d]: contiguous rows, whatever the stride of the
    axis of one head says."""
    bf16 = torch.bfloat16
    x = torch.zeros(1, T, D, dtype=bf16).transpose(0, 1)
    assert x.is_contiguous() and x.stride(1) != D
    for rows in (x, torch.zeros(1, T, 2 * D, dtype=bf16).transpose(0, 1)[..., :D]):
        assert ua._token_rows(rows, "k_new", T, -1, bf16)[:2] == (rows.data_ptr(), rows.stride(0))
    with pytest.raises(ValueError):
        ua._token_rows(torch.zeros(T, D, 2, dtype=bf16).transpose(1, 2)[:, :1], "k_new", T, -1, bf16)
    with pytest.raises(ValueError):
        ua._token_rows(torch.zeros(T, 2, 2 * D, dtype=bf16)[..., :D], "k_new", T, -1, bf16)


@pytest.mark.parametrize("cu", [[0, T], iter([0, T]), (0, T, T + 9), [0, T, 0, 0], range(0, 2 * T, T)])
def test_a_plans_tokens_are_those_of_its_sequences(library, cu):
    """Whatever holds the offsets, and whatever follows the last sequence's."""
    def create(handle, cu, kv, n, *rest):
        handle._obj.value = 16
        return ua.UA_OK
    library.ua_plan_create_ex = create
    library.ua_plan_destroy = lambda handle: ua.UA_OK
    with ua.Plan(cu, [20], HQ, num_kv_heads=HKV, head_dim=D, block_size=16, max_blocks_per_seq=2) as plan:
        assert (plan.num_tokens, plan.num_q_heads, plan.num_kv_heads, plan.head_dim) == (T, HQ, HKV, D)
