"""Rotary append: rows that are not the plan's are refused before a launch, and
every way of holding the plan's rows is taken."""
import pytest
import torch

import paged_kv_attention_unified_gb300 as ua

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_attention_unified_gb300 import build
    build.build()


HQ, HKV, D, T, BS = 4, 2, 64, 5, 16


class Append:
    def __init__(self, hkv=HKV):
        g = torch.Generator().manual_seed(3)
        randn = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()  # noqa: E731
        self.fused = randn(T, 4 * (HQ + 2 * hkv), D)
        self.hkv = hkv
        self.cache = torch.zeros(2, 3, BS, hkv, D, dtype=torch.bfloat16, device="cuda")
        self.table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
        self.plan = ua.Plan([0, T], [20], HQ, hkv, D, BS, 2)
        self.rope = ua.Rope([0.5 ** i for i in range(D // 2)])

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.plan.close()

    def rows(self, hq=HQ, hk=None, hv=None):
        k, f = self.hkv, self.fused
        return f[:, :hq], f[:, HQ:HQ + (k if hk is None else hk)], f[:, HQ + k:HQ + k + (k if hv is None else hv)]

    def call(self, q, k, v, q_out, through="plan"):
        rest = (self.rope.handle, q, k, v, q_out, self.cache[0], self.cache[1], self.table, 3)
        if through == "plan":
            self.plan.rope_append_kv(*rest)
        else:
            ua.ua_rope_append_kv(self.plan.handle, *rest)
        return q_out


@pytest.mark.parametrize("through", ["plan", "handle"])
def test_views_of_other_heads_are_refused(through):
    with Append() as s:
        assert ua.ua_plan_get_batch(s.plan.handle) == (T, HQ, HKV, D)
        for heads in (dict(hq=1), dict(hq=HQ - 1), dict(hq=HQ + 1), dict(hk=1), dict(hk=3), dict(hv=1), dict(hv=3)):
            q, k, v = s.rows(**heads)
            out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
            with pytest.raises(ua.UAError) as e:
                s.call(q, k, v, out, through)
            assert e.value.status == ua.UA_ERR_INVALID_ARG
            assert torch.all(out == 7.0)
        assert int(s.cache.count_nonzero()) == 0
        q, k, v = s.rows()
        s.call(q, k, v, torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda"), through)
        at = lambda c: torch.cat([c[2, 15:], c[0, :4]])  # noqa: E731  positions 15 .. 19
        assert torch.equal(at(s.cache[1]), v)
        assert s.plan.last_device_error() == 0


def test_one_key_head_from_a_transpose():
    with Append(hkv=1) as s:
        q = s.rows()[0].contiguous()
        k, v = (torch.randn(1, T, D, device="cuda").to(torch.bfloat16).transpose(0, 1) for _ in range(2))
        want = torch.empty(T, HQ, D, dtype=torch.bfloat16, device="cuda")
        s.call(q, k.clone(memory_format=torch.contiguous_format).view(T, 1, D), v.reshape(T, 1, D), want)
        cache = s.cache.clone()
        s.cache.zero_()
        assert torch.equal(s.call(q, k, v, torch.empty_like(want)), want)
        assert torch.equal(s.cache, cache)
