"""What Plan.rope_append_kv does in Python, without a GPU."""
import torch

import paged_kv_attention_unified_gb300 as ua


def test_a_temporary_rope_lives_through_the_call(monkeypatch):
    """A rope that only the call refers to is not destroyed before the library has read it."""
    plan = ua.Plan.__new__(ua.Plan)
    plan.handle = None
    plan.num_tokens, plan.num_q_heads, plan.num_kv_heads, plan.head_dim = 2, 4, 2, 64
    closed, seen = [], []
    monkeypatch.setattr(ua.Rope, "close", lambda self: closed.append(self.num_axes))

    def library(handle, batch, rope, axes, *rest):
        seen.append((rope, axes, list(closed)))
        return 0

    monkeypatch.setattr(ua, "_rope_append", library)

    def rope():
        r = ua.Rope.__new__(ua.Rope)
        r.handle, r.num_axes = 77, 3
        return r

    plan.rope_append_kv(rope(), torch.zeros(2, 4, 64), None, None, None, None, None, None, 1)
    assert seen == [(77, 3, [])] and closed == [3]
