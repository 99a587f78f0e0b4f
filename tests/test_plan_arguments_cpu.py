"""How a plan's host arguments are taken: no GPU, no launch."""
import pytest

import paged_kv_attention_unified_gb300 as ua


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_attention_unified_gb300 import build
    build.build()


@pytest.mark.parametrize("prefix", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32 + 5, -2 ** 40])
def test_a_negative_prefix_is_refused_whatever_its_size(prefix):
    """Also where its low 32 bits are a number that would do."""
    with pytest.raises(ua.UAError) as e:
        ua.ua_schedule([0, 4], [4], 4, 4, 64, 16, 1, prefix_lens=[prefix])
    assert e.value.status == ua.UA_ERR_INVALID_ARG
