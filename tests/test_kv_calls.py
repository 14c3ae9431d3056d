"""Calls of the 4-bit key/value cache that are settled on the host, without a
GPU: what they refuse, and what they answer at once."""
import pytest

import bit_blockwise_weight_nf4_b200 as bnb4
from test_kv_abi import attn


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_blockwise_weight_nf4_b200 import build
    build.build()
    return bnb4.load()


def test_failure_diagnostic_checks_its_limit_and_arguments():
    for limit in (0, -1, 1000001):
        assert bnb4.bnb4_debug_attn_withhold(attn(), limit, None) == bnb4.ERR_INVALID_ARG
    assert bnb4.bnb4_debug_attn_withhold(attn(out=None), 1000, None) == bnb4.ERR_INVALID_ARG
    assert bnb4.bnb4_debug_attn_withhold(attn(window=-1), 1000, None) == bnb4.ERR_SHAPE
    assert bnb4.bnb4_debug_attn_withhold(attn(batch=0, total_q=0), 1000, None) == bnb4.OK
