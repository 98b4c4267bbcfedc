"""The most keys that a call of the scaled attention takes: refused on the host, without a GPU."""
import ctypes

import pytest

from speculative_decoding_mla_gb300 import build as vbuild
from tests.test_scaled_cpu import ATTEND


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("keys", [2 ** 31 - 511, 2 ** 31 - 128, 2 ** 31 - 1, 2 ** 31])
def test_more_keys_than_positions_hold(B, keys):
    n = ctypes.c_size_t(0)
    assert B.lib().verify_attn_mla_scaled(*{**ATTEND, "max_kv": keys}.values()) == B.VMLA_ERR_SHAPE
    assert B.lib().verify_attn_mla_scaled_workspace_size(2, 16, 6, keys, ctypes.byref(n)) == B.VMLA_ERR_SHAPE


def test_the_most_keys_that_are_taken(B):
    n = ctypes.c_size_t(0)
    assert B.MAX_SCALED_KV == 2 ** 31 - 512
    assert B.lib().verify_attn_mla_scaled_workspace_size(2, 16, 6, B.MAX_SCALED_KV, ctypes.byref(n)) in (B.VMLA_OK, B.VMLA_ERR_DEVICE)
