"""Refusals that keep a call from reading what it was not given; none of them needs a GPU."""
import ctypes

import numpy as np
import pytest

from speculative_decoding_mla_gb300 import build as vbuild
from tests.test_shared_cpu import KVH, QOH
from tests.test_shared_cpu import _call as _shared


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 62, 2 ** 63 - 10, 2 ** 63 - 1])
def test_shared_rows_past_every_integer(B, rows):
    """The sum of shared and own rows is not taken before the shared ones are known to fit."""
    assert _shared(B, rows=rows) == B.VMLA_ERR_SHAPE
    size = ctypes.c_size_t(0)
    f = B.lib().verify_attn_mla_shared_workspace_size
    assert f(2, 16, rows, QOH.ctypes.data, KVH.ctypes.data, 0, ctypes.byref(size)) == B.VMLA_ERR_SHAPE
