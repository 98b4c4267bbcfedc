"""Calls of the scaled attention past the bounds of its plan."""
import pytest
import torch

from tests.test_gpu_scaled import D, DV, SM, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def test_more_work_than_the_plan_counts(B):
    """64 drafts of 128 heads are 256 row blocks: over one tile more than 2^27 allows the call is refused and touches no output."""
    n = (2 ** 27 // 256 - 8 + 1) * 128
    q = torch.zeros((64, 128, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full((64, 128, DV), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((64, 128), 7.0, device="cuda")
    pool, scales = torch.zeros((16, D), dtype=torch.uint8, device="cuda"), torch.ones(16, device="cuda")
    kv = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(1, 128, 64, n), dtype=torch.uint8, device="cuda")
    B.verify_attn_mla_scaled(q, pool, scales, ints([0, n]), kv, ints([0, 64]), out, lse, ws, SM)
    assert B.verify_attn_mla_check(ws) == B.VMLA_ERR_SHAPE
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
