"""Blocks whose scale is next to the largest power of two (another writer's): their codes are the quotients all the same."""
import pytest
import torch

from tests.test_gpu_append_scaled import DV, Case, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("scale", [2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** 127, 2.0 ** -119, 2.0 ** -100])
def test_codes_under_the_blocks_scale(B, scale):
    c = Case([(0, 4, 2), (1, 7, 1)], 8, seed=1, gain=1.0)
    c.kv = (c.kv.double() * scale).clamp(-3e38, 3e38).to(torch.bfloat16)
    c.kv[:, DV:] = 0
    c.scales.fill_(scale)
    pool0 = c.pool.clone()
    c.call(B)
    if scale >= 2.0 ** -100:
        assert bool((c.scales == scale).all())
        assert torch.equal(c.pool[:4], pool0[:4]) and torch.equal(c.pool[8:15], pool0[8:15])
    now = c.scales[c.slots.long() // 8].double()[:, None]
    want = (c.kv[:, :DV].double() / now).float().to(torch.float8_e4m3fn).float()
    assert torch.equal(values(c.pool[c.slots.long()])[:, :DV], want)
    # (values of 2^-119 under the smallest scale, 2^-100, are 2^-19: below half of the smallest code, 2^-10)
    assert bool((want != 0).any()) == (scale >= 2.0 ** -100)
