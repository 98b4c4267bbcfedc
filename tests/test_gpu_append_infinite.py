"""Infinities among the rows of a block: they are coded as the largest code, and the other rows, old and new, are what they
would be without them."""
import math

import pytest
import torch

from tests.test_gpu_append_scaled import DV, Case, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("block,runs", [(2, [(0, 1, 1), (3, 0, 2)]), (8, [(2, 3, 2), (0, 0, 8), (1, 7, 1)]), (64, [(1, 20, 9), (2, 0, 64), (0, 63, 1)]),
                                        (128, [(1, 5, 123), (2, 0, 128), (3, 100, 1)]), (16, [(b, b % 16, 16 - b % 16) for b in range(250)])])
def test_other_rows_are_as_without_them(B, block, runs):
    T = sum(n for _, _, n in runs)
    at = [(0, 0, math.inf), (0, DV - 1, -math.inf), (T - 1, 77, -math.inf), (T // 2, 300, math.inf), (T // 2, 301, math.inf)]
    c, want = Case(runs, block, heads=3, seed=block), Case(runs, block, heads=3, seed=block)
    for t, col, v in at:
        c.kv[t, col] = v
        want.kv[t, col] = 0
    c.call(B)
    want.call(B)
    assert c.status.tolist() == [0, 0] and torch.equal(c.scales, want.scales) and torch.equal(c.q, want.q)
    got, pool = values(c.pool), values(want.pool)
    for t, col, v in at:
        s = int(c.slots[t])
        assert float(got[s, col]) == math.copysign(448.0, v)
        got[s, col] = pool[s, col]
    assert torch.equal(got.nan_to_num(1e9), pool.nan_to_num(1e9))
    assert not torch.equal(want.scales, Case(runs, block, seed=block).scales)


def test_in_the_rotated_columns_and_alone(B):
    """An infinity among the turned columns (its pair turns infinite or NaN), and rows of nothing else."""
    for value in (math.inf, -math.inf):
        c, want = Case([(0, 2, 3), (1, 0, 4)], 8, seed=1), Case([(0, 2, 3), (1, 0, 4)], 8, seed=1)
        c.kv[1, DV + 10] = value
        want.kv[1, DV + 10] = want.kv[1, DV + 11] = 0
        c.kv[1, DV + 11] = 0
        c.call(B)
        want.call(B)
        assert torch.equal(c.scales, want.scales)
        s = int(c.slots[1])
        got, pool = values(c.pool), values(want.pool)
        pair = got[s, DV + 10:DV + 12].abs()
        assert bool(((pair == 448) | pair.isnan()).all())
        got[s, DV + 10:DV + 12] = pool[s, DV + 10:DV + 12]
        assert torch.equal(got.nan_to_num(1e9), pool.nan_to_num(1e9))
    c = Case([(0, 0, 2), (1, 3, 1)], 8, seed=2)
    c.kv[:, :DV] = math.inf
    c.kv[:, DV:] = 0
    old = c.scales.clone()
    c.call(B)
    assert float(c.scales[0]) == 2.0 ** -100 and float(c.scales[1]) == float(old[1])
    assert bool((values(c.pool[c.slots.long()])[:, :DV] == 448).all())


def test_numbers_that_need_the_largest_scale(B):
    """The largest finite numbers count as they did, beside infinities or not."""
    for value in (3.3895e38, -3.3895e38):
        c = Case([(0, 0, 3)], 4, seed=3)
        c.kv[1, 9] = value
        c.kv[2, 11] = math.inf
        c.call(B)
        assert float(c.scales[0]) == 2.0 ** 120
        assert float(values(c.pool[int(c.slots[2])])[11]) == 448.0


def test_a_rejected_row_takes_nothing_with_it(B):
    """A draft with an infinity is rejected and written over: the rows in front of it are still what they were."""
    c = Case([(1, 0, 5)], 8, seed=4)
    c.call(B)
    kept, scale = c.pool[8:13].clone(), float(c.scales[1])
    bad = Case([(1, 5, 2)], 8, seed=5, gain=0.01)
    bad.pool, bad.scales = c.pool, c.scales
    bad.kv[0, 100] = math.inf
    bad.call(B)
    assert torch.equal(c.pool[8:13], kept) and float(c.scales[1]) == scale
    good = Case([(1, 5, 2)], 8, seed=6, gain=0.01)
    good.pool, good.scales = c.pool, c.scales
    good.call(B)
    assert torch.equal(c.pool[8:13], kept) and float(c.scales[1]) == scale
    want = (good.kv[:, :DV].float() / scale).to(torch.float8_e4m3fn).float()
    assert torch.equal(values(c.pool[13:15])[:, :DV], want)
