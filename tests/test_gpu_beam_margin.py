"""Beams whose scores lie next to each other, over rows whose sums single precision puts off the furthest: a token that is
nearly the whole sum and lies far above the first logits its thread met, beside another thread's that is nearly as large."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_beam import expected, select

pytestmark = pytest.mark.gpu
V = 4000

# (x[0], x[1024], x[4]), all others -20: x[0] and x[1024] are a thread's first two granules, x[4] is another thread's.  With
# differences from x[0], and their products with log2 e, each rounded in single precision, the logarithm of the sum comes out
# too high by 2.7e-6 to 3.1e-6 in the first rows, too low by as much in the others (calculated).
HIGH = [(0.28051853, 19.83278656, 16.57664299), (2.78057194, 22.2160797, 19.1559353), (1.9152441, 21.511713, 17.9658546),
        (2.90297604, 22.8549519, 19.1909027), (0.730031013, 20.2854271, 16.8308353)]
LOW = [(0.92206478, 20.22616959, 17.90712547), (2.61458874, 21.6932259, 18.6274166), (2.69394207, 21.9687233, 19.0234356),
       (2.88488483, 22.8218899, 19.6275368), (1.88779545, 21.8486309, 17.9388008)]


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def log_sums(x):
    x = x.astype(np.float64)
    m = x.max(1, keepdims=True)
    return (m + np.log(np.exp(x - m).sum(1, keepdims=True)))[:, 0]


def check_order(B, x, c, beams, keep):
    x, c = torch.from_numpy(x).cuda(), torch.from_numpy(c).cuda()
    got, want = select(B, x, c, beams, keep), expected(x, c, beams, keep)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("keep", [1, 2, 4])
@pytest.mark.parametrize("gap", [1e-6, -1e-6, 2e-6])
def test_a_dominating_token_far_above_the_first_ones(B, gap, keep):
    """The first beam's best is ahead by `gap`, far more than 2^-27."""
    pairs = [(h, l) for h in HIGH for l in LOW] + [(l, h) for h in HIGH for l in LOW]
    x = np.full((2 * len(pairs), V), -20.0, np.float32)
    for k, pair in enumerate(pairs):
        for w, (first, large, other) in enumerate(pair):
            x[2 * k + w, [0, 1024, 4]] = first, large, other
    lse = log_sums(x)
    c = np.full(2 * len(pairs), -0.75, np.float32)
    best = x.max(1).astype(np.float64) - lse
    c[1::2] = (c[::2] + best[::2] - gap - best[1::2]).astype(np.float32)  # (steps of 2^-24: the gap is off by 3e-8)
    ahead = (c + best)[::2] - (c + best)[1::2]
    assert (np.abs(ahead - gap) < 1e-7).all()
    check_order(B, x, c, 2, keep)


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("vocab", [5000, 40003])
def test_many_rows_with_scores_a_millionth_apart(B, fp32, vocab):
    r = np.random.default_rng(vocab + fp32)
    R, W = 200, 4
    x = r.normal(-14.0, 1.0, (R * W, vocab)).astype(np.float32)
    first = r.uniform(0.0, 3.0, R * W).astype(np.float32)
    step = 256 * (4 if fp32 else 8)  # a thread's next granule
    x[:, 0], x[:, 17] = first, first + r.uniform(10.0, 18.0, R * W)
    x[:, step] = first + r.uniform(15.0, 20.0, R * W)
    x[::3, 2 * step] = first[::3] + r.uniform(20.0, 21.0, len(first[::3]))
    if not fp32:
        x = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    best = x.max(1).astype(np.float64) - log_sums(x)
    target = -1.0 - np.cumsum(r.uniform(1e-6, 5e-6, (R, W)), 1)
    target = r.permuted(target, axis=1).reshape(-1)
    c = (target - best).astype(np.float32)
    score = np.sort((c + best).reshape(R, W), 1)
    clear = (np.diff(score, axis=1) > 2.0 ** -22).all(1)  # (c is rounded)
    assert clear.sum() > 190
    rows = np.repeat(clear, W)
    x, c = x[rows], c[rows]
    if fp32:
        check_order(B, x, c, W, W)
        return
    t, c = torch.from_numpy(x).cuda().to(torch.bfloat16), torch.from_numpy(c).cuda()
    got, want = select(B, t, c, W, W), expected(t, c, W, W)
    assert np.array_equal(got[0].cpu().numpy(), want[0]) and np.array_equal(got[1].cpu().numpy(), want[1])


def test_new_scores_are_as_good_as_the_bound(B):
    """Scores of beams that are not near one another: within 4e-6, and half a step of single precision."""
    rows = HIGH + LOW
    x = np.full((len(rows), V), -20.0, np.float32)
    for k, v in enumerate(rows):
        x[k, [0, 1024, 4]] = v
    c = np.linspace(-1.0, -3.0, len(rows)).astype(np.float32)
    got = select(B, torch.from_numpy(x).cuda(), torch.from_numpy(c).cuda(), len(rows), 4)
    want = expected(torch.from_numpy(x), torch.from_numpy(c), len(rows), 4)
    off = np.abs(got[2].cpu().numpy() - want[2])
    assert (off <= 4e-6 + np.abs(want[2]) * 2.0 ** -24).all()
    assert not math.isnan(off.max())
