"""Draws and cuts right next to a running sum, where the kernel's single-precision sums must not decide.

Borders are aimed at with the random number (or top-p) nearest to them, some 10^-8 of the mass away.  What the kernel's
own definition leaves open: a weight (of at most 1) is a whole number of units of 2^-45, so it is off by at most half a
unit, 2^-46, and by 2^-37 of itself; u W - C (C the running sum up to token j) takes errors of tokens past j times u and
of the others times 1 - u.  So it is off by at most V 2^-46 + 2 u (1 - u) 2^-37 W, the `open_` of the code below: about
1.9e-9 for 131,072 tokens, where the single-precision sums that must not decide are off by 10^-8 to 10^-7.  The token has
to be one that the definition draws for some value of u W within that; for most rows there is one."""
import numpy as np
import pytest

from tests.test_gpu_sample import draw, host, reference

pytestmark = pytest.mark.gpu


def open_(V, u, W):
    return V * 2.0 ** -46 + 2 * u * (1 - u) * 2.0 ** -37 * W


def ends(x, u, top_k=None):
    """First and last token that rows of temperature 1 may draw."""
    lo, hi = np.empty(len(x), np.int32), np.empty(len(x), np.int32)
    for r in range(len(x)):
        w = np.exp(x[r].astype(np.float64) - x[r].max())
        w[w < 2.0 ** -46] = 0.0
        if top_k is not None:
            w[np.argsort(-x[r], kind="stable")[top_k[r]:]] = 0.0
        c = np.cumsum(w)
        last = int(np.searchsorted(c, c[-1], side="left"))
        goal, off = float(u[r]) * c[-1], open_(x.shape[1], float(u[r]), c[-1])
        lo[r], hi[r] = (min(int(np.searchsorted(c, g, side="right")), last) for g in (goal - off, goal + off))
        if u[r] == 1:
            lo[r] = last
    return lo, hi


def check(got, x, u, top_k=None):
    lo, hi = ends(x, u, top_k)
    bad = (got < lo) | (got > hi)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:5].ravel(), got[bad][:5], lo[bad][:5])
    assert (lo == hi).mean() > 0.85


def dominant_rows(rng, R, V, fp32, spread, same_granule):
    """Rows of one token with about 0.97 of the mass and a tail, and for each row a random number next to the running sum
    of a token soon after the large one (in its 16-byte granule, or within the next 3,000)."""
    x = (np.log(0.03 / V) + rng.normal(0, spread, (R, V))).astype(np.float32)
    vec = 4 if fp32 else 8
    at = rng.integers(0, V // 2 // vec, R) * vec
    x[np.arange(R), at] = 0.0
    x = host(x, fp32)
    u = np.empty(R, np.float32)
    for r in range(R):
        w = np.exp(x[r].astype(np.float64))
        c = np.cumsum(w)
        j = at[r] + (rng.integers(0, vec - 1) if same_granule else rng.integers(1, 3000))
        u[r] = np.float32(c[j] / c[-1])
        if rng.random() < 0.3:
            u[r] = np.nextafter(u[r], np.float32(rng.integers(0, 2)))
    return x, u


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("same_granule", [False, True])
@pytest.mark.parametrize("filters", ["none", "min_p", "top_k"])
def test_draws_next_to_borders_behind_a_large_token(filters, same_granule, fp32):
    rng = np.random.default_rng(17)
    R, V = 256, 131072
    x, u = dominant_rows(rng, R, V, fp32, 0.3, same_granule)
    full = lambda v, t=np.float32: np.full(R, v, t)  # noqa: E731
    # (min-p keeps every token; top-k all but some of the smallest, and some of those equal to its last one)
    k = {"none": {}, "min_p": dict(min_p=full(1e-12)), "top_k": dict(top_k=full(V - 100, np.int32))}[filters]
    check(draw(x, u, fp32, **k), x, u, k.get("top_k"))


@pytest.mark.parametrize("fp32", [False, True])
def test_the_largest_random_numbers_behind_a_large_token(fp32):
    """1 draws the last token of weight, and the numbers just below it the tokens ahead of that."""
    rng = np.random.default_rng(18)
    R, V = 256, 131072
    x, _ = dominant_rows(rng, R, V, fp32, 0.3, False)
    u = (1.0 - np.arange(R) * 2.0 ** -24).astype(np.float32)
    x[::2, V // 2 + 7:] = -np.inf
    assert ends(x, u)[0][0] == V // 2 + 6
    check(draw(x, u, fp32), x, u)
    check(draw(x, u, fp32, min_p=np.full(R, 1e-12, np.float32)), x, u)


@pytest.mark.parametrize("fp32", [False, True])
def test_draws_next_to_borders_of_broad_rows(fp32):
    rng = np.random.default_rng(19)
    R, V = 512, 131072
    x = host(rng.normal(0, 2, (R, V)).astype(np.float32), fp32)
    u = np.empty(R, np.float32)
    for r in range(R):
        c = np.cumsum(np.exp(x[r].astype(np.float64)))
        u[r] = np.float32(c[rng.integers(0, V)] / c[-1])
    check(draw(x, u, fp32), x, u)


@pytest.mark.parametrize("filters", ["none", "min_p"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_at_the_ends_of_the_single_precision_range(sign, filters):
    """Rows whose largest exponent max x log2(e) / T lies within some hundred of +-2^20: tokens of weight on both sides of
    the number from which on exponents are not taken in single precision."""
    rng = np.random.default_rng(21)
    R, V = 96, 9001
    temp = np.resize(np.array([2.0 ** -20, 1e-3, 1.0, 300.0], np.float32), R)
    t = temp.astype(np.float64)[:, None]
    base = (sign * 2.0 ** 20 + np.linspace(-130, 130, R)[:, None]) * np.log(2.0) * t
    x = (base + t * rng.normal(0, 1.5, (R, V))).astype(np.float32)
    # one token just above 2^20 less, all others just beyond it (their weights are 0.94)
    for r in range(0, 8):
        x[r] = -np.float32(np.log(2.0))
        x[r, 7 + 900 * r] = np.nextafter(x[r, 0], np.float32(0))
        temp[r] = 2.0 ** -20
    u = rng.random(R).astype(np.float32)
    k = dict(temp=temp)
    if filters != "none":
        k["min_p"] = np.full(R, 1e-12, np.float32)
    assert np.array_equal(draw(x, u, True, **k), reference(x, u, **k))


@pytest.mark.parametrize("with_k", [False, True])
def test_top_p_cuts_where_large_tokens_share_granules_with_small_ones(with_k):
    """64 tokens of weight 1, each beside one of 5.9e-8 (lost when the two are added in single precision), and a tail
    whose values fall with the index: with u = 1 the token drawn is the last of top-p's prefix."""
    rng = np.random.default_rng(23)
    R, V, big = 64, 100000, 64
    x = np.full((R, V), -np.inf, np.float32)
    x[:, 0:4 * big:4] = 0.0
    x[:, 2:4 * big:4] = np.float32(np.log(5.9e-8))
    n = V - 4 * big
    x[:, 4 * big:] = np.linspace(-13.6, -14.0, n)
    p = rng.uniform(0.9987, 0.9999, R).astype(np.float32)
    ones = np.ones(R, np.float32)
    k = dict(top_p=p)
    if with_k:
        k["top_k"] = rng.integers(V - 3000, V - 2000, R).astype(np.int32)
    got = draw(x, ones, True, **k)
    for r in range(R):
        order = np.argsort(-x[r], kind="stable")[:k["top_k"][r] if with_k else V]
        c = np.cumsum(np.exp(x[r][order].astype(np.float64)))
        goal, off = float(p[r]) * c[-1], open_(V, float(p[r]), c[-1])
        lo, hi = (order[np.searchsorted(c, g, side="left")] for g in (goal - off, goal + off))
        assert lo <= got[r] <= hi <= lo + 1, (r, got[r], lo, hi)
