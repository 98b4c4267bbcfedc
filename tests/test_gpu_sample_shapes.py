"""Forms of the sampling kernel that only certain sizes take: one CTA a row that reads the row again, the longest bf16
rows of one CTA, and the same row on every number of CTAs.  Tokens are equal to the 64-bit definition's."""
import numpy as np
import pytest

from tests.test_gpu_sample import draw, host, logits, reference, settings

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp32", [False, True])
def test_one_cta_a_row_read_again(fp32):
    """More rows than find two CTAs each, and more of a row than stays in shared memory."""
    rng = np.random.default_rng(31)
    R, V = (150, 50000) if not fp32 else (310, 30011)
    for on in (("temp", "top_p"), ("temp", "top_k"), ("temp", "min_p"), ("temp", "top_k", "top_p", "min_p")):
        x, s, u = logits(rng, R, V), settings(rng, R, V), rng.random(R).astype(np.float32)
        k = {n: s[n] for n in on}
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), on


@pytest.mark.parametrize("V", [126977, 131072, 135161, 135168])
def test_values_next_to_zero_at_the_end_of_long_rows(V):
    """32 or 33 iterations of one CTA (rows of 135,168 tokens are the longest).  Most of the mass is in values next to
    zero that only the last iterations of a warp meet: every one of them counts for top-p's cut."""
    rng = np.random.default_rng(V)
    R = 310
    iters = -(-V // 4096)
    x = rng.normal(-4, 1, (R, V)).astype(np.float32)
    place = np.arange(V) % (iters * 256) // 256  # iteration of a token (of its warp)
    for r in range(R):
        late = np.flatnonzero(place == 30 + r % (iters - 30)) if r % 3 else np.flatnonzero(place >= 29)
        x[r, late] = rng.uniform(-2.0 ** -11, 2.0 ** -11, len(late))
    u, s = rng.random(R).astype(np.float32), settings(rng, R, V)
    s["top_p"] = rng.uniform(0.05, 0.95, R).astype(np.float32)
    for on in (("top_p",), ("temp", "top_k", "top_p", "min_p")):
        k = {n: s[n] for n in on}
        assert np.array_equal(draw(x, u, False, **k), reference(host(x, False), u, **k)), on


@pytest.mark.parametrize("fp32,V", [(False, 131072), (False, 32000), (True, 64001), (True, 9000)])
def test_a_row_draws_the_same_token_in_every_batch(fp32, V):
    """Batches of 1 to 512 rows give a row eight to one CTAs."""
    rng = np.random.default_rng(V)
    R = 512
    x = rng.normal(0, 2, (R, V)).astype(np.float32)
    u, s = rng.random(R).astype(np.float32), settings(rng, R, V)
    few = 8
    for on in ((), ("temp",), ("temp", "top_p"), ("temp", "top_k", "top_p", "min_p")):
        k = {n: s[n] for n in on}
        want = reference(host(x[:few], fp32), u[:few], **{n: v[:few] for n, v in k.items()})
        for rows in (1, 2, 8, 40, 64, 76, 150, 300, 512):
            got = draw(x[:rows], u[:rows], fp32, **{n: v[:rows] for n, v in k.items()})
            assert np.array_equal(got[:few], want[:rows]), (on, rows)
