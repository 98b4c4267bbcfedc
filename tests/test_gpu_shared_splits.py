"""The shared-prefix call with one and the same input cut into different numbers of pieces."""
import numpy as np
import pytest

from tests.test_gpu_shared import CASES, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["past_a_tile", "many_queries", "trees", "codes"])
def test_split_counts_agree(name):
    """Each result is within the tolerance derived in tests/test_gpu_shared.py of the same exact value, so two of them
    are within twice that of each other; and each split count gives the same bits when called again."""
    c = Case(**CASES[name])
    _, _, mag = c.reference()
    first = None
    for splits in (0, 1, 2, 5, 64, -1):
        assert c.run(splits) == 0
        bits = (c.out.clone(), c.lse.clone())
        assert c.run(splits) == 0
        assert (bits[0] == c.out).all() and (bits[1] == c.lse).all()
        out, lse = c.out.double().cpu().numpy(), c.lse.double().cpu().numpy()
        if first is None:
            first = (out, lse)
            continue
        slack = (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12) * mag
        assert (abs(out - first[0]) <= 2 * (slack + 2.0 ** -8 * (abs(out) + 2 * slack))).all(), splits
        assert np.abs(lse - first[1]).max() < 2e-3
