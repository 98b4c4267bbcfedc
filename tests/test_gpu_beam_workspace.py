"""One workspace of the beams' selection, made for a largest batch, serves every smaller one."""
import pytest
import torch

from tests.test_gpu_beam import check, expected, logits, select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("largest,vocab", [(512, 32000), (1000, 8192), (200, 262144), (3, 100)])
def test_smaller_batches_and_vocabularies(B, largest, vocab):
    n, guard = B.verify_attn_mla_beam_select_workspace_size(largest, vocab, 8), 4096
    whole = torch.full((n + guard,), 0xA5, dtype=torch.uint8, device="cuda")
    for rows in sorted({largest, largest * 55 // 64 // 4 * 4, largest * 3 // 5 // 4 * 4, 300, 8, 4}):
        if rows > largest or rows % 4:
            continue
        for v in {vocab, vocab - 1, vocab // 3} if rows < 450 else {vocab}:
            x, c = logits(rows, v, False, rows)
            got = select(B, x, c, 4, 8, ws=whole[:n])
            few = min(rows, 32)
            check([t[:few // 4] for t in got], expected(x[:few], c[:few], 4, 8))
    assert bool((whole[n:] == 0xA5).all())


def test_sizes_never_fall(B):
    for vocab in (1, 4096, 8192, 32768, 65536, 262144):
        sizes = [B.verify_attn_mla_beam_select_workspace_size(rows, vocab, 1) for rows in range(0, 1200)]
        assert sizes == sorted(sizes)
    for rows in (1, 28, 29, 57, 113, 114, 455, 456, 2000):
        sizes = [B.verify_attn_mla_beam_select_workspace_size(rows, vocab, 1) for vocab in range(1, 262145, 997)]
        assert sizes == sorted(sizes)
