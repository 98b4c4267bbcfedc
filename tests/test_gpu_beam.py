"""Beam selection and the reordering of the beams' states, against their definitions in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def select(B, x, score, beams, keep, finished=None, pad=0, ws=None):
    rows, V = x.shape
    R = rows // beams
    out = [torch.full((R, keep), 77, dtype=torch.int32, device="cuda"), torch.full((R, keep), 77, dtype=torch.int32, device="cuda"),
           torch.full((R, keep), 77.0, device="cuda")]
    if ws is None:
        ws = torch.full((B.verify_attn_mla_beam_select_workspace_size(rows, V, keep),), 0xA5, dtype=torch.uint8, device="cuda")
    B.verify_attn_mla_beam_select(x, score, *out, ws, beams=beams, finished=finished, pad_token=pad)
    return out


def expected(x, score, beams, keep, finished=None, pad=0):
    """parent, token, new_score by sorting every candidate (ties: the lowest index)."""
    x = x.double().cpu().numpy()
    score = score.double().cpu().numpy()
    rows, V = x.shape
    R = rows // beams
    parent, token = np.full((R, keep), -1), np.full((R, keep), -1)
    value = np.full((R, keep), -math.inf)
    for r in range(R):
        found = []
        for w in range(beams):
            a = r * beams + w
            c, y = score[a], np.where(np.isnan(x[a]), -math.inf, x[a])
            if not c > -math.inf:
                continue
            if finished is not None and int(finished[a]):
                found.append((-c, w * V + pad))
                continue
            if (y == math.inf).any():
                n = int((y == math.inf).sum())
                found += [(-(c - math.log(n)), w * V + int(v)) for v in np.flatnonzero(y == math.inf)[:keep]]
                continue
            if not (y > -math.inf).any():
                continue
            m = y.max()
            log_sum = math.log(np.exp(y - m).sum())  # (added to a difference: beside logits of 1e30 it would be lost)
            at = np.lexsort((np.arange(V), -y))[:keep]
            found += [(-(c + ((y[v] - m) - log_sum)), w * V + int(v)) for v in at if y[v] > -math.inf]
        for k, (v, i) in enumerate(sorted(found)[:keep]):
            parent[r, k], token[r, k], value[r, k] = i // V, i % V, -v
    return parent, token, value


def check(got, want):
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    v, w = got[2].double().cpu().numpy(), want[2]
    none = np.isinf(w)
    assert np.array_equal(v[none], w[none])
    # the sum in single precision (see the kernel's margin), and one rounding to fp32
    tol = 2e-6 + 1.5e-8 * (100 + 30) + np.abs(w[~none]) * 2.0 ** -24
    assert (np.abs(v[~none] - w[~none]) <= tol).all()


def logits(rows, V, fp32, seed, sigma=2.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, V), generator=g, device="cuda") * sigma
    return (x if fp32 else x.to(torch.bfloat16)), -10.0 - 5.0 * torch.rand((rows,), generator=g, device="cuda")


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R,W,K,V", [(1, 1, 1, 1), (2, 3, 5, 2), (3, 4, 4, 31), (1, 16, 32, 1000), (5, 8, 8, 8192), (2, 5, 10, 32000),
                                     (9, 3, 7, 50257), (1, 2, 32, 262144), (40, 4, 4, 4096)])
def test_against_sorting(B, R, W, K, V, fp32):
    x, c = logits(R * W, V, fp32, R * 31 + V)
    check(select(B, x, c, W, K), expected(x, c, W, K))


@pytest.mark.parametrize("offset", [1, 3, 5, 7])
def test_strided_rows_of_any_alignment(B, offset):
    for fp32 in (False, True):
        whole, c = logits(12, 5011, fp32, offset)
        x = whole[:, offset:offset + 4999]
        check(select(B, x, c, 4, 8), expected(x, c, 4, 8))


def test_ties_go_to_the_lowest_index(B):
    """Few distinct values, equal rows, equal beams: everything is decided by indexes."""
    for V in (40, 9001):
        x = torch.zeros((8, V), dtype=torch.bfloat16, device="cuda")
        c = torch.full((8,), -3.0, device="cuda")
        check(select(B, x, c, 4, 12), expected(x, c, 4, 12))
        x = torch.randint(0, 3, (8, V), device="cuda").to(torch.bfloat16)
        x[1] = x[0]
        x[5] = x[4]
        check(select(B, x, c, 4, 12), expected(x, c, 4, 12))
        x[:, 1::2] = -0.0  # equal to 0
        check(select(B, x, c, 4, 12), expected(x, c, 4, 12))


def test_equal_beams_at_other_alignments(B):
    """The same logits in rows that start at other addresses have exactly equal scores."""
    g = torch.Generator(device="cuda").manual_seed(3)
    row = torch.randn((10007,), generator=g, device="cuda").to(torch.bfloat16)
    x = row.repeat(12, 1)
    c = torch.full((12,), -7.25, device="cuda")
    check(select(B, x, c, 6, 20), expected(x, c, 6, 20))


def test_beams_closer_than_single_precision_tells(B):
    """Two beams whose scores differ by some 1e-7 to 1e-6: told apart by exact sums."""
    g = torch.Generator(device="cuda").manual_seed(4)
    for k in range(12):
        x = (torch.randn((2, 20011), generator=g, device="cuda") * 2).float()
        x[1] = x[0].flip(0)                       # the same sum, in another order
        x[1, 5 * k] += 2.0 ** -(6 + k)            # moves it a little
        c = torch.full((2,), -1.0, device="cuda")
        check(select(B, x, c, 2, 8), expected(x, c, 2, 8))


def test_many_large_tokens_in_few_places(B):
    """More tokens above the bound than are ranked at once: the 64 granules of 40 threads hold rising values."""
    V = 131072
    x = torch.full((2, V), -5.0, dtype=torch.bfloat16, device="cuda")
    thread = torch.arange(V, device="cuda") // 8 % 256
    noise = torch.rand((V,), device="cuda")
    x[0] = torch.where(thread < 40, 100.0 + thread + noise, -5.0).to(torch.bfloat16)
    x[1] = torch.where(thread < 40, 140.0 - thread, -5.0).to(torch.bfloat16)
    c = torch.tensor([-1.0, -1.5], device="cuda")
    check(select(B, x, c, 2, 32), expected(x, c, 2, 32))


def test_forbidden_and_broken_logits(B):
    x, c = logits(12, 3001, True, 5)
    x[0] = -math.inf
    x[1, 2:] = -math.inf
    x[2, ::3] = math.nan
    x[3] = math.nan
    x[4, 17] = x[4, 9] = math.inf
    x[5] = math.inf
    x[6] = -1e30
    x[7] = 3e38
    c[8] = -math.inf
    c[9] = math.nan
    got, want = select(B, x, c, 4, 16), expected(x, c, 4, 16)
    check(got, want)
    x = torch.full((4, 100), -math.inf, device="cuda")
    got = select(B, x, c[:4], 2, 3)
    assert bool((got[0] == -1).all()) and bool((got[1] == -1).all()) and bool((got[2] == -math.inf).all())
    x = x.to(torch.bfloat16)
    x[2, 99] = 1.0
    check(select(B, x, c[:4], 2, 3), expected(x, c[:4], 2, 3))


def test_finished_beams(B):
    x, c = logits(32, 5000, False, 6)
    done = torch.tensor([0, 1, 0, 0] * 7 + [1, 1, 1, 1], dtype=torch.int32, device="cuda")
    c[1] = -0.5          # ahead of all others
    c[5] = -500.0        # behind all others
    got, want = select(B, x, c, 4, 8, finished=done, pad=2), expected(x, c, 4, 8, finished=done, pad=2)
    check(got, want)
    assert int(got[0][0, 0]) == 1 and int(got[1][0, 0]) == 2 and float(got[2][0, 0]) == -0.5
    assert int((got[0][-1] >= 0).sum()) == 4  # four finished beams offer four continuations


def test_captured_and_replayed(B):
    x, c = logits(16, 32000, False, 7)
    ws = torch.empty(B.verify_attn_mla_beam_select_workspace_size(16, 32000, 8), dtype=torch.uint8, device="cuda")
    out = [torch.zeros((2, 8), dtype=torch.int32, device="cuda"), torch.zeros((2, 8), dtype=torch.int32, device="cuda"),
           torch.zeros((2, 8), device="cuda")]
    call = lambda: B.verify_attn_mla_beam_select(x, c, *out, ws, beams=8)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed in (8, 9):
        y, d = logits(16, 32000, False, seed)
        x.copy_(y)
        c.copy_(d)
        g.replay()
        torch.cuda.synchronize()
        check(out, expected(x, c, 8, 8))


@pytest.mark.parametrize("words,stride", [(1, 1), (7, 7), (64, 64), (1001, 1003), (4096, 4100)])
def test_reorder(B, words, stride):
    r = np.random.default_rng(words)
    R, W, K = 5, 3, 6
    base = torch.from_numpy(r.integers(-2 ** 31, 2 ** 31, (R * W, stride)).astype(np.int32)).cuda()
    src = base[:, :words]
    length = torch.from_numpy(r.integers(0, words + 1, R * W).astype(np.int32)).cuda()
    parent = torch.from_numpy(r.integers(-1, W, (R, K)).astype(np.int32)).cuda()
    parent[0] = torch.tensor([0, 0, 1, 1, 2, 2])
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    for with_length in (False, True):
        dst = torch.full((R * K, stride), -9, dtype=torch.int32, device="cuda")
        new_length = torch.full((R * K,), 5, dtype=torch.int32, device="cuda")
        B.verify_attn_mla_beam_reorder(src, dst[:, :words], parent, beams=W, length=length if with_length else None,
                                       new_length=new_length if with_length else None, status_word=status)
        want = np.full((R * K, stride), -9, np.int32)
        s, ln, p = base.cpu().numpy(), length.cpu().numpy(), parent.cpu().numpy()
        for q in range(R * K):
            w = p[q // K, q % K]
            n = (ln[q // K * W + w] if with_length else words) if w >= 0 else 0
            if n:
                want[q, :n] = s[q // K * W + w, :n]
            if with_length:
                assert int(new_length[q]) == n
        assert np.array_equal(dst.cpu().numpy(), want)
        assert status.tolist() == [0, 0]


def test_reorder_of_states_in_bf16_and_faults(B):
    src = torch.randn((4, 130), device="cuda").to(torch.bfloat16)
    dst = torch.zeros((6, 130), dtype=torch.bfloat16, device="cuda")
    parent = torch.tensor([[1, 1, 0], [0, 1, 1]], dtype=torch.int32, device="cuda")
    B.verify_attn_mla_beam_reorder(src, dst, parent, beams=2)
    assert torch.equal(dst, src[torch.tensor([1, 1, 0, 2, 3, 3], device="cuda")])
    table = torch.arange(40, dtype=torch.int32, device="cuda").view(4, 10)
    for bad, row in (([[0, 2], [1, 0]], 1), ([[0, 1], [-2, 0]], 2)):
        status = torch.zeros(2, dtype=torch.int32, device="cuda")
        new = torch.full((4, 10), -1, dtype=torch.int32, device="cuda")
        B.verify_attn_mla_beam_reorder(table, new, torch.tensor(bad, dtype=torch.int32, device="cuda"), beams=2, status_word=status)
        assert status.tolist() == [B.VMLA_ERR_INDEX, row]
        assert bool((new[row] == -1).all())
    status = torch.zeros(2, dtype=torch.int32, device="cuda")
    new = torch.full((4, 10), -1, dtype=torch.int32, device="cuda")
    length = torch.tensor([3, 11, 2, 2], dtype=torch.int32, device="cuda")
    B.verify_attn_mla_beam_reorder(table, new, torch.tensor([[0, 1], [1, 0]], dtype=torch.int32, device="cuda"), beams=2, length=length,
                                   status_word=status)
    assert status.tolist() == [B.VMLA_ERR_INDEX, 1]
    assert torch.equal(new[1], table[1])  # cut to the row's words
