"""Weights far below a row's largest, and references raised behind a unit's first tile.

A unit is what one CTA has of a stream (32 rows of one sequence over its tiles), and its weights are held against a
reference of its own.  So that units are whole streams of many tiles here, a call has as many sequences as there are SMs, all
alike, of 128 heads: four streams per SM, of equal cost, so that every share of the work is four whole streams.  Equal units
give equal bits, which the tests require."""
import math

import pytest
import torch

from tests.test_gpu_scaled import D, DV, SM, check, ints, pool_of

pytestmark = pytest.mark.gpu
H, TILE, ROWS = 128, 128, 32


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def whole_streams(B, q, pool, scales, kv, sm):
    """One sequence (q [H, 576], its slots kv) as whole streams: out [H, 512] and lse [H]."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, tiles = kv.numel(), -(-kv.numel() // TILE)
    cost = sms * (H // ROWS) * (tiles + 8)
    assert sms <= 512 and -(-cost // sms) == H // ROWS * (tiles + 8)
    out = torch.full((sms, H, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((sms, H), 7.0, device="cuda")
    ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(sms, H, sms, sms * n), dtype=torch.uint8, device="cuda")
    B.verify_attn_mla_scaled(q[None].repeat(sms, 1, 1), pool, scales, ints([k * n for k in range(sms + 1)]), kv.repeat(sms),
                             ints(list(range(sms + 1))), out, lse, ws, sm)
    assert B.verify_attn_mla_check(ws) == 0
    assert torch.equal(out, out[:1].expand_as(out)) and torch.equal(lse, lse[:1].expand_as(lse))
    return out[0], lse[0]


def code(v):
    return int(torch.tensor(v).to(torch.float8_e4m3fn).view(torch.uint8))


def test_each_weight_in_one_tile(B):
    """Key j of 128 has weight 2^-drop and a column of its own, so that its weight can be read off: 9 bits down to 2^-19 of the
    largest, within 2^-28 of the largest below that, and nothing is cut to one side."""
    n = TILE
    drop = torch.linspace(0.0, 36.0, n, dtype=torch.float64)
    pool = torch.zeros((n, D), dtype=torch.uint8, device="cuda")
    pool[:, DV] = code(-1.0)                                  # scores fall with the keys' scales
    pool[torch.arange(n), torch.arange(n)] = code(16.0)
    scales = (1.0 + drop / 64.0).float().cuda()
    q = torch.zeros((H, D), dtype=torch.bfloat16, device="cuda")
    q[:, DV] = 64.0
    out, _ = whole_streams(B, q, pool, scales, torch.arange(n, dtype=torch.int32, device="cuda"), math.log(2.0))
    score = -64.0 * scales.double() * math.log(2.0)
    want = (score - torch.logsumexp(score, 0)).exp() * scales.double() * 16.0
    got = out[0, :n].double()
    # one rounding to bf16 (8 bits: half a step is at most 2^-8 of the value), the weight's 9 bits (2^-9), and the score (single
    # precision about 100 ln 2, times its rounding)
    rel = 2.0 ** -8 + 2.0 ** -9 + 100 * math.log(2.0) * 2.0 ** -23 * 4
    floor = float(want[0]) * 2.0 ** -28
    off = (got - want).abs()
    assert bool((off <= want * rel + floor).all()), float(((off - want * rel) / floor).max())
    # the weights between 2^-19 and 2^-27 together: errors of either sign
    some = (drop.cuda() > 19) & (drop.cuda() < 27)
    assert abs(float(got[some].sum() / want[some].sum()) - 1) < rel


@pytest.mark.parametrize("place", ["first", "middle", "last"])
@pytest.mark.parametrize("drop", [17.7, 22.3, 24.5, 25.2, 26.4, 28.3])
def test_many_small_weights_beside_a_large_one(B, drop, place):
    """12,799 keys of weight 2^-drop beside one of weight 1 whose values are zero where theirs are not: their sum is what
    those columns show."""
    n = 100 * TILE
    at = {"first": 0, "middle": n // 2 + 5, "last": n - 1}[place]
    pool = torch.zeros((n, D), dtype=torch.uint8, device="cuda")
    pool[:, :256] = code(1.0)
    pool[:, DV] = code(-448.0)
    pool[at] = 0
    pool[at, 256:DV] = code(1.0)
    q = torch.zeros((H, D), dtype=torch.bfloat16, device="cuda")
    q[:, DV] = 1.0
    out, lse = whole_streams(B, q, pool, torch.ones(n, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"), drop * math.log(2.0) / 448.0)
    w = 2.0 ** -drop
    total = 1 + (n - 1) * w
    small, large = (n - 1) * w / total, 1 / total
    # a weight, held times 2^9, is off by half of 2^-22 and by half a step of 9 bits, or of 3 where it is below 2^-16; its score's
    # rounding (drop ln 2); bf16
    held = w * 2.0 ** 9
    rel = 2.0 ** -23 / held + (2.0 ** -4 if held < 2.0 ** -15 else 2.0 ** -9) + drop * 2.0 ** -21 + 2.0 ** -8
    assert bool(((out[:, :256].double() - small).abs() <= small * rel).all()), (float(out[0, 0]) / small, rel)
    assert bool(((out[:, 256:].double() - large).abs() <= large * (2.0 ** -9 + 2.0 ** -8)).all())
    # sums of at most n / 128 numbers by a thread
    assert bool(((lse.double() - math.log(total)).abs() <= 2.0 ** -20 + n / 128 * 2.0 ** -24).all())


@pytest.mark.parametrize("spread", [0.0, 1.5])
def test_references_raised_in_many_tiles(B, spread):
    """Keys in rising order of their scores for half of the heads, falling for the others: what has been summed is scaled down
    again and again."""
    n = 47 * TILE - 31
    g = torch.Generator(device="cuda").manual_seed(int(spread * 10))
    pool, scales = pool_of(g, n, 1, True, spread)
    rows = pool.view(torch.float8_e4m3fn).double() * scales.double()[:, None]
    base = torch.randn((1, D), generator=g, device="cuda")
    gain = torch.linspace(-9.0, 9.0, H, device="cuda")[:, None]
    q = (base * gain + 0.05 * torch.randn((H, D), generator=g, device="cuda")).to(torch.bfloat16)
    kv = (rows @ base[0].double()).argsort().to(torch.int32)
    z = (q.double() @ rows[kv.long()].t()) * SM / math.log(2.0) + scales.double()[kv.long()].log2()
    tops = torch.stack([t.amax(1) for t in z.split(TILE, 1)], 1)  # each row's largest weight per tile, as a power of two
    reach = tops.cummax(1).values
    rises = torch.zeros(H, dtype=torch.int64, device="cuda")
    ref = reach[:, 0].clone()
    for t in range(1, reach.shape[1]):  # (2^6 above the reference: raised)
        up = reach[:, t] > ref + 6.01
        rises += up
        ref = torch.where(up, reach[:, t], ref)
    assert int((rises >= 3).sum()) >= H // 4 and int((rises == 0).sum()) >= H // 4
    out, lse = whole_streams(B, q, pool, scales, kv, SM)
    c = dict(q=q[None], pool=pool, scales=scales, kv=kv, block=1, nk=[n], nq=[1])
    check(c, out[None], lse[None])
