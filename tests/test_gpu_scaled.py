"""Attention over an e4m3 pool with a scale per block of slots, against the definition in 64 bits."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D, DV = 576, 512
SM = 1 / math.sqrt(192.0)


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def pool_of(g, blocks, block, powers=True, spread=0.4):
    x = torch.randn((blocks, block * D), generator=g, device="cuda") * (
        0.5 * torch.exp(spread * torch.randn((blocks, 1), generator=g, device="cuda")))
    scale = x.abs().amax(1) / 448.0
    if powers:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    codes = (x / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes.view(blocks * block, D).contiguous(), scale.contiguous()


def case(nk, nq, heads, block=1, powers=True, seed=0, sigma=1.5, spread=0.4, extra=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    blocks = [-(-n // block) for n in nk]
    pool, scales = pool_of(g, sum(blocks) + extra, block, powers, spread)
    perm = torch.randperm(sum(blocks) + extra, generator=g, device="cuda")
    rows, at = [], 0
    for n, b in zip(nk, blocks):
        p = torch.arange(n, device="cuda")
        rows.append(perm[at:at + b][p // block] * block + p % block if n else p)
        at += b
    kv = torch.cat(rows).to(torch.int32)
    ind = lambda c: torch.tensor(np.concatenate([[0], np.cumsum(c)]), dtype=torch.int32, device="cuda")  # noqa: E731
    q = (torch.randn((sum(nq), heads, D), generator=g, device="cuda") * sigma).to(torch.bfloat16)
    return dict(q=q, pool=pool, scales=scales, kv=kv, kv_indptr=ind(nk), qo_indptr=ind(nq), block=block, nk=list(nk), nq=list(nq))


def run(B, c, parent=None, draft_mask=None, sm=SM, pad_q=0, pad_kv=0, ws=None, stream=None):
    T, H, _ = c["q"].shape
    q = torch.cat([c["q"], torch.zeros((pad_q, H, D), dtype=torch.bfloat16, device="cuda")])
    kv = torch.cat([c["kv"], torch.full((pad_kv,), -7, dtype=torch.int32, device="cuda")])
    out = torch.full((T + pad_q, H, DV), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + pad_q, H), 7.0, device="cuda")
    if ws is None:
        n = B.verify_attn_mla_scaled_workspace_size(len(c["nk"]), H, T + pad_q, kv.numel())
        ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
    pad = lambda t: None if t is None else torch.cat([t, torch.full((pad_q,), -99, dtype=t.dtype, device="cuda")])  # noqa: E731
    B.verify_attn_mla_scaled(q, c["pool"], c["scales"], c["kv_indptr"], kv, c["qo_indptr"], out, lse, ws, sm,
                             block_tokens=c["block"], parent=pad(parent), draft_mask=pad(draft_mask), stream=stream)
    return out, lse, ws


def visible(c, parent, draft_mask):
    """[T][Q_b] truth values: which drafts a query sees."""
    rows = []
    t0 = 0
    for n in c["nq"]:
        for i in range(n):
            if draft_mask is not None:
                word = int(draft_mask[t0 + i]) & (2 ** 64 - 1)
                rows.append([bool(word >> k & 1) for k in range(n)])
            elif parent is not None:
                see, k = [False] * n, i
                while k >= 0:
                    see[k] = True
                    k = int(parent[t0 + k])
                rows.append(see)
            else:
                rows.append([k <= i for k in range(n)])
        t0 += n
    return rows


def reference(c, parent=None, draft_mask=None, sm=SM):
    """out, lse in 64 bits, sum_j w_j |v_j|, and a bound of the scores' error (per row)."""
    T, H, _ = c["q"].shape
    lut = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    sees = visible(c, parent, draft_mask)
    outs, lses, mags, errs = [], [], [], []
    t0 = k0 = 0
    S = c["pool"].shape[0]
    for n, m in zip(c["nk"], c["nq"]):
        slot = c["kv"][k0:k0 + n].long()
        ok = (slot >= 0) & (slot < S)
        at = torch.where(ok, slot, 0)
        rows = lut[c["pool"][at].int()] * c["scales"].double()[at // c["block"]][:, None] * ok[:, None]
        if m:
            q = c["q"][t0:t0 + m].double()
            z = torch.einsum("thd,nd->thn", q, rows) * sm
            mag = torch.einsum("thd,nd->thn", q.abs(), rows.abs()) * sm
            vis = torch.ones((m, n), dtype=torch.bool, device="cuda")
            vis[:, n - m:] = torch.tensor(sees[t0:t0 + m], device="cuda")
            z = z.masked_fill(~vis[:, None, :], -math.inf)
            l = torch.logsumexp(z, -1)
            w = torch.where(torch.isfinite(l)[..., None], (z - l[..., None]).exp(), 0.0)
            outs.append(w @ rows[:, :DV])
            lses.append(l)
            mags.append(w @ rows[:, :DV].abs())
            # queries in two parts: 2^-22.8 of the row's largest, for every element of the key; the dot product's own
            # sums in single precision
            split = q.abs().amax(-1) * 2.0 ** -22 * (rows.abs().sum(1).max() * sm)
            errs.append(mag.amax(-1) * (D + 8) * 2.0 ** -24 + split)
        t0 += m
        k0 += n
    cat = lambda x: torch.cat(x) if x else torch.zeros(0, H, device="cuda")  # noqa: E731
    return cat(outs), cat(lses), cat(mags), cat(errs)


def check(c, out, lse, parent=None, draft_mask=None, sm=SM):
    T = c["q"].shape[0]
    o, l, mag, es = reference(c, parent, draft_mask, sm)
    got_o, got_l = out[:T].double(), lse[:T].double()
    none = torch.isinf(l)
    assert bool((got_l[none] == -math.inf).all()) and bool((got_o[none] == 0).all())
    use = ~none
    n = max(c["nk"])
    # exponentials to 2^-22, their arguments' rounding, sums of at most n numbers by 128 threads, log2
    rel = 2.0 ** -22 * 4 + (n / 128 + 400) * 2.0 ** -24
    err_l = (got_l - l).abs()[use]
    tol_l = (es + rel + l.abs() * 2.0 ** -22)[use]
    assert bool((err_l <= tol_l).all()), float((err_l / tol_l).max())
    # weights of 9 bits (half a step: 2^-9), relative errors of the weights and of their sum, one rounding to bf16
    tol_o = o.abs() * 2.0 ** -8 + mag * (2.0 ** -9 + 2 * (es + rel))[..., None] * (1 + 2.0 ** -7) + 1e-30
    err_o = (got_o - o).abs()
    assert bool((err_o <= tol_o)[use].all()), float((err_o / tol_o)[use].max())
    return float(err_l.max()) if err_l.numel() else 0.0


@pytest.mark.parametrize("n", [1, 2, 31, 127, 128, 129, 700, 5000])
@pytest.mark.parametrize("heads,nq", [(64, 1), (8, 1), (1, 1), (24, 3)])
def test_lengths(B, n, heads, nq):
    c = case([n + nq - 1], [nq], heads, seed=n)
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse)


def test_one_key_gives_its_score(B):
    """With one key lse is the score itself: how exactly the tensor cores sum, at several sizes of the queries."""
    for seed, sigma in enumerate([0.01, 1.0, 30.0]):
        c = case([1] * 64, [1] * 64, 32, seed=seed, sigma=sigma)
        out, lse, ws = run(B, c)
        assert B.verify_attn_mla_check(ws) == 0
        print("one key", sigma, check(c, out, lse))


@pytest.mark.parametrize("block,powers", [(1, True), (16, False), (64, True), (128, False)])
def test_ragged_batch(B, block, powers):
    nk = [300, 5, 0, 4097, 1, 129, 64, 2000]
    nq = [1, 5, 0, 3, 0, 2, 64, 7]
    c = case(nk, nq, 16, block=block, powers=powers, seed=block)
    out, lse, ws = run(B, c, pad_q=5, pad_kv=9)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse)
    assert bool((out[c["q"].shape[0]:] == 7.0).all()) and bool((lse[c["q"].shape[0]:] == 7.0).all())


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_trees(B, heads):
    nq = [64, 17, 40]
    nk = [900, 17, 3000]
    r = np.random.default_rng(heads)
    parent = np.concatenate([[int(r.integers(-1, i)) if i else -1 for i in range(n)] for n in nq]).astype(np.int32)
    parent = torch.tensor(parent, device="cuda")
    c = case(nk, nq, heads, block=8, seed=heads)
    out, lse, ws = run(B, c, parent=parent, pad_q=3)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse, parent=parent)


def test_masks_that_leave_nothing(B):
    """Words without a bit, with no prefix: out 0, lse -inf; with a prefix: the prefix alone."""
    nq, nk = [4, 6, 64], [4, 200, 64]
    words = torch.zeros(74, dtype=torch.int64, device="cuda")
    words[1] = 0b10
    words[5] = 0b100001
    words[20] = -1
    c = case(nk, nq, 8, seed=5)
    out, lse, ws = run(B, c, draft_mask=words)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse, draft_mask=words)
    assert bool((lse[0] == -math.inf).all()) and bool((out[0] == 0).all())


def test_many_shapes_of_the_plan(B):
    """Batches whose streams are cut by lanes in many ways, groups of one to eight."""
    r = np.random.default_rng(3)
    for seed in range(8):
        batch = int(r.integers(1, 60))
        nq = r.integers(0, 9, batch)
        nk = nq + np.exp(r.uniform(0, np.log(3000), batch)).astype(int)
        c = case(nk.tolist(), nq.tolist(), int(r.choice([8, 16, 64, 128])), block=int(r.choice([1, 32])), seed=seed)
        out, lse, ws = run(B, c)
        assert B.verify_attn_mla_check(ws) == 0
        check(c, out, lse)


def test_largest_batch(B):
    c = case([3] * 512, [1] * 512, 8, seed=9)
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse)


def test_scores_that_rise_and_fall(B):
    """Keys in rising and falling order of their scores, with scales over eleven powers of two: the references are
    raised in many tiles, and weights far below the largest still count."""
    for seed, order in enumerate([1, -1]):
        c = case([6000], [1], 64, seed=seed, sigma=6.0, spread=1.5)
        s = (c["q"][0, 0].double() @ (c["pool"][c["kv"].long()].view(torch.float8_e4m3fn).double()
                                      * c["scales"].double()[c["kv"].long()][:, None]).t())
        c["kv"] = c["kv"][(order * s).argsort()].contiguous()
        out, lse, ws = run(B, c)
        assert B.verify_attn_mla_check(ws) == 0
        check(c, out, lse)


def test_a_key_of_much_weight_beside_many_of_little(B):
    """One key far above 40,000 equal ones whose weights sum to as much."""
    n = 40001
    c = case([n], [1], 8, seed=4, sigma=1.0, spread=0.0)
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    sc = float(c["scales"][0])
    c["scales"].fill_(sc)
    c["pool"][:, 0] = torch.zeros(1, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    one = torch.tensor([448.0], device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    c["pool"][c["kv"][77].long(), 0] = one
    sm = math.log(40000.0) / (448.0 * sc)
    out, lse, ws = run(B, c, sm=sm)
    check(c, out, lse, sm=sm)


def test_weights_at_their_floor(B):
    """A column in which the key of most weight has a zero shows what becomes of the small ones: 9 bits down to 2^-17 of the
    largest, steps of 2^-25 below that."""
    n, H = 512, 16
    drop = torch.linspace(0.0, 30.0, n, dtype=torch.float64)  # key j's weight is 2^-drop[j]
    pool = torch.zeros((n, D), dtype=torch.float8_e4m3fn, device="cuda")
    pool[:, DV] = -1.0                                        # scores fall with the keys' scales
    pool[torch.arange(n), torch.arange(n)] = 16.0             # column j: key j alone
    scales = (1.0 + drop / 64.0).float().cuda()
    q = torch.zeros((1, H, D), dtype=torch.bfloat16, device="cuda")
    q[:, :, DV] = 64.0
    c = dict(q=q, pool=pool.view(torch.uint8), scales=scales, kv=torch.arange(n, dtype=torch.int32, device="cuda"), block=1, nk=[n], nq=[1],
             kv_indptr=ints([0, n]), qo_indptr=ints([0, 1]))
    sm = math.log(2.0)                                        # in powers of two: 2^-(64 scale) = 2^-64 2^-drop
    out, lse, _ = run(B, c, sm=sm)
    score = -64.0 * scales.double() * sm
    p = (score - torch.logsumexp(score, 0)).exp()
    want = p * 16.0 * scales.double()
    err = (out[0, 0].double() - want).abs()
    floor = float(p.max()) * 2.0 ** -26 * 16.0 * 1.5          # half a step of the weight times scale (at most 1.5 of the first key's)
    rel = 2.0 ** -8 + 2.0 ** -9 + 1e-4                        # bf16, the weight's bits, the scores (fp32 about 64 ln 2)
    assert bool((err <= want * rel + floor).all()), float(((err - want * rel) / floor).max())


def test_zero_scales_and_zero_rows(B):
    c = case([500], [2], 16, block=4, seed=6)
    c["scales"][c["kv"][:200].long() // 4] = 0.0
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse)
    c["scales"].zero_()
    out, lse, ws = run(B, c)
    check(c, out, lse)
    assert bool((out == 0).all())


def test_slots_outside_the_pool_read_zeros(B):
    c = case([700, 300], [1, 2], 16, seed=7)
    S = c["pool"].shape[0]
    c["kv"][[5, 300, 800]] = torch.tensor([-1, S, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == B.VMLA_ERR_INDEX
    assert int(ws[:8].view(torch.int32)[1]) in (5, 300, 800)
    check(c, out, lse)


def test_rows_of_very_different_sizes(B):
    """A row's precision does not depend on the rows beside it, and an infinite or broken one spoils no other."""
    c = case([700, 300], [3, 2], 16, seed=21)
    c["q"][1, 4] *= 2.0 ** 24
    c["q"][2, 5] *= 2.0 ** -60
    c["q"][3, 0] *= 2.0 ** 16
    out, lse, _ = run(B, c)
    check(c, out, lse)
    c["q"][0, 7, 100] = math.inf
    c["q"][4, 9, 570] = math.nan
    broken = torch.zeros((5, 16), dtype=torch.bool, device="cuda")
    broken[0, 7] = broken[4, 9] = True
    got, got_l, _ = run(B, c)
    assert bool(got[broken].isnan().all()) and bool(got_l[broken].isnan().all())
    want, want_l, _ = run(B, {**c, "q": torch.where(broken[:, :, None], 0, c["q"])})
    # (the others as without them, but for when their references rise)
    assert torch.allclose(got[~broken].float(), want[~broken].float(), rtol=2.0 ** -6, atol=1e-2)
    assert torch.allclose(got_l[~broken], want_l[~broken], rtol=2.0 ** -18, atol=1e-5)


@pytest.mark.parametrize("power", [-90, -40, 40, 100, 110])
def test_scales_far_from_one(B, power):
    """Scales anywhere in their range, queries that bring the scores back to where softmax has work."""
    c = case([600, 77], [2, 1], 24, block=16, seed=power + 200)
    c["scales"] *= 2.0 ** power
    c["q"] = (c["q"].float() * 2.0 ** -power).to(torch.bfloat16)
    out, lse, _ = run(B, c)
    assert bool(torch.isfinite(lse).all())
    check(c, out, lse)


@pytest.mark.parametrize("power,queries", [(40, 2.0 ** -12), (40, 1.0), (20, 2.0 ** 9), (0, 2.0 ** 30), (0, 2.0 ** 60)])
def test_scores_beyond_their_precision(B, power, queries):
    """Scores whose last place is whole powers of e: each row gets its largest key's values, or, where two are as large
    within that place, something between keys."""
    c = case([900, 300], [1, 3], 16, block=4, seed=3)
    c["scales"] *= 2.0 ** power
    c["q"] = (c["q"].float() * queries).to(torch.bfloat16)
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == 0
    o, l, mag, es = reference(c)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert bool(((lse - l).abs() <= es + l.abs() * 2.0 ** -21 + 1).all())
    t0 = k0 = clear = 0
    for n, m in zip(c["nk"], c["nq"]):
        slot = c["kv"][k0:k0 + n].long()
        rows = c["pool"][slot].view(torch.float8_e4m3fn).double() * c["scales"].double()[slot // c["block"]][:, None]
        z = torch.einsum("thd,nd->thn", c["q"][t0:t0 + m].double(), rows) * SM
        z[:, :, n - m:].masked_fill_(torch.ones((m, m), device="cuda").triu(1).bool()[:, None, :], -math.inf)
        two = z.topk(2, -1).values
        sure = two[..., 0] - two[..., 1] > 2 * es[t0:t0 + m] + two[..., 0].abs() * 2.0 ** -21 + 64
        got, want = out[t0:t0 + m].double(), rows[z.argmax(-1)][..., :DV]
        assert bool(((got - want).abs() <= want.abs() * 2.0 ** -6)[sure].all())
        clear += int(sure.sum())
        t0, k0 = t0 + m, k0 + n
    assert clear > 30


def test_two_streams_at_once(B):
    """Calls that run side by side, each with its own workspace."""
    a, b = case([9000, 4000], [4, 2], 16, seed=5), case([700] * 40, [3] * 40, 16, block=16, seed=6)
    want_a, want_b = run(B, a), run(B, b)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for s, c in ((one, a), (two, b)):
            with torch.cuda.stream(s):
                got.append((c is a, run(B, c)))
    torch.cuda.synchronize()
    for is_a, (o, l, _) in got:
        w = want_a if is_a else want_b
        assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_pool_past_32_bits(B):
    """Slots whose bytes lie beyond 2^32 and 2^33: written by the append, read by the attention."""
    S, n = 16_000_000, 300
    pool = torch.zeros((S, D), dtype=torch.uint8, device="cuda")
    c = case([n], [2], 16, block=8, seed=9)
    slots = torch.cat([torch.arange(40), 7_456_540 + torch.arange(100), 14_913_080 + torch.arange(100), S - 60 + torch.arange(60)]).to(torch.int32).cuda()
    scales = torch.zeros(S // 8, device="cuda")
    kv = torch.randn((n, D), device="cuda").to(torch.bfloat16)
    one = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).cuda()
    B.verify_attn_mla_append_scaled(kv[:, :DV], kv[:, DV:], torch.zeros(n, dtype=torch.int32, device="cuda"), slots, one, pool, scales, block_tokens=8)
    rows = pool[slots.long()].view(torch.float8_e4m3fn).double() * scales.double()[slots.long() // 8][:, None]
    assert bool(((rows - kv.double()).abs() <= kv.double().abs() * 2.0 ** -4 * 2.1 + scales.double()[slots.long() // 8][:, None] * 2.0 ** -9).all())
    assert int((pool.view(-1, 8 * D)[::9973] != 0).any(1).sum()) < 50 and int((scales != 0).sum()) <= 45
    c.update(pool=pool, scales=scales, kv=slots)
    out, lse, _ = run(B, c)
    check(c, out, lse)


@pytest.mark.parametrize("nk,heads", [(1, 16), (130, 16), (700, 1), (5000, 40)])
def test_nan_in_masked_places(B, nk, heads):
    """A draft whose codes are NaN makes NaN of the rows that see it and of no other."""
    nq = min(nk, 9)
    c = case([nk, 40], [nq, 1], heads, seed=nk)
    bad = nq // 2
    slot = int(c["kv"][nk - nq + bad])
    keep = c["pool"].clone()
    c["pool"][slot, 5] = 0x7F
    c["pool"][slot, 300:500] = 0xFF
    c["pool"][slot, 575] = 0x7F
    sees = torch.zeros((nq, nq), dtype=torch.bool)
    for i in range(nq):
        sees[i, :i + 1] = True
        sees[i, bad] = i in (bad, nq - 1)
    words = [int(sum(1 << k for k in range(nq) if sees[i, k])) for i in range(nq)] + [1]
    mask = torch.tensor(words, dtype=torch.int64, device="cuda")
    out, lse, _ = run(B, c, draft_mask=mask)
    for i in range(nq):
        if sees[i, bad]:
            assert bool(out[i].isnan().all()) and bool(lse[i].isnan().all())
    # the others: as if the place were not there
    zero = {**c, "pool": keep}
    zero["pool"][slot] = 0
    o, l, mag, es = reference(zero, draft_mask=mask)
    rows = [i for i in range(nq) if not sees[i, bad]] + [nq]
    want_o, want_l, _ = run(B, zero, draft_mask=mask)
    check(zero, want_o, want_l, draft_mask=mask)
    for i in rows:
        assert torch.equal(out[i], want_o[i]) and torch.equal(lse[i], want_l[i])


def test_malformed_parents(B):
    c = case([100, 100], [3, 3], 16, seed=8)
    parent = torch.tensor([-1, 0, 2, -1, 0, 1], dtype=torch.int32, device="cuda")  # the third's parent is itself
    out, lse, ws = run(B, c, parent=parent)
    assert B.verify_attn_mla_check(ws) == B.VMLA_ERR_PARENT
    words = torch.tensor([1, 3, 0, 1, 3, 7], dtype=torch.int64, device="cuda")
    check(c, out, lse, draft_mask=words)


def test_bad_lengths_compute_nothing(B):
    def refused(c, **change):
        T, H, _ = c["q"].shape
        out = torch.full((T, H, DV), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, H), 7.0, device="cuda")
        ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(len(c["nk"]), H, T, c["kv"].numel()), dtype=torch.uint8,
                         device="cuda")
        d = dict(kv_indptr=c["kv_indptr"], qo_indptr=c["qo_indptr"])
        d.update({k: torch.tensor(v, dtype=torch.int32, device="cuda") for k, v in change.items()})
        B.verify_attn_mla_scaled(c["q"], c["pool"], c["scales"], d["kv_indptr"], c["kv"], d["qo_indptr"], out, lse, ws, SM)
        assert B.verify_attn_mla_check(ws) == B.VMLA_ERR_SHAPE
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())

    c = case([100, 50], [3, 3], 16, seed=8)
    refused(c, kv_indptr=[0, 100, 151])       # past the entries there are
    refused(c, qo_indptr=[0, 3, 7])           # past the rows there are
    refused(c, kv_indptr=[0, 110, 100])       # falling
    refused(c, qo_indptr=[0, 4, 3])
    refused(c, kv_indptr=[0, 2, 50])          # more drafts than keys
    refused(c, kv_indptr=[1, 100, 150])
    refused(c, kv_indptr=[0, -5, 100])
    big = case([100, 100], [65, 1], 8, seed=8)
    refused(big)                              # more than 64 drafts


def test_captured_and_replayed_with_other_lengths(B):
    """One graph, captured once, replayed as the lengths, slots and queries change; two streams with workspaces of
    their own at the same time."""
    H, T, N = 16, 12, 4000
    first = case([900, 30, 1000], [1, 4, 1], H, seed=11)
    q = torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda")
    kv = torch.zeros(N, dtype=torch.int32, device="cuda")
    out = torch.zeros((T, H, DV), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((T, H), device="cuda")
    ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(3, H, T, N), dtype=torch.uint8, device="cuda")
    kvp, qop = first["kv_indptr"].clone(), first["qo_indptr"].clone()
    pool, scales = torch.zeros((5000, D), dtype=torch.uint8, device="cuda"), torch.zeros(5000, device="cuda")

    def fill(c):
        q.zero_()
        q[:c["q"].shape[0]] = c["q"]
        kv.fill_(-5)
        kv[:c["kv"].numel()] = c["kv"]
        kvp.copy_(c["kv_indptr"])
        qop.copy_(c["qo_indptr"])
        pool[:c["pool"].shape[0]] = c["pool"]
        scales[:c["scales"].numel()] = c["scales"]

    fill(first)
    call = lambda: B.verify_attn_mla_scaled(q, pool, scales, kvp, kv, qop, out, lse, ws, SM)  # noqa: E731
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for seed, (nk, nq) in enumerate([([900, 30, 1000], [1, 4, 1]), ([5, 2000, 700], [5, 2, 4]), ([0, 0, 1], [0, 0, 1]),
                                     ([64, 64, 3000], [0, 0, 12])]):
        c = case(nk, nq, H, seed=20 + seed)
        fill(c)
        g.replay()
        torch.cuda.synchronize()
        assert B.verify_attn_mla_check(ws) == 0
        check(c, out, lse)
        again = out.clone()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(again, out)
    a, b = case([3000], [2], H, seed=31), case([2500], [3], H, seed=32)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for _ in range(3):
        for c, s in ((a, sa), (b, sb)):
            with torch.cuda.stream(s):
                results.append((c, *run(B, c)[:2]))
    torch.cuda.synchronize()
    for c, o, l in results:
        check(c, o, l)


def test_a_wait_that_runs_out_is_reported(B):
    c = case([700], [1], 64, seed=13)
    B.verify_attn_mla_test_fault(1, 2_000_000)
    try:
        out, lse, ws = run(B, c)
        torch.cuda.synchronize()
        assert B.verify_attn_mla_check(ws) == B.VMLA_ERR_TIMEOUT
    finally:
        B.verify_attn_mla_test_fault(0, 0)
    out, lse, ws = run(B, c)
    assert B.verify_attn_mla_check(ws) == 0
    check(c, out, lse)
