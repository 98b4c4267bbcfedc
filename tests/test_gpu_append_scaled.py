"""Append of rows as e4m3 codes with a scale per block of slots."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D, DV, DR = 576, 512, 64


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def values(codes):
    return codes.view(torch.float8_e4m3fn).float()


class Case:
    def __init__(self, runs, block, heads=0, interleaved=True, seed=0, gain=None, pad=()):
        """runs: (block, first row in it, rows) in the call's order; pad: places of padding tokens."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.block, self.runs, self.interleaved = block, runs, interleaved
        blocks = max(b for b, _, _ in runs) + 2
        self.pool = (torch.randn((blocks * block, D), generator=g, device="cuda") * 100).to(torch.float8_e4m3fn).view(torch.uint8)
        self.scales = torch.exp2(torch.randint(-9, -5, (blocks,), generator=g, device="cuda").float())
        slots = [b * block + r + k for b, r, n in runs for k in range(n)]
        for p in pad:
            slots.insert(p, -1)
        T = len(slots)
        self.slots = torch.tensor(slots, dtype=torch.int32, device="cuda")
        self.positions = torch.randint(0, 5000, (T,), generator=g, device="cuda", dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
        angle = torch.arange(5000, dtype=torch.float64, device="cuda")[:, None] * freq
        self.table = torch.cat([angle.cos(), angle.sin()], 1).float()
        size = torch.exp(torch.randn((T, 1), generator=g, device="cuda")) if gain is None else gain
        self.kv = (torch.randn((T, D), generator=g, device="cuda") * size).to(torch.bfloat16)
        self.q = self.q_rope = None
        if heads:
            self.q = torch.randn((T, heads, D), generator=g, device="cuda").to(torch.bfloat16)
            self.q_rope = torch.randn((T, heads, DR), generator=g, device="cuda").to(torch.bfloat16)
        self.status = torch.zeros(2, dtype=torch.int32, device="cuda")

    def call(self, B):
        B.verify_attn_mla_append_scaled(self.kv[:, :DV], self.kv[:, DV:], self.positions, self.slots, self.table, self.pool, self.scales,
                                        block_tokens=self.block, q_rope=self.q_rope, q=self.q, interleaved=self.interleaved,
                                        status_word=self.status)

    def rows(self):
        cs = self.table[self.positions.long().clamp(max=4999)].double()  # (a token left out has any row)
        z = torch.complex(cs[:, :32], cs[:, 32:])
        r = self.kv[:, DV:].double()
        r = (torch.complex(r[:, 0::2], r[:, 1::2]) if self.interleaved else torch.complex(r[:, :32], r[:, 32:])) * z
        r = torch.view_as_real(r).flatten(-2) if self.interleaved else torch.cat([r.real, r.imag], -1)
        return torch.cat([self.kv[:, :DV].double(), r], 1)

    def check(self, pool0, scales0, use=None):
        """use: which tokens were written (all with a slot)."""
        rows, slots = self.rows(), self.slots.cpu().numpy()
        use = slots >= 0 if use is None else use
        pool, scales = values(pool0).double().cpu(), scales0.double().cpu().numpy().copy()
        got, got_scales = values(self.pool).double().cpu(), self.scales.double().cpu().numpy()
        tol = torch.zeros_like(pool)
        t = 0
        order = [k for k in range(len(slots))]
        while t < len(order):
            if slots[t] < 0:
                t += 1
                continue
            e, run = t, []  # padding may stand between a block's tokens
            while e < len(order) and (slots[e] < 0 or slots[e] // self.block == slots[t] // self.block):
                run += [e] if use[e] else []
                e += 1
            t = e
            if not run:
                continue
            b, first = slots[run[0]] // self.block, slots[run[0]] % self.block
            most = float(rows[run].abs().max())
            need = 2.0 ** -100
            if most > 0:
                need = max(need, 2.0 ** math.ceil(math.log2(most / 448) - 1e-12))
                if 448 * need < most * (1 - 1e-12):
                    need *= 2
            now = need if first == 0 else max(scales[b], need)
            if first and now > scales[b]:
                at = slice(b * self.block, b * self.block + first)
                exact = pool[at] * (scales[b] / now)
                pool[at] = exact.float().to(torch.float8_e4m3fn).double()
            scales[b] = now
            for k in run:
                exact = rows[k].cpu() / now
                pool[slots[k], :DV] = exact[:DV].clamp(-448, 448).float().to(torch.float8_e4m3fn).double()
                pool[slots[k], DV:] = exact[DV:].clamp(-448, 448)
                # the rotated columns are off by their fp32 sums and one rounding: half of 2^-3, or half the smallest code
                tol[slots[k], DV:] = exact[DV:].abs() * (2.0 ** -4 * (1 + 2.0 ** -20)) + 2.0 ** -10
        assert np.array_equal(got_scales, scales)
        # (codes of NaN among what the pool held before stay)
        assert bool((((got - pool).abs() <= tol) | (torch.isnan(got) & torch.isnan(pool))).all())


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("block,runs", [
    (1, [(3, 0, 1), (0, 0, 1), (7, 0, 1)]),
    (8, [(2, 0, 8), (0, 3, 1), (1, 5, 3), (4, 0, 1), (5, 7, 1)]),
    (64, [(0, 63, 1), (1, 0, 64), (2, 0, 17), (4, 20, 9)]),
    (128, [(1, 100, 28), (2, 0, 128), (3, 0, 1)]),
    (2, [(k, k % 2, 1) for k in range(50)]),
])
def test_codes_and_scales(B, block, runs, interleaved):
    c = Case(runs, block, heads=5, interleaved=interleaved, seed=block, pad=(0, 2))
    pool0, scales0, q0 = c.pool.clone(), c.scales.clone(), c.q.clone()
    c.call(B)
    c.check(pool0, scales0)
    assert c.status.tolist() == [0, 0]
    # the queries' turn is the other append's, bit for bit
    want, other = q0.clone(), torch.zeros((int(c.slots.max()) + 1, D), dtype=torch.bfloat16, device="cuda")
    B.verify_attn_mla_append(c.kv[:, :DV], c.kv[:, DV:], c.positions, c.slots, c.table, other, q_rope=c.q_rope, q=want, interleaved=interleaved)
    assert torch.equal(c.q, want)
    # appending the same rows again changes nothing
    pool1, scales1 = c.pool.clone(), c.scales.clone()
    c.call(B)
    assert torch.equal(c.pool, pool1) and torch.equal(c.scales, scales1)


def test_prompts_longer_than_a_window(B):
    """Many tokens: windows of a block, runs that begin in one window and end in the next."""
    for block in (8, 64):
        runs, left, b = [], 3001, 0
        first = block - 3
        while left:
            n = min(block - first, left)
            runs.append((b, first, n))
            left -= n
            b, first = b + 1, 0
        c = Case(runs, block, heads=3, seed=block, pad=(5, 1000))
        pool0, scales0 = c.pool.clone(), c.scales.clone()
        c.call(B)
        c.check(pool0, scales0)


def test_scales_at_the_borders(B):
    """448 x 2^k exactly, the next bf16 above, zeros, the largest and smallest numbers."""
    sizes = [448.0, 450.0, 0.0, 1.75, 1.7578125, 3.3895e38, 1e-38, 2.0 ** -94, 2.0 ** -90]
    c = Case([(k, 0, 1) for k in range(len(sizes))], 1, seed=2)
    c.kv.zero_()
    for k, s in enumerate(sizes):
        c.kv[k, 7 * k] = -s
    pool0, scales0 = c.pool.clone(), c.scales.clone()
    c.call(B)
    c.check(pool0, scales0)
    want = [1.0, 2.0, 2.0 ** -100, 2.0 ** -8, 2.0 ** -7]
    assert c.scales[:5].tolist() == want
    assert bool((values(c.pool[2]) == 0).all())


def test_rows_in_front_are_coded_again_once(B):
    c = Case([(1, 5, 2)], 16, seed=3, gain=300.0)
    pool0, scales0 = c.pool.clone(), c.scales.clone()
    c.call(B)
    c.check(pool0, scales0)
    assert float(c.scales[1]) > float(scales0[1])
    assert torch.equal(c.pool[:16], pool0[:16]) and torch.equal(c.pool[23:], pool0[23:])  # other rows keep their codes


def test_scales_that_are_no_powers_of_two(B):
    """A block of another writer: its scale stays while the rows fit, and their codes are divided."""
    c = Case([(0, 4, 2), (1, 0, 3)], 8, seed=4, gain=0.01)
    c.scales.fill_(0.0173)
    pool0, scales0 = c.pool.clone(), c.scales.clone()
    c.call(B)
    assert float(c.scales[0]) == float(scales0[0])
    want = (c.kv[:2, :DV].float() / scales0[0]).to(torch.float8_e4m3fn).float()
    assert torch.equal(values(c.pool[4:6])[:, :DV], want)
    assert torch.equal(c.pool[:4], pool0[:4])


def test_infinities_and_nan(B):
    c = Case([(0, 0, 1), (1, 0, 1)], 1, seed=5)
    c.kv[0, 3] = math.inf
    c.kv[1, 4] = math.nan
    c.call(B)
    assert float(values(c.pool[0])[3]) == 448.0 and float(c.scales[0]) == 2.0 ** 120
    assert bool(torch.isnan(values(c.pool[1])[4])) and int(torch.isnan(values(c.pool[1])).sum()) == 1


def test_bad_slots_and_positions_are_left_out(B):
    for block in (1, 8):
        runs = [(0, 0, 1), (1, 0, 1), (2, 0, 1), (3, 0, 1)] if block == 1 else [(0, 2, 4)]
        c = Case(runs, block, heads=2, seed=6)
        q0 = c.q.clone()
        c.kv[1] = 1000.0  # takes no part in the scale
        c.positions[1] = 5000
        pool0, scales0 = c.pool.clone(), c.scales.clone()
        c.call(B)
        assert c.status.tolist() == [B.VMLA_ERR_INDEX, 1]
        c.check(pool0, scales0, use=np.array([True, False, True, True]))
        assert torch.equal(c.q[1], q0[1]) and torch.equal(c.pool[int(c.slots[1])], pool0[int(c.slots[1])])
        for bad in (-2, c.pool.shape[0], 2 ** 31 - 1):
            c = Case(runs, block, seed=7)
            c.slots[3] = bad
            pool0, scales0 = c.pool.clone(), c.scales.clone()
            c.call(B)
            assert c.status.tolist() == [B.VMLA_ERR_INDEX, 3]
            c.slots[3] = -1
            c.check(pool0, scales0)


def test_captured_and_replayed(B):
    c = Case([(0, 3, 2), (1, 0, 5)], 8, heads=4, seed=8)
    c.call(B)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.call(B)
    for seed in (9, 10):
        d = Case([(1, 6, 2), (0, 0, 5)], 8, heads=4, seed=seed)
        for name in ("kv", "slots", "positions", "pool", "scales", "q_rope"):
            getattr(c, name).copy_(getattr(d, name))
        pool0, scales0 = c.pool.clone(), c.scales.clone()
        g.replay()
        torch.cuda.synchronize()
        c.check(pool0, scales0)


@pytest.mark.parametrize("tokens", [600, 9000])
def test_padding_in_front_between_and_behind(B, tokens):
    """A padded batch: long stretches without slots, few tokens to write."""
    runs = [(3, 0, 64), (1, 60, 4), (7, 5, 20)]
    c = Case(runs, 64, heads=2, seed=tokens, pad=[0] * (tokens // 3) + [tokens // 3 + 40] * 100 + [tokens // 3 + 100 + 88] * (tokens // 2))
    pool0, scales0, q0 = c.pool.clone(), c.scales.clone(), c.q.clone()
    c.call(B)
    c.check(pool0, scales0)
    assert c.status.tolist() == [0, 0]
    pad = c.slots < 0
    assert torch.equal(c.q[pad], q0[pad]) and not torch.equal(c.q[~pad], q0[~pad])
