"""The shared-prefix verify call on the GPU against a plain masked softmax attention in 64 bits.

Tolerances, fixed before the first run.  For one row, with mag = sum_j p_j |v_j| (p the softmax weights):
  - the weights are rounded to bf16 ahead of the product with the values: at most 2^-8 mag;
  - the scores are fp32 sums of 576 exact products and the exponential is good to 2^-22: the weights move by at
    most 2 x 576 x 2^-24 x scale x sum|q k| < 2^-9 relatively for the unit-variance inputs used here (sum|q k|
    below 250, scale 1/sqrt(192)): at most 2^-9 mag;
  - sums in fp32 and the merge: below 2^-12 mag;
  - the output is rounded to bf16: at most 2^-8 (|out| + the above).
lse: the score's error, below 576 x 2^-24 x scale x 250 < 1e-3."""
import numpy as np
import pytest

import oracle
from speculative_decoding_mla_gb300 import synth

pytestmark = pytest.mark.gpu
SCALE = synth.SM_SCALE


def _mods():
    import torch
    from speculative_decoding_mla_gb300 import build as vbuild
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return torch, binding


class Case:
    """A shared prefix of P rows and sequences of own_prefix[b] + drafts[b] own rows, slots permuted."""

    def __init__(self, P, own_prefix, drafts, H, *, tree=None, mask=None, fp8=False, seed=1, q_sigma=1.0, extra=7):
        torch, self.binding = _mods()
        g = torch.Generator().manual_seed(seed)
        nk = [p + d for p, d in zip(own_prefix, drafts)]
        self.kvh = np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)
        self.qoh = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.P, self.H, self.T, N = P, H, int(self.qoh[-1]), int(self.kvh[-1])
        S = P + N + extra
        perm = torch.randperm(S, generator=g).to(torch.int32)
        self.q = (torch.randn((self.T, H, 576), generator=g) * q_sigma).to(torch.bfloat16).cuda()
        pool = torch.randn((S, 576), generator=g) * 0.5
        self.kv_scale = 0.0
        if fp8:
            self.kv_scale = 0.0125
            self.pool = (pool / self.kv_scale).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
            self.values = (self.pool.view(torch.float8_e4m3fn).float() * self.kv_scale).to(torch.bfloat16)
        else:
            self.pool = pool.to(torch.bfloat16).cuda()
            self.values = self.pool
        self.shared, self.kvi = perm[:P].cuda(), perm[P:P + N].cuda()
        self.kvp, self.qop = torch.from_numpy(self.kvh).cuda(), torch.from_numpy(self.qoh).cuda()
        self.parent = None
        if tree:
            par = np.concatenate([synth.tree_parents(seed, d, tree, b) for b, d in enumerate(drafts) if d]).astype(np.int32)
            self.parent = torch.from_numpy(par).cuda()
        self.mask = None if mask is None else torch.from_numpy(np.asarray(mask, np.uint64).view(np.int64)).cuda()
        self.drafts = drafts
        if mask is not None:
            self.words = np.asarray(mask, np.uint64)
        elif tree:
            self.words = oracle.tree_masks(par, self.qoh)
        else:
            self.words = np.array([(1 << (i + 1)) - 1 for d in drafts for i in range(d)], np.uint64)

    def alloc(self, splits=0):
        import torch
        self.out = torch.full((self.T, self.H, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T, self.H), 7.0, device="cuda")
        n = self.binding.verify_attn_mla_shared_workspace_size(self.P, self.qoh, self.kvh, self.H, splits)
        self.ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda").fill_(0xFF)
        return self

    def args(self):
        return (self.q, self.pool, self.shared, self.kvp, self.kvi, self.qop, self.kvh, self.qoh, self.out, self.lse,
                self.ws, SCALE)

    def run(self, splits=0, stream=None):
        import torch
        self.alloc(splits)
        self.binding.verify_attn_mla_shared(*self.args(), kv_scale=self.kv_scale, draft_mask=self.mask,
                                            parent=self.parent, splits=splits, stream=stream)
        st = self.binding.verify_attn_mla_check(self.ws, stream)
        torch.cuda.synchronize()
        return st

    def reference(self):
        """(out, lse, mag) in 64 bits, rows of no visible key as out 0, lse -inf."""
        vals = self.values.double().cpu().numpy()
        q = self.q.double().cpu().numpy()
        sh, kvi = self.shared.cpu().numpy(), self.kvi.cpu().numpy()
        out, mag = np.zeros((self.T, self.H, 512)), np.zeros((self.T, self.H, 512))
        lse = np.full((self.T, self.H), -np.inf)
        for b, d in enumerate(self.drafts):
            rows = vals[np.concatenate([sh, kvi[self.kvh[b]:self.kvh[b + 1]]])]
            pre = len(rows) - d
            for i in range(d):
                t = self.qoh[b] + i
                see = np.concatenate([np.ones(pre, bool), [(int(self.words[t]) >> k) & 1 == 1 for k in range(d)]]).astype(bool)
                use = rows[see]
                if not len(use):
                    continue
                s = (q[t] @ use.T) * SCALE
                m = s.max(1, keepdims=True)
                e = np.exp(s - m)
                p = e / e.sum(1, keepdims=True)
                out[t], mag[t] = p @ use[:, :512], p @ abs(use[:, :512])
                lse[t] = (m + np.log(e.sum(1, keepdims=True)))[:, 0]
        return out, lse, mag

    def compare(self, ref=None):
        out, lse, mag = ref or self.reference()
        got, gl = self.out.double().cpu().numpy(), self.lse.double().cpu().numpy()
        slack = (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12) * mag
        bad = abs(got - out) > slack + 2.0 ** -8 * (abs(out) + slack)
        assert not bad.any(), (np.argwhere(bad)[:5], abs(got - out).max())
        assert np.array_equal(np.isneginf(gl), np.isneginf(lse))
        fin = np.isfinite(lse)
        assert fin.sum() == 0 or abs(gl[fin] - lse[fin]).max() < 1e-3


CASES = {
    "one_key_each": dict(P=1, own_prefix=[0], drafts=[1], H=1),
    "tile_edges": dict(P=127, own_prefix=[0, 1, 127, 128, 129], drafts=[1, 1, 1, 2, 3], H=8),
    "one_tile": dict(P=128, own_prefix=[5, 0], drafts=[1, 64], H=64),
    "past_a_tile": dict(P=129, own_prefix=[300, 20], drafts=[2, 1], H=33),
    "empty_sequences": dict(P=700, own_prefix=[40, 10, 0, 0, 200], drafts=[3, 0, 0, 5, 0], H=16),
    "many_queries": dict(P=1500, own_prefix=[90] * 20, drafts=[1] * 20, H=64),
    "wide_heads": dict(P=513, own_prefix=[64, 33], drafts=[7, 9], H=128),
    "trees": dict(P=900, own_prefix=[100, 0, 31], drafts=[64, 17, 40], H=16, tree=6),
    "codes": dict(P=640, own_prefix=[100, 17], drafts=[5, 1], H=24, fp8=True),
    "long_own": dict(P=40, own_prefix=[3000, 10], drafts=[4, 4], H=16),
}


@pytest.mark.parametrize("name", list(CASES))
@pytest.mark.parametrize("splits", [0, 1, 2, 7, 64, -1])
def test_against_64_bits(name, splits):
    c = Case(**CASES[name])
    assert c.run(splits) == 0
    c.compare()


def test_splits_agree_and_calls_repeat():
    """The same call twice gives the same bits; another split count the same up to rounding."""
    torch, _ = _mods()
    c = Case(**CASES["many_queries"])
    c.run()
    first = (c.out.clone(), c.lse.clone())
    c.run()
    assert torch.equal(first[0].view(torch.int16), c.out.view(torch.int16)) and torch.equal(first[1], c.lse)


def test_explicit_masks_with_hidden_drafts():
    """A draft that sees no draft at all still sees the shared rows; one that sees only itself, too."""
    drafts = [3, 2]
    c = Case(200, [0, 50], drafts, 16, mask=[0, 0b010, 0b111, 0, 0b01])
    assert c.run() == 0
    c.compare()


def test_nothing_shared_is_the_plain_call():
    torch, binding = _mods()
    c = Case(0, [300, 40], [4, 1], 16)
    assert c.run() == 0
    c.compare()
    out, lse = c.out.clone(), c.lse.clone()
    n = binding.verify_attn_mla_workspace_size(c.qoh, c.kvh, c.H)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    binding.verify_attn_mla(c.q, c.pool, c.kvp, c.kvi, c.qop, c.kvh, c.qoh, c.out, c.lse, ws, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), c.out.view(torch.int16)) and torch.equal(lse, c.lse)


def test_nothing_asked():
    c = Case(100, [10, 20], [0, 0], 16)
    assert c.run() == 0


@pytest.mark.parametrize("strong", ["shared", "own"])
def test_one_side_outweighs_the_other(strong):
    """Scores that differ by hundreds between the shared and the own rows: one side's weight vanishes."""
    torch, _ = _mods()
    c = Case(300, [200, 100], [2, 3], 16, seed=4)
    at = (c.shared if strong == "shared" else c.kvi).long()
    # a common direction: the queries lie along it and only one side's rows have it
    d = torch.randn(576, device="cuda").sign()
    c.q = (c.q.float() * 0.1 + 0.9 * d).to(torch.bfloat16)
    rows = c.pool.float()
    rows -= (rows @ d)[:, None] * d / 576
    rows[at] += 6.0 * d / 576 ** 0.5 * torch.rand((len(at), 1), device="cuda")
    c.pool = c.values = rows.to(torch.bfloat16)
    assert c.run() == 0
    c.compare()


def test_other_sequences_rows_do_not_matter():
    """Sequence 1's own rows hold NaN and infinities: the others' results keep their bits."""
    torch, _ = _mods()
    c = Case(1000, [70, 50, 33, 10], [3, 2, 4, 1], 16, seed=2)
    assert c.run() == 0
    out, lse = c.out.clone(), c.lse.clone()
    mine = c.kvi[c.kvh[1]:c.kvh[2]].long()
    c.pool[mine] = float("nan")
    c.pool[mine[::2]] = float("inf")
    free = torch.ones(c.pool.shape[0], dtype=torch.bool, device="cuda")
    free[torch.cat([c.shared, c.kvi]).long()] = False
    c.pool[free] = float("nan")  # and so do slots that nobody reads
    c.run()
    for b in (0, 2, 3):
        r = slice(int(c.qoh[b]), int(c.qoh[b + 1]))
        assert torch.equal(out[r].view(torch.int16), c.out[r].view(torch.int16)) and torch.equal(lse[r], c.lse[r])


def test_bad_slots_are_reported():
    torch, binding = _mods()
    for where, at in (("shared", 40), ("kvi", 77)):
        c = Case(64, [60, 20], [2, 3], 8)
        getattr(c, where)[at] = c.pool.shape[0] if where == "shared" else -1
        assert c.run() == binding.VMLA_ERR_INDEX
        assert int(c.ws[4:8].view(torch.int32)) == (40 if where == "shared" else 64 + 77)
        # the row counts as zeros
        full = torch.cat([c.pool, torch.zeros_like(c.pool[:1])])
        c.values = full
        getattr(c, where)[at] = c.pool.shape[0]
        c.compare()


def test_malformed_parent_is_reported():
    _, binding = _mods()
    c = Case(100, [10, 10], [4, 5], 8, tree=3)
    c.parent[6] = 5
    assert c.run() == binding.VMLA_ERR_PARENT


def test_workspace_checks():
    torch, binding = _mods()
    c = Case(**CASES["many_queries"]).alloc()
    full = c.ws
    for n in (0, 256, full.numel() - 256):
        c.ws = full[:n] if n else full[:0]
        with pytest.raises(binding.VmlaError) as e:
            binding.verify_attn_mla_shared(*c.args())
        assert e.value.status in (binding.VMLA_ERR_WORKSPACE, binding.VMLA_ERR_NULL)
    torch.cuda.synchronize()
    assert (c.out == 7).all() and (c.lse == 7).all()


def test_two_streams_and_two_workspaces():
    torch, _ = _mods()
    a, b = Case(**CASES["trees"]), Case(**CASES["many_queries"])
    ra, rb = a.reference(), b.reference()
    a.alloc(), b.alloc()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        a.binding.verify_attn_mla_shared(*a.args(), parent=a.parent, stream=sa)
        b.binding.verify_attn_mla_shared(*b.args(), stream=sb)
    torch.cuda.synchronize()
    assert a.binding.verify_attn_mla_check(a.ws) == 0 and b.binding.verify_attn_mla_check(b.ws) == 0
    a.compare(ra)
    b.compare(rb)


def test_captured_and_replayed():
    """A captured call reads new indices, rows and queries at the replay (lengths as captured)."""
    torch, _ = _mods()
    c = Case(**CASES["long_own"])
    c.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.binding.verify_attn_mla_shared(*c.args())
    c.q.copy_(torch.randn(c.q.shape, device="cuda").to(torch.bfloat16))
    c.shared.copy_(c.shared.flip(0))
    c.pool.copy_(c.pool.flip(0))
    c.out.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    c.compare()


def test_prepared_call():
    torch, binding = _mods()
    c = Case(**CASES["past_a_tile"]).alloc()
    call = binding.prepare_verify_attn_mla_shared(*c.args())
    call()
    call()
    torch.cuda.synchronize()
    c.compare()


def test_equals_the_plain_call_on_joined_rows():
    """Against verify_attn_mla with the shared slots in front of every sequence: both within rounding of each other
    (twice the tolerance of one)."""
    torch, binding = _mods()
    c = Case(3000, [500, 20, 100], [4, 4, 4], 64, seed=9)
    assert c.run() == 0
    kvi = torch.cat([x for b in range(3) for x in (c.shared, c.kvi[c.kvh[b]:c.kvh[b + 1]])]).contiguous()
    kvh = (c.kvh + 3000 * np.arange(4)).astype(np.int32)
    out, lse = torch.empty_like(c.out), torch.empty_like(c.lse)
    ws = torch.empty(binding.verify_attn_mla_workspace_size(c.qoh, kvh, 64), dtype=torch.uint8, device="cuda")
    binding.verify_attn_mla(c.q, c.pool, torch.from_numpy(kvh).cuda(), kvi, c.qop, kvh, c.qoh, out, lse, ws, SCALE)
    assert binding.verify_attn_mla_check(ws) == 0
    assert (out.float() - c.out.float()).abs().max() < 2e-2 and (lse - c.lse).abs().max() < 2e-3


def test_over_64_sequences_and_many_launches():
    """More sequences than the piece-size search covers and more units than one launch holds."""
    c = Case(700, [3] * 100, [1] * 100, 16, seed=6)
    assert c.run() == 0
    c.compare()
    c = Case(130, [1] * 511, [8] * 511, 64, seed=7)  # 511 own units x 2 row blocks, 1,022 row blocks over the prefix
    assert c.run(splits=2) == 0
    t = np.random.default_rng(0).choice(c.T, 40, replace=False)
    sub = set(t.tolist())
    full = c.drafts
    out, lse, mag = _rows_reference(c, sorted(sub))
    got = c.out[sorted(sub)].double().cpu().numpy()
    slack = (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12) * mag
    assert (abs(got - out) <= slack + 2.0 ** -8 * (abs(out) + slack)).all()
    assert abs(c.lse[sorted(sub)].double().cpu().numpy() - lse).max() < 1e-3
    assert len(full) == 511


def _rows_reference(c, rows):
    vals, q = c.values.double().cpu().numpy(), c.q.double().cpu().numpy()
    sh, kvi = c.shared.cpu().numpy(), c.kvi.cpu().numpy()
    out, lse, mag = [], [], []
    for t in rows:
        b = int(np.searchsorted(c.qoh, t, side="right")) - 1
        own = kvi[c.kvh[b]:c.kvh[b + 1]]
        i = t - c.qoh[b]
        use = vals[np.concatenate([sh, own[:len(own) - c.drafts[b] + i + 1]])]
        s = (q[t] @ use.T) * SCALE
        m = s.max(1, keepdims=True)
        e = np.exp(s - m)
        p = e / e.sum(1, keepdims=True)
        out.append(p @ use[:, :512])
        mag.append(p @ abs(use[:, :512]))
        lse.append((m + np.log(e.sum(1, keepdims=True)))[:, 0])
    return np.array(out), np.array(lse), np.array(mag)
