"""The tables of a step from its requests' lengths, against a plain loop."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def ints(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Step:
    """Tables with room to spare, and what they ought to become."""

    def __init__(self, cached, added, block, room_kv=7, room_q=3, room_free=5, width=None, seed=0, pad=0):
        r = np.random.default_rng(seed)
        n = [c + a for c, a in zip(cached, added)]
        need, have = [-(-x // block) for x in n], [-(-c // block) for c in cached]
        self.block, Bn = block, len(cached)
        self.width = max(need + [0]) + 2 if width is None else width
        ids = r.permutation(sum(need) + room_free + 11).astype(np.int32)
        base = np.full((max(Bn, 0), self.width + pad), -1, np.int32)
        at = 0
        for b in range(Bn):
            base[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        free = ids[at:at + sum(need) - sum(have) + room_free]
        self.cached, self.added = ints(cached), ints(added)
        self.base = torch.from_numpy(base).cuda()
        self.table = self.base[:, :self.width]
        self.free, self.count = ints(free), ints([len(free)])
        self.left, self.scratch = ints([99]), ints([0])
        self.kv_indptr, self.qo_indptr = ints([9] * (Bn + 1)), ints([9] * (Bn + 1))
        self.kv = ints([-3] * (sum(n) + room_kv))
        self.positions, self.slots = ints([-3] * (sum(added) + room_q)), ints([-3] * (sum(added) + room_q))
        self.status = ints([0, 0])
        # the plain loop
        want = base.copy()
        left, kv, pos, slots = len(free), [], [], []
        for b in range(Bn):
            for k in range(have[b], need[b]):
                left -= 1
                want[b, k] = free[left]
            s = [int(want[b, p // block]) * block + p % block for p in range(n[b])]
            kv += s
            pos += list(range(cached[b], n[b]))
            slots += s[cached[b]:]
        self.want = dict(base=want, left=[left], kv_indptr=np.concatenate([[0], np.cumsum(n)]), qo_indptr=np.concatenate([[0], np.cumsum(added)]),
                         kv=kv + [-3] * room_kv, positions=pos + [0] * room_q, slots=slots + [-1] * room_q)

    def call(self, B, in_place=False):
        B.verify_attn_mla_step_tables(self.cached, self.added, self.table, self.free, self.count, self.count if in_place else self.left,
                                      self.scratch, self.kv_indptr, self.qo_indptr, self.kv, self.positions, self.slots,
                                      block_tokens=self.block, status_word=self.status)

    def check(self, in_place=False):
        for name, want in self.want.items():
            got = self.count if name == "left" and in_place else getattr(self, name)
            assert np.array_equal(got.cpu().numpy(), np.asarray(want)), name
        assert self.scratch.tolist() == [0] and self.status.tolist() == [0, 0]


@pytest.mark.parametrize("block", [1, 2, 16, 64, 128])
@pytest.mark.parametrize("cached,added", [([0], [1]), ([5, 0, 128, 63, 64], [1, 0, 4, 1, 64]), ([0, 0, 0], [0, 0, 0]),
                                          ([1000, 1, 4097], [3000, 2, 1]), ([127, 128, 129], [1, 1, 1])])
def test_against_a_loop(B, cached, added, block):
    for in_place in (False, True):
        s = Step(cached, added, block, seed=block, pad=3)
        s.call(B, in_place)
        s.check(in_place)


def test_largest_batch_and_long_requests(B):
    r = np.random.default_rng(1)
    for block in (1, 64):
        s = Step(r.integers(0, 900, 512).tolist(), r.integers(0, 5, 512).tolist(), block)
        s.call(B)
        s.check()
        s = Step([300000, 5, 131072], [1, 1, 64], block)
        s.call(B)
        s.check()


def test_no_requests(B):
    s = Step([], [], 16)
    s.call(B)
    s.check()


def refused(B, s, code, info):
    before = {k: getattr(s, k).clone() for k in ("base", "kv", "count")}
    s.call(B)
    assert s.status.tolist() == [code, info]
    for k, v in before.items():
        assert torch.equal(getattr(s, k), v), k
    assert bool((s.kv_indptr == 0).all()) and bool((s.qo_indptr == 0).all()) and bool((s.slots == -1).all())
    assert s.left.tolist() == s.count.tolist() and s.scratch.tolist() == [0]


def test_steps_that_do_not_fit_are_empty(B):
    refused(B, Step([5, 9], [1, 2], 4, room_kv=-1), B.VMLA_ERR_FULL, 0)
    refused(B, Step([5, 9], [1, 2], 4, room_q=-1), B.VMLA_ERR_FULL, 0)
    refused(B, Step([4, 8], [1, 2], 4, room_free=-1), B.VMLA_ERR_FULL, 0)
    s = Step([4, 8, 4], [1, 2, 5], 4)
    s.added[1] = -1
    refused(B, s, B.VMLA_ERR_SHAPE, 1)
    s = Step([4, 8, 4], [1, 2, 5], 4)
    s.cached[2] = -4
    refused(B, s, B.VMLA_ERR_SHAPE, 2)
    s = Step([4, 8, 4], [1, 2, 5], 4)
    s.added[2] = 2 ** 31 - 1
    refused(B, s, B.VMLA_ERR_SHAPE, 2)
    s = Step([4, 8], [1, 2], 4)
    s.count[0] = 10 ** 6  # more than the list holds
    refused(B, s, B.VMLA_ERR_FULL, 0)


def test_broken_entries_give_no_slot(B):
    s = Step([8, 8], [1, 1], 4)
    s.table[0, 1] = -7
    s.table[1, 0] = 2 ** 30  # its slots pass 2^31
    s.call(B)
    kv = s.kv.tolist()
    assert kv[4:8] == [-1] * 4 and kv[9:13] == [-1] * 4
    assert all(v >= 0 for v in kv[:4] + kv[8:9] + kv[13:18])


def test_captured_steps_go_on_where_the_last_stopped(B):
    """One graph, replayed: the lengths grow by the step's tokens, the free list shrinks in place."""
    cached, added, block = [3, 0, 17], [2, 1, 4], 4
    s = Step(cached, added, block, room_kv=200, room_q=0, room_free=60, width=30)
    s.call(B, True)
    torch.cuda.synchronize()
    s.check(True)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call(B, True)
    # the first call's blocks are taken; each replay appends the same numbers of tokens again
    base, free = s.base.cpu().numpy().copy(), s.free.cpu().numpy()
    lengths, left = [c + a for c, a in zip(cached, added)], int(s.count[0])
    for _ in range(5):
        s.cached.copy_(ints(lengths))
        g.replay()
        torch.cuda.synchronize()
        kv = []
        for b, (c, a) in enumerate(zip(lengths, added)):
            for k in range(-(-c // block), -(-(c + a) // block)):
                left -= 1
                base[b, k] = free[left]
            kv += [int(base[b, p // block]) * block + p % block for p in range(c + a)]
        assert np.array_equal(s.base.cpu().numpy(), base)
        assert s.count.tolist() == [left] and s.kv.tolist()[:len(kv)] == kv
        lengths = [c + a for c, a in zip(lengths, added)]


@pytest.mark.parametrize("block", [1, 4, 32, 128])
def test_long_requests_with_broken_entries_and_outputs_of_any_alignment(B, block):
    """Whole stretches of keys in old blocks: negative blocks, blocks whose slots pass 2^31, arrays off 16 bytes."""
    r = np.random.default_rng(block)
    for off in range(4):
        s = Step([5000, 300, 2049, 256, 255], [3, 0, 64, 1, 257], block, seed=off)
        broken = {}
        for b, n in enumerate([5000, 300, 2049, 256, 255]):
            for k in r.integers(0, -(-n // block), 3):
                broken[b, int(k)] = int(r.choice([-1, -2 ** 31, 2 ** 31 - 1, 2 ** 31 // block - 1]))
        for (b, k), v in broken.items():
            s.base[b, k] = v
            s.want["base"][b, k] = v
        whole = torch.full((s.kv.numel() + off,), -3, dtype=torch.int32, device="cuda")
        s.kv = whole[off:]
        s.call(B)
        kv, first = np.array(s.want["kv"]), s.want["kv_indptr"]
        for (b, k), v in broken.items():
            for p in range(k * block, min((k + 1) * block, int(first[b + 1] - first[b]))):
                slot = v * block + p % block
                kv[first[b] + p] = slot if 0 <= slot < 2 ** 31 else -1
        s.want["kv"] = kv
        slots = []
        for b, n in enumerate([3, 0, 64, 1, 257]):
            slots += list(kv[first[b + 1] - n:first[b + 1]])
        s.want["slots"] = slots + [-1] * 3
        s.check()
        assert bool((whole[:off] == -3).all())
