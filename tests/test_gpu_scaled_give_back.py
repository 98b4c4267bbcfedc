"""Slots of dropped beams go back to the free list, on the device: steps go on where they would otherwise end in a full pool."""
import pytest
import torch

from tests.test_gpu_scaled_step import Beams, i32

pytestmark = pytest.mark.gpu
PROMPTS, PAIRS = [50, 1, 200], 12


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


class Small(Beams):
    """The same beams in a pool with `room` slots behind the prompts; the other slots are nobody's."""

    def __init__(self, B, prompts, room):
        super().__init__(B, prompts)
        held = torch.ones(self.slots_all + 1, dtype=torch.int32, device="cuda")
        held[self.free[:room].long()] = 0
        held[self.table[self.table >= 0].long()] = 0
        self.held, self.free, self.count[0] = held, torch.cat([self.free[:room], i32(self.slots_all - room)]), room

    def give_back(self):
        used = self.held.clone()
        live = torch.arange(self.table.shape[1], device="cuda") < self.cached[:, None]
        used.scatter_(0, torch.where(live & (self.table >= 0), self.table, self.slots_all).view(-1).long(), 1)
        used = used[:self.slots_all]
        self.free.copy_(used.argsort(stable=True))  # free slots first
        self.count.copy_(self.slots_all - used.sum())


def live_slots(b):
    return b.table[torch.arange(b.table.shape[1], device="cuda") < b.cached[:, None]].unique()


@pytest.fixture(scope="module")
def room(B):
    """As many slots as the beams' tables reach at the most, and a pair of steps' tokens."""
    b, most = Beams(B, PROMPTS), 0
    for _ in range(PAIRS):
        b.two_steps()
        most = max(most, live_slots(b).numel() - sum(PROMPTS))
    taken = b.slots_all - sum(PROMPTS) - int(b.count)
    assert b.status.tolist() == [0, 0] and taken == 2 * PAIRS * b.R * b.W and most + 4 * b.R * b.W < taken
    return most + 2 * b.R * b.W


def same(a, b):
    for x, y in ((a.token, b.token), (a.score, b.score), (a.out, b.out), (a.lse, b.lse), (a.cached, b.cached), (a.parent, b.parent)):
        assert torch.equal(x, y)


def test_without_it_the_pool_is_full(B, room):
    b = Small(B, PROMPTS, room)
    for _ in range(PAIRS):
        b.two_steps()
    assert b.status.tolist() == [B.VMLA_ERR_FULL, 0]


def test_steps_go_on(B, room):
    b, wide = Small(B, PROMPTS, room), Beams(B, PROMPTS)
    for _ in range(PAIRS):
        b.two_steps()
        wide.two_steps()
        assert b.status.tolist() == wide.status.tolist() == [0, 0]
        same(b, wide)
        b.give_back()
        now = b.free[:int(b.count)]
        assert now.unique().numel() == now.numel() == room - (live_slots(b).numel() - sum(PROMPTS))
        assert not bool(torch.isin(now, live_slots(b)).any()) and not bool((b.held[now.long()] != 0).any())


def test_captured(B, room):
    eager, b = Small(B, PROMPTS, room), Small(B, PROMPTS, room)
    start = [t.clone() for t in vars(b).values() if torch.is_tensor(t)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.two_steps()  # (warm-up)
        b.give_back()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.two_steps()
            b.give_back()
    torch.cuda.current_stream().wait_stream(side)
    for t, v in zip([t for t in vars(b).values() if torch.is_tensor(t)], start):
        t.copy_(v)
    for _ in range(PAIRS):
        eager.two_steps()
        eager.give_back()
        graph.replay()
    torch.cuda.synchronize()
    same(eager, b)
    assert b.status.tolist() == [0, 0] and int(b.count) == int(eager.count)
