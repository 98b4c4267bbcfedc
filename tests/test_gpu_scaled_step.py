"""Decode steps over the scaled pool of the pieces as they would be used together: the tables from the lengths, the
append with its scales, the attention, a stand-in output projection, and the selection of beams with the reordering of
their slot tables, or the acceptance of drafts.  Each stage is checked against its plain form on the values that it
really got; captured steps give the eager ones' bits.  Tolerances as derived in the stages' own tests."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_beam import check as check_beams
from tests.test_gpu_beam import expected as expected_beams
from tests.test_gpu_scaled import D, DV, SM
from tests.test_gpu_scaled import check as check_attention

pytestmark = pytest.mark.gpu
DR = D - DV


@pytest.fixture(scope="module")
def B():
    from speculative_decoding_mla_gb300 import binding
    return binding


def angles(rows):
    freq = 10000.0 ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    a = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([a.cos(), a.sin()], 1).float()


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32, device="cuda")


class Beams:
    """R requests of W beams: a table of slots each, prompts shared by a request's beams."""
    H, V, W, EOS = 16, 501, 4, 7

    def __init__(self, B, prompts):
        self.B, R, W = B, len(prompts), self.W
        self.R, T = R, R * W
        g = torch.Generator(device="cuda").manual_seed(4)
        r = lambda *s, k=1.0: (torch.randn(s, generator=g, device="cuda") * k).to(torch.bfloat16)  # noqa: E731
        self.slots_all, width = 700, max(prompts) + 40
        self.rows_of, self.q_of, self.turn_of = r(self.V, D, k=0.7), r(self.V, self.H, D), r(self.V, self.H, DR)
        self.head = r(self.H * DV, self.V, k=0.05)
        self.cos_sin = angles(1000)
        perm = torch.randperm(self.slots_all, generator=g, device="cuda").to(torch.int32)
        self.pool = torch.zeros((self.slots_all, D), dtype=torch.uint8, device="cuda")
        self.scales = torch.ones(self.slots_all, device="cuda")
        self.table, self.spare = torch.full((T, width), -1, dtype=torch.int32, device="cuda"), torch.full((T, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for k, n in enumerate(prompts):
            self.table[k * W:(k + 1) * W, :n] = perm[at:at + n]
            kv = r(n, D, k=0.7)
            B.verify_attn_mla_append_scaled(kv[:, :DV], kv[:, DV:], torch.arange(n, dtype=torch.int32, device="cuda"), perm[at:at + n].contiguous(),
                                            self.cos_sin, self.pool, self.scales)
            at += n
        self.free = perm[at:].contiguous()
        self.count = torch.tensor([self.free.numel()], dtype=torch.int32, device="cuda")
        self.cached = torch.tensor([n for n in prompts for _ in range(W)], dtype=torch.int32, device="cuda")
        self.one = torch.ones(T, dtype=torch.int32, device="cuda")
        self.token = torch.randint(0, self.V, (R, W), generator=g, device="cuda", dtype=torch.int32)
        self.score = torch.full((R, W), -math.inf, device="cuda")
        self.score[:, 0] = 0.0  # at first a request's beams are one
        self.done = i32(T)
        N = (sum(prompts) + 40 * R) * W
        self.scratch, self.status = i32(1), i32(2)
        self.kv_indptr, self.qo_indptr, self.kv_indices, self.positions, self.slots = i32(T + 1), i32(T + 1), i32(N), i32(T), i32(T)
        self.kv, self.q = torch.zeros((T, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, self.H, D), dtype=torch.bfloat16, device="cuda")
        self.turn, self.out = torch.zeros((T, self.H, DR), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, self.H, DV), dtype=torch.bfloat16, device="cuda")
        self.lse, self.logits = torch.zeros((T, self.H), device="cuda"), torch.zeros((T, self.V), dtype=torch.bfloat16, device="cuda")
        self.ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(T, self.H, T, N), dtype=torch.uint8, device="cuda")
        self.ws2 = torch.empty(B.verify_attn_mla_beam_select_workspace_size(T, self.V, W), dtype=torch.uint8, device="cuda")
        self.parent, self.new_token, self.new_score = i32(R, W), i32(R, W), torch.zeros((R, W), device="cuda")

    def attend(self, table):
        tok = self.token.view(-1).clamp(min=0).long()
        self.kv.copy_(self.rows_of[tok])
        self.q.copy_(self.q_of[tok])
        self.turn.copy_(self.turn_of[tok])
        self.B.verify_attn_mla_step_tables(self.cached, self.one, table, self.free, self.count, self.count, self.scratch, self.kv_indptr, self.qo_indptr,
                                           self.kv_indices, self.positions, self.slots, status_word=self.status)
        self.B.verify_attn_mla_append_scaled(self.kv[:, :DV], self.kv[:, DV:], self.positions, self.slots, self.cos_sin, self.pool, self.scales,
                                             q_rope=self.turn, q=self.q, status_word=self.status)
        self.B.verify_attn_mla_scaled(self.q, self.pool, self.scales, self.kv_indptr, self.kv_indices, self.qo_indptr, self.out, self.lse, self.ws, SM)
        torch.mm(self.out.view(-1, self.H * DV), self.head, out=self.logits)

    def choose(self, table, to):
        R, W = self.R, self.W
        self.B.verify_attn_mla_beam_select(self.logits, self.score.view(-1), self.parent, self.new_token, self.new_score, self.ws2, beams=W,
                                           finished=self.done, pad_token=0)
        length = self.cached + self.one
        self.B.verify_attn_mla_beam_reorder(table, to, self.parent, beams=W, length=length, new_length=self.cached, status_word=self.status)
        before = self.done.view(R, W).gather(1, self.parent.clamp(min=0).long())
        self.done.copy_((before.bool() | (self.new_token == self.EOS)).to(torch.int32).view(-1))
        self.token.copy_(self.new_token)
        self.score.copy_(self.new_score)

    def two_steps(self):
        for table, to in ((self.table, self.spare), (self.spare, self.table)):
            self.attend(table)
            self.choose(table, to)

    def state(self):
        return [t.clone() for t in (self.token, self.score, self.done, self.cached, self.table, self.count, self.pool, self.scales, self.out, self.lse,
                                    self.kv_indices, self.parent, self.status)]


def test_beam_search(B):
    b = Beams(B, [50, 1, 200])
    R, W, T = b.R, b.W, b.R * b.W
    histories = [b.table[k, :int(b.cached[k])].tolist() for k in range(T)]
    for step in range(6):
        table, to = (b.table, b.spare) if step % 2 == 0 else (b.spare, b.table)
        cached, count = b.cached.tolist(), int(b.count)
        b.attend(table)
        # tables: a fresh slot each, from the free list's end
        fresh = b.free[count - T:count].flip(0).tolist()
        for k in range(T):
            histories[k] = histories[k][:cached[k]] + [fresh[k]]
        assert b.kv_indptr.tolist() == np.concatenate([[0], np.cumsum([n + 1 for n in cached])]).tolist()
        assert b.kv_indices[:int(b.kv_indptr[-1])].tolist() == sum(histories, [])
        assert b.slots.tolist() == fresh and b.positions.tolist() == cached and int(b.count) == count - T
        c = dict(q=b.q, pool=b.pool, scales=b.scales, kv=b.kv_indices[:int(b.kv_indptr[-1])], block=1, nk=[n + 1 for n in cached], nq=[1] * T)
        check_attention(c, b.out, b.lse)
        want = expected_beams(b.logits, b.score.view(-1), W, W, b.done, 0)
        b.choose(table, to)
        check_beams([b.parent, b.new_token, b.new_score], want)
        parent = b.parent.view(-1).tolist()
        assert min(parent) >= 0
        histories = [list(histories[k // W * W + parent[k]]) for k in range(T)]
        assert b.cached.tolist() == [len(h) for h in histories]
        for k in range(T):
            assert to[k, :len(histories[k])].tolist() == histories[k]
    assert b.status.tolist() == [0, 0] and len({tuple(h) for h in histories}) > R


def test_beam_search_captured(B):
    eager, b = Beams(B, [50, 1, 200]), Beams(B, [50, 1, 200])
    for _ in range(3):
        eager.two_steps()
    start = [t.clone() for t in vars(b).values() if torch.is_tensor(t)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # (warm-up: the matrix product's workspace)
        torch.mm(b.out.view(T := b.R * b.W, -1), b.head, out=b.logits)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            b.two_steps()
    torch.cuda.current_stream().wait_stream(side)
    for t, v in zip([t for t in vars(b).values() if torch.is_tensor(t)], start):
        t.copy_(v)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert T == 12
    for got, want in zip(b.state(), eager.state()):
        assert torch.equal(got, want)


@pytest.mark.parametrize("block", [16, 128])
def test_drafts_that_are_rejected_are_written_over(B, block):
    """Chains of drafts behind growing caches: what is rejected stays in its slots until the next step's rows come."""
    g = torch.Generator(device="cuda").manual_seed(block)
    rng = np.random.default_rng(block)
    n, H, most = 5, 8, 6
    cached = np.array([0, 15, 16, 130, 257])
    width, blocks = 40, 200
    pool = torch.zeros((blocks * block, D), dtype=torch.uint8, device="cuda")
    scales = torch.ones(blocks, device="cuda")
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    count, scratch, status = torch.tensor([blocks], dtype=torch.int32, device="cuda"), i32(1), i32(2)
    cos_sin = angles(2000)
    history = [np.zeros((0, D)) for _ in range(n)]  # the true rows
    writes = [np.zeros(0, int) for _ in range(n)]    # calls that wrote to a row's block since it came
    lut = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    lengths = np.zeros(n, int)
    for step in range(5):
        added = cached if step == 0 else rng.integers(0, most, n)  # the prompts, then drafts
        if step:
            added[step % n] = most - 1
        T, N = int(added.sum()) + 3, int((lengths + added).sum()) + 7
        kv_indptr, qo_indptr, kv_indices, positions, slots = i32(n + 1), i32(n + 1), i32(N), i32(T), i32(T)
        B.verify_attn_mla_step_tables(torch.tensor(lengths, dtype=torch.int32).cuda(), torch.tensor(added, dtype=torch.int32).cuda(), table, free, count,
                                      count, scratch, kv_indptr, qo_indptr, kv_indices, positions, slots, block_tokens=block, status_word=status)
        kv = (torch.randn((T, D), generator=g, device="cuda") * (0.5 * torch.exp(torch.randn((T, 1), generator=g, device="cuda")))).to(torch.bfloat16)
        q = torch.randn((T, H, D), generator=g, device="cuda").to(torch.bfloat16)
        turn = torch.randn((T, H, DR), generator=g, device="cuda").to(torch.bfloat16)
        B.verify_attn_mla_append_scaled(kv[:, :DV], kv[:, DV:], positions, slots, cos_sin, pool, scales, block_tokens=block, q_rope=turn, q=q,
                                        status_word=status)
        assert status.tolist() == [0, 0]
        # rows as they stand against the true ones: each coding is off by half a step, and a call may code a block again
        z = torch.complex(*cos_sin[positions.long()].double().chunk(2, 1)) * torch.view_as_complex(kv[:, DV:].double().view(T, -1, 2))
        rows = torch.cat([kv[:, :DV].double(), torch.view_as_real(z).flatten(-2)], 1).cpu().numpy()
        at, index = 0, kv_indices.cpu().numpy()
        codes, held = pool.cpu().numpy(), scales.double().cpu().numpy()
        ki = 0
        for b in range(n):
            m = int(added[b])
            history[b] = np.concatenate([history[b][:lengths[b]], rows[at:at + m]])
            writes[b] = np.concatenate([writes[b][:lengths[b]], np.zeros(m, int)])
            if m:
                writes[b][lengths[b] // block * block:] += 1
            at += m
            total = lengths[b] + m
            s = index[ki:ki + total]
            ki += total
            scale = held[s // block][:, None]
            off = np.abs(lut[codes[s]] * scale - history[b])
            tol = writes[b][:, None] * (np.abs(history[b]) * 2.0 ** -4 * (1 + 2.0 ** -4) ** 5 + scale * 2.0 ** -10) + np.abs(history[b]) * 2.0 ** -20
            assert (off <= tol).all(), float((off / tol).max())
        if step:  # (a prompt of 257 tokens is no draft)
            out, lse = torch.full((T, H, DV), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, H), 3.0, device="cuda")
            ws = torch.empty(B.verify_attn_mla_scaled_workspace_size(n, H, T, N), dtype=torch.uint8, device="cuda")
            B.verify_attn_mla_scaled(q, pool, scales, kv_indptr, kv_indices, qo_indptr, out, lse, ws, SM, block_tokens=block)
            t = int(qo_indptr[-1])
            c = dict(q=q[:t], pool=pool, scales=scales, kv=kv_indices[:int(kv_indptr[-1])], block=block, nk=(lengths + added).tolist(), nq=added.tolist())
            check_attention(c, out, lse)
            assert bool((out[t:] == 3).all()) and bool((lse[t:] == 3).all())
            small = torch.empty(ws.numel() - 256, dtype=torch.uint8, device="cuda")
            with pytest.raises(RuntimeError):
                B.verify_attn_mla_scaled(q, pool, scales, kv_indptr, kv_indices, qo_indptr, out, lse, small, SM, block_tokens=block)
        accepted = added if step == 0 else np.minimum(added, rng.integers(0, most, n))
        lengths = lengths + accepted
    assert int(count) < blocks
