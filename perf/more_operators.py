"""Cases of the operators of a decode step over a latent cache held in 8 bits with a scale for each block of
tokens: the tables of a step from its requests' lengths, the append that writes the rows and their scales, the
attention that reads them, and beam search's selection with the reordering of the beams' slot tables.  `run`
computes them in elementary torch operations, or, where `own` is set, through this framework's entry points."""
import math
import random

import numpy as np
import torch

own = False

D, DV, DR = 576, 512, 64  # latent row, latent part (also the values), rotated part
SM_SCALE = 1.0 / math.sqrt(192.0)
ROPE_BASE = 10000.0
LARGEST = 448.0  # of the 8-bit codes


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one stream's next token over a short chat: latency
        dict(name="attend_1k", op="attend", batch=1, lo=1024, hi=1024, q_lo=1, q_hi=1, tree=False, heads=64, block=1, exact2=True, lens=1),
        # a decode step of 32 requests of uneven lengths, blocks of 64 tokens
        dict(name="attend_step", op="attend", batch=32, lo=2000, hi=60000, q_lo=1, q_hi=1, tree=False, heads=64, block=64, exact2=True, lens=2),
        # the same on one of eight ranks that share the heads, with four drafts each, scales that are no powers of two
        dict(name="attend_rank", op="attend", batch=64, lo=1000, hi=32768, q_lo=4, q_hi=4, tree=False, heads=8, block=16, exact2=False, lens=3),
        # eight draft trees of ragged widths, 16 heads
        dict(name="attend_tree", op="attend", batch=8, lo=9001, hi=16411, q_lo=40, q_hi=64, tree=True, heads=16, block=1, exact2=True, lens=4),
        # a very long document, a chain of drafts
        dict(name="attend_185k", op="attend", batch=1, lo=185000, hi=185000, q_lo=4, q_hi=4, tree=False, heads=64, block=128, exact2=True, lens=5),
        # a step of 32 requests with 4 drafts each, padded to a fixed size, blocks partly filled
        dict(name="write_step", op="write", seqs=32, new_lo=4, new_hi=4, pad=16, heads=64, block=64, interleaved=True, context=131072, lens=6),
        # four prompts' rows, an odd count, halves rotated
        dict(name="write_prompt", op="write", seqs=4, new_lo=3001, new_hi=4999, pad=0, heads=16, block=64, interleaved=False, context=32768, lens=7),
        # the tables of a step of 32 requests, slot by slot
        dict(name="tables_step", op="tables", batch=32, lo=500, hi=30000, new_lo=1, new_hi=4, block=1, lens=8),
        # of many long requests in blocks
        dict(name="tables_many", op="tables", batch=256, lo=4000, hi=65536, new_lo=1, new_hi=16, block=64, lens=9),
        # one request with four beams: latency
        dict(name="beam_one", op="beam", requests=1, beams=4, keep=4, vocab=32000, fp32=False, masked=False, done=0.0, length=500),
        # a batch of requests with eight beams each
        dict(name="beam_step", op="beam", requests=64, beams=8, keep=8, vocab=131072, fp32=False, masked=False, done=0.1, length=4000),
        # few requests with many beams, twice as many kept, float logits of an odd vocabulary under a grammar
        dict(name="beam_wide", op="beam", requests=9, beams=15, keep=30, vocab=151001, fp32=True, masked=True, done=0.1, length=16001),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "tables", "beam"])
    if op == "attend":
        heads = rng.choice([8, 16, 24, 64, 128])
        q_hi = rng.choice([1, 1, 2, 4, 5, 16, 64])
        hi = _log_int(rng, 1, 185000)
        batch = _log_int(rng, 1, max(1, min(128, int(4e7 / (heads * q_hi * (hi + q_hi))), 600000 // (hi + q_hi))))
        return dict(op=op, batch=batch, lo=rng.randint(max(1, hi // 8), hi), hi=hi, q_lo=rng.randint(0, q_hi) if batch > 1 else q_hi, q_hi=q_hi,
                    tree=rng.random() < 0.3, heads=heads, block=rng.choice([1, 1, 16, 32, 64, 128]), exact2=rng.random() < 0.7,
                    lens=rng.randrange(1 << 30))
    if op == "write":
        hi = _log_int(rng, 1, 4999)
        seqs = _log_int(rng, 1, max(1, min(256, 16000 // hi)))
        return dict(op=op, seqs=seqs, new_lo=rng.randint(1, hi), new_hi=hi, pad=rng.randrange(0, 20), heads=rng.choice([0, 1, 8, 16, 24, 64]),
                    block=rng.choice([1, 8, 16, 64, 128]), interleaved=rng.random() < 0.5, context=rng.randint(hi + 200, 200000),
                    lens=rng.randrange(1 << 30))
    if op == "tables":
        hi = _log_int(rng, 1, 65536)
        batch = _log_int(rng, 1, max(1, min(512, 256 * 30000 // (hi + 100))))
        new_hi = _log_int(rng, 1, 64)
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, new_lo=rng.randint(0, new_hi), new_hi=new_hi,
                    block=rng.choice([1, 2, 16, 64, 128]), lens=rng.randrange(1 << 30))
    vocab = _log_int(rng, 50, 262144)
    beams = rng.randint(1, 16)
    requests = _log_int(rng, 1, max(1, min(128, 60000000 // (vocab * beams))))
    return dict(op="beam", requests=requests, beams=beams, keep=min(rng.choice([beams, 2 * beams]), 32), vocab=vocab,
                fp32=rng.random() < 0.5 and requests * beams * vocab <= 1 << 25, masked=rng.random() < 0.5, done=rng.choice([0.0, 0.2]),
                length=_log_int(rng, 1, 20000))


def _spread(case, n, lo, hi, salt):
    """n whole numbers between lo and hi, evenly over the logarithm, hi among them: of the case alone."""
    r = random.Random(case["lens"] * 7 + salt)
    v = [min(hi, max(lo, int(round(math.exp(r.uniform(math.log(lo + 1), math.log(hi + 1))) - 1)))) for _ in range(n)]
    v[r.randrange(n)] = hi
    return v


def _lengths(case):
    """Key counts (drafts included) and draft counts of an attend case's sequences."""
    nq = _spread(case, case["batch"], case["q_lo"], case["q_hi"], 1)
    nk = [p + q for p, q in zip(_spread(case, case["batch"], case["lo"], case["hi"], 2), nq)]
    return nk, nq


def _parents(case, nq):
    """Parents of the drafts: a random tree's (depth at most 8), or a chain's; and their depths."""
    r = random.Random(case["lens"] + 1)
    all_parents, all_depths = [], []
    for n in nq:
        depth, parent = [], []
        for i in range(n):
            p = i - 1
            if case["tree"] and i > 0:
                p = r.choice([j for j in range(i) if depth[j] < 7])
            depth.append(depth[p] + 1 if p >= 0 else 0)
            parent.append(p)
        all_parents += parent
        all_depths += depth
    return all_parents, all_depths


def _indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def _blocks(n, block):
    return [-(-x // block) for x in n]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 29)
    s = {"attend": _prepare_attend, "write": _prepare_write, "tables": _prepare_tables, "beam": _prepare_beam}[case["op"]](case, g)
    s["op"] = case["op"]
    if own:
        s["call"] = {"attend": _own_attend, "write": _own_write, "tables": _own_tables, "beam": _own_beam}[case["op"]](s)
    return s


def _normal(g, *shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def _codes(g, blocks, block, exact2):
    """Rows of blocks whose sizes differ, as codes with the scale of their block."""
    x = torch.randn((blocks, block * D), generator=g, device="cuda") * (0.5 * torch.exp(0.4 * torch.randn((blocks, 1), generator=g, device="cuda")))
    scale = x.abs().amax(1) / LARGEST
    if exact2:
        scale = torch.exp2(torch.ceil(torch.log2(scale)))
    pool = (x / scale[:, None]).clamp(-LARGEST, LARGEST).to(torch.float8_e4m3fn).view(torch.uint8).view(blocks * block, D)
    return pool, scale


def _slots(blocks_of, n, block):
    """Slots of a sequence's n rows in its blocks (on the GPU)."""
    p = torch.arange(n, device="cuda")
    return blocks_of[p // block] * block + p % block


def _prepare_attend(case, g):
    nk, nq = _lengths(case)
    B, H, bt = case["batch"], case["heads"], case["block"]
    nb = _blocks(nk, bt)
    total = sum(nb) + 3
    pool, scales = _codes(g, total, bt, case["exact2"])
    perm = torch.randperm(total, generator=g, device="cuda")
    first = _indptr(nb)
    kv = torch.cat([_slots(perm[int(first[b]):int(first[b + 1])], nk[b], bt) for b in range(B)]).to(torch.int32)
    T = sum(nq)
    kv_h, qo_h = _indptr(nk), _indptr(nq)
    parent = torch.tensor(_parents(case, nq)[0], dtype=torch.int32).cuda() if case["tree"] else None
    return dict(q=_normal(g, T, H, D, sigma=1.5), pool=pool, scales=scales, kv_indices=kv, kv_h=kv_h, qo_h=qo_h, kv_indptr=torch.from_numpy(kv_h).cuda(),
                qo_indptr=torch.from_numpy(qo_h).cuda(), parent=parent, block=bt,
                out=torch.empty((T, H, DV), dtype=torch.bfloat16, device="cuda"), lse=torch.empty((T, H), dtype=torch.float32, device="cuda"))


def _rope_table(rows):
    """cos | sin of position x frequency, [rows, 64] fp32, angles in 64 bits."""
    freq = ROPE_BASE ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _write_plan(case):
    """Per sequence: its new tokens and where in its blocks they begin (prompts begin anywhere in a chat)."""
    new = _spread(case, case["seqs"], case["new_lo"], case["new_hi"], 3)
    r = random.Random(case["lens"] + 5)
    begin = [r.choice([0, r.randint(0, 150)]) for _ in new]
    return new, begin


def _prepare_write(case, g):
    new, begin = _write_plan(case)
    bt, H, pad = case["block"], case["heads"], case["pad"]
    nb = _blocks([n + b for n, b in zip(new, begin)], bt)
    total = sum(nb) + 3
    pool, scales = _codes(g, total, bt, True)
    perm = torch.randperm(total, generator=g, device="cuda")
    first = _indptr(nb)
    slots = torch.cat([_slots(perm[int(first[i]):int(first[i + 1])], b + n, bt)[b:] for i, (n, b) in enumerate(zip(new, begin))])
    positions = torch.cat([torch.arange(b, b + n, device="cuda") for n, b in zip(new, begin)])
    T = sum(new) + pad
    kv = torch.randn((T, D), generator=g, device="cuda") * (0.5 * torch.exp(0.4 * torch.randn((T, 1), generator=g, device="cuda")))
    s = dict(kv=kv.to(torch.bfloat16), slots=torch.full((T,), -1, dtype=torch.int32, device="cuda"), positions=torch.zeros((T,), dtype=torch.int32, device="cuda"),
             table=_rope_table(case["context"]), pool=pool, scales=scales, block=bt, interleaved=case["interleaved"], q=None, q_rope=None)
    s["slots"][:T - pad] = slots
    s["positions"][:T - pad] = positions
    s["latent"], s["k_rope"] = s["kv"][:, :DV], s["kv"][:, DV:]
    if H:
        s["q"] = _normal(g, T, H, D)
        s["q_rope"] = _normal(g, T, H, DR)
    return s


def _prepare_tables(case, g):
    B, bt = case["batch"], case["block"]
    cached = _spread(case, B, case["lo"], case["hi"], 4)
    new = _spread(case, B, case["new_lo"], case["new_hi"], 5)
    have, need = _blocks(cached, bt), _blocks([c + n for c, n in zip(cached, new)], bt)
    width = max(need) + 3
    total = sum(need) + 40
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    first = _indptr(have)
    for b in range(B):
        table[b, :have[b]] = perm[int(first[b]):int(first[b + 1])]
    free = perm[int(first[-1]):].contiguous()
    N, T = sum(cached) + sum(new), sum(new)
    ints = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    return dict(cached=torch.tensor(cached, dtype=torch.int32).cuda(), new=torch.tensor(new, dtype=torch.int32).cuda(), table=table, free=free, block=bt,
                count=torch.tensor([free.numel()], dtype=torch.int32).cuda(), left=ints(1), scratch=ints(1), kv_indptr=ints(B + 1), qo_indptr=ints(B + 1),
                # room for a fixed size: some entries stay unused
                kv_indices=ints(N + 100), positions=ints(T + 10), slots=ints(T + 10))


def _prepare_beam(case, g):
    R, W, V, K = case["requests"], case["beams"], case["vocab"], case["keep"]
    # a language model's logits: a broad bulk, and a few tokens well above it
    x = torch.randn((R * W, V), generator=g, device="cuda") * 2.0
    likely = torch.randint(0, V, (R * W, 24), generator=g, device="cuda")
    x.scatter_add_(1, likely, 4.0 + 9.0 * torch.rand((R * W, 24), generator=g, device="cuda"))
    if case["masked"]:  # tokens that a grammar forbids
        x.masked_fill_(torch.rand((R * W, V), generator=g, device="cuda") < 0.3, -math.inf)
    L = case["length"]
    table = torch.randint(0, 1 << 20, (R * W, L + 64), generator=g, device="cuda", dtype=torch.int32)
    length = torch.randint(max(1, L // 2), L + 1, (R, 1), generator=g, device="cuda", dtype=torch.int32).repeat(1, W).reshape(-1).contiguous()
    return dict(logits=x if case["fp32"] else x.to(torch.bfloat16), score=-20.0 - 6.0 * torch.rand((R * W,), generator=g, device="cuda"), beams=W, keep=K,
                done=(torch.rand((R * W,), generator=g, device="cuda") < case["done"]).to(torch.int32), pad=min(2, V - 1), table=table, length=length,
                parent=torch.zeros((R, K), dtype=torch.int32, device="cuda"), token=torch.zeros((R, K), dtype=torch.int32, device="cuda"),
                new_score=torch.zeros((R, K), device="cuda"), new_table=torch.zeros((R * K, L + 64), dtype=torch.int32, device="cuda"),
                new_length=torch.zeros((R * K,), dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ the framework's calls
def _own_attend(s):
    from speculative_decoding_mla_gb300 import binding
    T, H, _ = s["q"].shape
    n = binding.verify_attn_mla_scaled_workspace_size(s["kv_indptr"].numel() - 1, H, T, s["kv_indices"].numel())
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return binding.prepare_verify_attn_mla_scaled(s["q"], s["pool"], s["scales"], s["kv_indptr"], s["kv_indices"], s["qo_indptr"], s["out"], s["lse"],
                                                  s["workspace"], SM_SCALE, block_tokens=s["block"], parent=s["parent"])


def _own_write(s):
    from speculative_decoding_mla_gb300 import binding
    return binding.prepare_verify_attn_mla_append_scaled(s["latent"], s["k_rope"], s["positions"], s["slots"], s["table"], s["pool"], s["scales"],
                                                         block_tokens=s["block"], q_rope=s["q_rope"], q=s["q"], interleaved=s["interleaved"])


def _own_tables(s):
    from speculative_decoding_mla_gb300 import binding
    return binding.prepare_verify_attn_mla_step_tables(s["cached"], s["new"], s["table"], s["free"], s["count"], s["left"], s["scratch"], s["kv_indptr"],
                                                       s["qo_indptr"], s["kv_indices"], s["positions"], s["slots"], block_tokens=s["block"])


def _own_beam(s):
    from speculative_decoding_mla_gb300 import binding
    n = binding.verify_attn_mla_beam_select_workspace_size(s["logits"].shape[0], s["logits"].shape[1], s["keep"])
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    select = binding.prepare_verify_attn_mla_beam_select(s["logits"], s["score"], s["parent"], s["token"], s["new_score"], s["workspace"],
                                                         beams=s["beams"], finished=s["done"], pad_token=s["pad"])
    reorder = binding.prepare_verify_attn_mla_beam_reorder(s["table"], s["new_table"], s["parent"], beams=s["beams"], length=s["length"],
                                                           new_length=s["new_length"])

    def call():
        select()
        reorder()
    return call


def run(state):
    op = state["op"]
    if own:
        state["call"]()
    else:
        {"attend": _plain_attend, "write": _plain_write, "tables": _plain_tables, "beam": _plain_beam}[op](state)
    if op == "attend":
        return {"out": state["out"], "lse": state["lse"]}
    if op == "write":
        r = {"pool": state["pool"].view(torch.float8_e4m3fn), "scales": state["scales"]}
        return dict(r, q=state["q"]) if state["q"] is not None else r
    if op == "tables":
        return {k: state[k] for k in ("table", "left", "kv_indptr", "qo_indptr", "kv_indices", "positions", "slots")}
    return {k: state[k] for k in ("parent", "token", "new_score", "new_table", "new_length")}


# ------------------------------------------------------------------ plain forms
def _plain_attend(s):
    q = s["q"].float()
    T, H, _ = q.shape
    for b in range(len(s["kv_h"]) - 1):
        t0, t1, k0, k1 = int(s["qo_h"][b]), int(s["qo_h"][b + 1]), int(s["kv_h"][b]), int(s["kv_h"][b + 1])
        n, m = k1 - k0, t1 - t0
        if m == 0:
            continue
        slot = s["kv_indices"][k0:k1].long()
        rows = s["pool"][slot].view(torch.float8_e4m3fn).float() * s["scales"][slot // s["block"], None]
        # drafts that draft i sees: itself and the chain of its parents (all earlier ones, without a tree)
        i = torch.arange(m, device="cuda")
        if s["parent"] is None:
            sees = i[:, None] >= i[None, :]
        else:
            near = torch.eye(m, device="cuda") + (s["parent"][t0:t1].long()[:, None] == i).float()
            for _ in range(6):
                near = ((near @ near) > 0).float()
            sees = near > 0
        score = (q[t0:t1].reshape(m * H, D) @ rows.t()).reshape(m, H, n) * SM_SCALE
        score[:, :, n - m:].masked_fill_(~sees[:, None, :], -math.inf)
        top = score.amax(-1, keepdim=True)
        p = (score - top).exp_()
        total = p.sum(-1, keepdim=True)
        s["out"][t0:t1] = ((p.reshape(m * H, n) @ rows[:, :DV]).reshape(m, H, DV) / total).to(torch.bfloat16)
        s["lse"][t0:t1] = (top + total.log())[..., 0]


def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :DR // 2], x[..., DR // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _power(amax):
    """The smallest power of two whose multiple by the largest code is no less (fp32, exact)."""
    m, e = torch.frexp(amax / 256.0)  # amax = 256 m 2^e, m in [1/2, 1); 448 = 256 x 1.75
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), torch.where(m > 0.875, e, e - 1)), torch.zeros_like(amax))


def _plain_write(s):
    bt = s["block"]
    keep = s["slots"] >= 0
    cs = s["table"][s["positions"].long()]
    cos, sin = cs[:, :DR // 2], cs[:, DR // 2:]
    row = torch.cat([s["latent"].float(), _rotate(s["k_rope"].float(), cos, sin, s["interleaved"])], 1)
    slot = s["slots"].long().clamp(min=0)
    block = slot // bt
    blocks = s["scales"].numel()
    # of each block: the largest value that comes, and the first row that comes
    most = torch.zeros(blocks, device="cuda").scatter_reduce(0, block, torch.where(keep, row.abs().amax(1), 0.0), "amax")
    begin = torch.full((blocks,), bt, device="cuda").scatter_reduce(0, block, torch.where(keep, slot % bt, bt), "amin")
    need, old = _power(most), s["scales"].clone()
    tiny = torch.full_like(need, 2.0 ** -100)
    scale = torch.where(begin < bt, torch.maximum(torch.where(begin == 0, tiny, old), torch.maximum(need, tiny)), old)
    # rows in front of those that come are coded again where their block's scale grew
    again = (torch.arange(bt, device="cuda") < begin[:, None]) & ((scale > old) & (begin < bt))[:, None]
    pool = s["pool"].view(torch.float8_e4m3fn).float().view(blocks, bt, D)
    pool = torch.where(again[..., None], pool * (old / scale)[:, None, None], pool).view(blocks * bt, D)
    # a padded token stands in as a copy of the first real one, so that nothing else is written
    at = torch.where(keep, torch.arange(keep.numel(), device="cuda"), keep.to(torch.int32).argmax())
    pool[slot[at]] = ((row / scale[block][:, None]).clamp(-LARGEST, LARGEST))[at]
    s["pool"].copy_(pool.to(torch.float8_e4m3fn).view(torch.uint8))
    s["scales"].copy_(scale)
    if s["q"] is not None:
        r = _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(torch.bfloat16)
        s["q"][..., DV:] = torch.where(keep[:, None, None], r, s["q"][..., DV:])


def _plain_tables(s):
    bt = s["block"]
    cached, new = s["cached"].long(), s["new"].long()
    B = cached.numel()
    n = cached + new
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    kv, qo = torch.cat([zero, n.cumsum(0)]), torch.cat([zero, new.cumsum(0)])
    have, need = (cached + bt - 1) // bt, (n + bt - 1) // bt
    taken = torch.cat([zero, (need - have).cumsum(0)])
    # the table's new entries: blocks from the end of the free list, in the order of the requests
    k = torch.arange(s["table"].shape[1], device="cuda")[None]
    at = s["count"].long() - 1 - (taken[:-1, None] + k - have[:, None])
    grown = (k >= have[:, None]) & (k < need[:, None])
    s["table"].copy_(torch.where(grown, s["free"][at.clamp(0, s["free"].numel() - 1)], s["table"]))
    s["left"].copy_(s["count"] - taken[-1:])
    s["kv_indptr"].copy_(kv)
    s["qo_indptr"].copy_(qo)
    j = torch.arange(s["kv_indices"].numel(), device="cuda")
    seq = torch.searchsorted(kv[1:].contiguous(), j, right=True).clamp(max=B - 1)
    p = j - kv[seq]
    slot = s["table"][seq, (p // bt).clamp(max=s["table"].shape[1] - 1)].long() * bt + p % bt
    s["kv_indices"].copy_(torch.where(j < kv[-1], slot, s["kv_indices"].long()))
    t = torch.arange(s["slots"].numel(), device="cuda")
    seq = torch.searchsorted(qo[1:].contiguous(), t, right=True).clamp(max=B - 1)
    p = t - qo[seq] + cached[seq]
    slot = s["table"][seq, (p // bt).clamp(max=s["table"].shape[1] - 1)].long() * bt + p % bt
    s["slots"].copy_(torch.where(t < qo[-1], slot, -1))
    s["positions"].copy_(torch.where(t < qo[-1], p, 0))


def _plain_beam(s):
    W, K = s["beams"], s["keep"]
    x = s["logits"].double()
    V = x.shape[1]
    R = x.shape[0] // W
    top = x.amax(1, keepdim=True)
    x -= top + (x - top).exp_().sum(1, keepdim=True).log()
    x += s["score"].double()[:, None]
    # a finished beam goes on as it is, by the padding token alone
    done = s["done"].bool()
    x = torch.where(done[:, None], -math.inf, x)
    x[:, s["pad"]] = torch.where(done, s["score"].double(), x[:, s["pad"]])
    best = x.view(R, W * V).sort(dim=1, descending=True, stable=True)  # ties: the lowest index first
    value, index = best.values[:, :K], best.indices[:, :K]
    if K > W * V:
        value = torch.cat([value, value.new_full((R, K - W * V), -math.inf)], 1)
        index = torch.cat([index, index.new_zeros((R, K - W * V))], 1)
    real = value > -math.inf
    s["parent"].copy_(torch.where(real, index // V, -1))
    s["token"].copy_(torch.where(real, index % V, -1))
    s["new_score"].copy_(value)
    parent = s["parent"].long()
    source = (torch.arange(R, device="cuda")[:, None] * W + parent.clamp(min=0)).view(-1)
    s["new_length"].copy_(torch.where(parent.view(-1) >= 0, s["length"][source], 0))
    use = torch.arange(s["table"].shape[1], device="cuda")[None] < s["new_length"][:, None]
    s["new_table"].copy_(torch.where(use, s["table"][source], s["new_table"]))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "attend":
        nk, nq = _lengths(case)
        H, T = case["heads"], sum(nq)
        depth = _parents(case, nq)[1]
        keys = sum(q * (n - q) for n, q in zip(nk, nq)) + sum(d + 1 for d in depth)
        rows = sum(n for n, q in zip(nk, nq) if q)
        return {"bytes": rows * (D + 4) + 4 * sum(_blocks(nk, case["block"])) + T * H * (2 * D + 2 * DV + 4), "flops": 2 * (D + DV) * H * keys}
    if case["op"] == "write":
        new, begin = _write_plan(case)
        T, H, bt = sum(new), case["heads"], case["block"]
        blocks = sum((b + n - 1) // bt - b // bt + 1 for n, b in zip(new, begin))
        # (a scale that has grown stays: appending the same rows again leaves the cache as it is)
        return {"bytes": T * (2 * D + D + 4 * DR + 8 + 2 * 2 * DR * H) + 8 * blocks, "flops": T * (3 * DR * (1 + H) + 2 * D)}
    if case["op"] == "tables":
        cached, new = _spread(case, case["batch"], case["lo"], case["hi"], 4), _spread(case, case["batch"], case["new_lo"], case["new_hi"], 5)
        n = [c + m for c, m in zip(cached, new)]
        return {"bytes": 4 * sum(n) + 8 * sum(new) + 4 * sum(_blocks(n, case["block"])) + 16 * case["batch"], "flops": 4 * sum(n)}
    rows = case["requests"] * case["beams"]
    kept = case["requests"] * case["keep"]
    return {"bytes": rows * case["vocab"] * (4 if case["fp32"] else 2) + kept * (12 + 8 * (3 * case["length"] // 4)), "flops": 4 * rows * case["vocab"]}


# ------------------------------------------------------------------ 64-bit results from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"attend": _exact_attend, "write": _exact_write, "tables": _exact_tables, "beam": _exact_beam}[case["op"]](case, s)


def _exact_attend(case, s):
    nk, nq = _lengths(case)
    H = case["heads"]
    if 2 * (D + DV) * H * sum(q * n for n, q in zip(nk, nq)) > 4e12:
        return None
    parents = _parents(case, nq)[0]
    lut = torch.arange(256, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    out, lse = [], []
    for b, (n, q) in enumerate(zip(nk, nq)):
        t0, k0 = int(s["qo_h"][b]), int(s["kv_h"][b])
        slot = s["kv_indices"][k0:k0 + n].long()
        rows = lut[s["pool"][slot].int()] * s["scales"].double()[torch.div(slot, case["block"], rounding_mode="floor")][:, None]
        z = torch.einsum("thd,nd->thn", s["q"][t0:t0 + q].double(), rows) * SM_SCALE
        for i in range(q):
            seen, at = [], i
            while at >= 0:
                seen.append(n - q + at)
                at = parents[t0 + at] if case["tree"] else at - 1
            z_i = torch.cat([z[i, :, :n - q], z[i][:, seen]], 1)
            use = torch.cat([rows[:n - q], rows[seen]])[:, :DV]
            l = torch.logsumexp(z_i, 1)
            out.append((z_i - l[:, None]).exp() @ use)
            lse.append(l)
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_write(case, s):
    bt = case["block"]
    new, begin = _write_plan(case)
    T = sum(new)
    angles = s["table"][s["positions"][:T].long()].double()
    c = torch.complex(angles[:, :32], angles[:, 32:])

    def turn(x, c):
        x = x.double()
        z = (torch.complex(x[..., 0::2], x[..., 1::2]) if case["interleaved"] else torch.complex(x[..., :32], x[..., 32:])) * c
        return torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)

    rows = torch.cat([s["latent"][:T].double(), turn(s["k_rope"][:T], c)], 1)
    pool = s["pool"].view(torch.float8_e4m3fn).double()
    scales = s["scales"].double()
    slots = s["slots"][:T].cpu().numpy()
    most = rows.abs().amax(1).cpu().numpy()
    old = scales.cpu().numpy()
    t = 0
    runs = []
    while t < T:
        e = t + 1
        while e < T and slots[e] // bt == slots[t] // bt:
            e += 1
        runs.append((t, e))
        t = e
    to = np.empty(T)
    for t, e in runs:
        block, at = slots[t] // bt, slots[t] % bt
        k = math.ceil(math.log2(most[t:e].max() / LARGEST)) if most[t:e].max() > 0 else -100
        while LARGEST * 2.0 ** (k - 1) >= most[t:e].max() and k > -100:
            k -= 1
        now = 2.0 ** max(k, -100)
        if at:
            now = max(now, old[block])
            if now > old[block]:
                pool[block * bt:block * bt + at] *= old[block] / now
        scales[block] = now
        to[t:e] = now
    pool[s["slots"][:T].long()] = (rows / torch.from_numpy(to).cuda()[:, None]).clamp(-LARGEST, LARGEST)
    r = {"pool": pool, "scales": scales}
    if s["q"] is not None:
        r["q"] = s["q"].double()
        r["q"][:T, :, DV:] = turn(s["q_rope"][:T], c[:, None])
    return r


def _exact_tables(case, s):
    host = {k: s[k].cpu().numpy().copy() for k in ("cached", "new", "table", "free", "count", "kv_indices")}
    bt, left = case["block"], int(host["count"][0])
    positions, slots = np.zeros(s["positions"].numel(), np.int32), np.full(s["slots"].numel(), -1, np.int32)
    kv, qo = [0], [0]
    for b, (c, m) in enumerate(zip(host["cached"].tolist(), host["new"].tolist())):
        for k in range(-(-c // bt), -(-(c + m) // bt)):
            left -= 1
            host["table"][b, k] = host["free"][left]
        p = np.arange(c + m)
        slot = host["table"][b, p // bt] * bt + p % bt
        host["kv_indices"][kv[-1]:kv[-1] + c + m] = slot
        positions[qo[-1]:qo[-1] + m] = p[c:]
        slots[qo[-1]:qo[-1] + m] = slot[c:]
        kv.append(kv[-1] + c + m)
        qo.append(qo[-1] + m)
    ints = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32)  # noqa: E731
    return {"table": ints(host["table"]), "left": ints([left]), "kv_indptr": ints(kv), "qo_indptr": ints(qo), "kv_indices": ints(host["kv_indices"]),
            "positions": ints(positions), "slots": ints(slots)}


def _exact_beam(case, s):
    R, W, V, K = case["requests"], case["beams"], case["vocab"], case["keep"]
    if R * W * V > 80e6:
        return None
    score, done = s["score"].double().cpu().numpy(), s["done"].cpu().numpy()
    parent, token = np.full((R, K), -1, np.int32), np.full((R, K), -1, np.int32)
    value = np.full((R, K), -math.inf)
    table, new_table = s["table"].cpu().numpy(), s["new_table"].cpu().numpy().copy()
    length, new_length = s["length"].cpu().numpy(), np.zeros(R * K, np.int32)
    for r in range(R):
        found = []
        for w in range(W):
            a = r * W + w
            if done[a]:
                found.append((-score[a], w * V + s["pad"]))
                continue
            x = s["logits"][a].double().cpu().numpy()
            m = x.max()
            base = score[a] - m - math.log(np.exp(x - m).sum())
            least = np.partition(x, max(0, V - K))[max(0, V - K)]
            # every token that can be among the kept: ties at the border too, the lowest indices of them
            at = np.flatnonzero(x >= least)
            at = at[np.lexsort((at, -x[at]))][:K]
            found += [(-(base + x[v]), w * V + int(v)) for v in at if x[v] > -math.inf]
        for k, (v, i) in enumerate(sorted(found)[:K]):
            parent[r, k], token[r, k], value[r, k] = i // V, i % V, -v
            a = r * W + i // V
            new_length[r * K + k] = length[a]
            new_table[r * K + k, :length[a]] = table[a, :length[a]]
    return {"parent": torch.from_numpy(parent), "token": torch.from_numpy(token), "new_score": torch.from_numpy(value),
            "new_table": torch.from_numpy(new_table), "new_length": torch.from_numpy(new_length)}
