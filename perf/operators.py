"""Cases of three operators of a speculative decode step on a paged latent cache: the append that
writes a step's rows (with the position rotation), the verify attention of a batch that shares a
prefix, and the sampling of the target's tokens from the verified logits.  `run` computes them in
elementary torch operations, or, where `own` is set, through this framework's entry points."""
import math
import random

import numpy as np
import torch

own = False

D, DV, DR = 576, 512, 64  # latent row, latent part (also the values), rotated part
SM_SCALE = 1.0 / math.sqrt(192.0)
ROPE_BASE = 10000.0


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a single stream's next token: latency
        dict(name="append_one", op="append", tokens=1, pad=0, heads=64, fp8=False, interleaved=True, context=200000, slots=65600),
        # a decode step of 32 sequences with 4 drafts each, the batch padded to a fixed graph size
        dict(name="append_step", op="append", tokens=144, pad=16, heads=64, fp8=False, interleaved=True, context=131072, slots=65600),
        # a prompt's rows into an e4m3 pool, halves rotated, an odd count
        dict(name="append_prompt_e4m3", op="append", tokens=16001, pad=0, heads=16, fp8=True, interleaved=False, context=32768, slots=65600),
        # a long prompt with the queries of all heads
        dict(name="append_prompt", op="append", tokens=16384, pad=0, heads=64, fp8=False, interleaved=True, context=185000, slots=65600),
        # four short chats behind one instruction text, one draft each: latency
        dict(name="shared_1k", op="shared", batch=4, prefix=1024, own_lo=17, own_hi=300, q_lo=1, q_hi=1, tree=False, heads=64, fp8=False, lens=1),
        # a batch of agents behind one long tool description, four drafts each
        dict(name="shared_32k", op="shared", batch=32, prefix=32768, own_lo=100, own_hi=2000, q_lo=4, q_hi=4, tree=False, heads=64, fp8=False, lens=2),
        # eight draft trees behind a document, ragged widths, an odd prefix, an e4m3 pool
        dict(name="shared_tree_e4m3", op="shared", batch=8, prefix=16411, own_lo=300, own_hi=4000, q_lo=40, q_hi=64, tree=True, heads=64, fp8=True, lens=3),
        # questions about one very long document, one draft each
        dict(name="shared_185k", op="shared", batch=48, prefix=185000, own_lo=30, own_hi=500, q_lo=1, q_hi=1, tree=False, heads=64, fp8=False, lens=4),
        # one row after the prefix: latency
        dict(name="sample_one", op="sample", rows=1, vocab=32000, fp32=False, filters="all", masked=False),
        # a step's rows with per-request settings, float logits of an odd vocabulary
        dict(name="sample_mixed", op="sample", rows=128, vocab=151001, fp32=True, filters="all", masked=True),
        # nucleus sampling of a tree step's rows
        dict(name="sample_top_p", op="sample", rows=512, vocab=131072, fp32=False, filters="top_p", masked=False),
        # plain temperature sampling of as many rows
        dict(name="sample_plain", op="sample", rows=512, vocab=131072, fp32=False, filters="none", masked=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "shared", "sample"])
    if op == "append":
        tokens = _log_int(rng, 1, 16384)
        return dict(op=op, tokens=tokens, pad=rng.randrange(0, max(1, tokens // 4)), heads=rng.choice([0, 1, 8, 16, 24, 64]),
                    fp8=rng.random() < 0.5, interleaved=rng.random() < 0.5, context=_log_int(rng, 64, 200000),
                    slots=_log_int(rng, tokens + 1, 65600))
    if op == "shared":
        heads = rng.choice([8, 16, 64, 64, 128])
        prefix = _log_int(rng, 1, 185000)
        tree = rng.random() < 0.3
        q_hi = rng.choice([1, 1, 2, 4, 5, 8, 16, 64])
        # no more than about the largest listed case's 48 x 64 rows over its prefix
        batch = min(64, max(1, int(48 * 64 * 185000 / (heads * q_hi * (prefix + 2000)))))
        batch = _log_int(rng, 1, batch)
        own_lo = _log_int(rng, 1, 400)
        return dict(op=op, batch=batch, prefix=prefix, own_lo=own_lo, own_hi=own_lo + _log_int(rng, 1, 2000), q_lo=rng.randint(0, q_hi) if batch > 1 else q_hi,
                    q_hi=q_hi, tree=tree, heads=heads, fp8=rng.random() < 0.3, lens=rng.randrange(1 << 30))
    vocab = _log_int(rng, 50, 262144)
    rows = _log_int(rng, 1, max(1, min(1024, 512 * 131072 // vocab)))
    return dict(op=op, rows=rows, vocab=vocab, fp32=rng.random() < 0.5 and rows * vocab <= 1 << 25, filters=rng.choice(["none", "top_k", "top_p", "min_p", "all"]),
                masked=rng.random() < 0.5)


def _lengths(case):
    """Own key counts (drafts included) and draft counts of a shared case's sequences: of the case alone."""
    r = random.Random(case["lens"])
    nq = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    nq[r.randrange(case["batch"])] = case["q_hi"]
    nk = [q + r.randint(case["own_lo"], case["own_hi"]) - 1 for q in nq]
    return nk, nq


def _parents(case, nq):
    """Parents of the drafts: a random tree's (depth at most 8), or a chain's."""
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


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    s = {"append": _prepare_append, "shared": _prepare_shared, "sample": _prepare_sample}[case["op"]](case, g)
    s["op"] = case["op"]
    if own:
        s["call"] = {"append": _own_append, "shared": _own_shared, "sample": _own_sample}[case["op"]](s)
    return s


def _normal(g, *shape, sigma=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).to(torch.bfloat16)


def _rope_table(rows):
    """cos | sin of position x frequency, [rows, 64] fp32, angles in 64 bits."""
    freq = ROPE_BASE ** (-torch.arange(0, DR, 2, dtype=torch.float64, device="cuda") / DR)
    angle = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def _pool(g, slots, fp8):
    if not fp8:
        return _normal(g, slots, D, sigma=0.5)
    return (torch.randn((slots, D), generator=g, device="cuda") * (0.5 / 0.0125)).to(torch.float8_e4m3fn).view(torch.uint8)


def _prepare_append(case, g):
    T, H = case["tokens"], case["heads"]
    # the projections leave the latent and the rotated part of a token side by side, the heads' rotated part apart
    kv = _normal(g, T, D, sigma=0.5)
    slots = torch.randperm(case["slots"], generator=g, device="cuda")[:T].to(torch.int32)
    if case["pad"]:
        slots[T - case["pad"]:] = -1
    s = dict(kv=kv, latent=kv[:, :DV], k_rope=kv[:, DV:], slots=slots,
             positions=torch.randint(0, case["context"], (T,), generator=g, device="cuda", dtype=torch.int32),
             table=_rope_table(case["context"]), pool=_pool(g, case["slots"], case["fp8"]), interleaved=case["interleaved"],
             fp8=case["fp8"], scale=0.0125 if case["fp8"] else 0.0, scale_t=torch.tensor(0.0125, device="cuda"), q=None, q_rope=None)
    if H:
        s["q"] = _normal(g, T, H, D)
        s["q_rope"] = _normal(g, T, H, DR)
    return s


def _prepare_shared(case, g):
    B, P, H = case["batch"], case["prefix"], case["heads"]
    nk, nq = _lengths(case)
    kv_h = np.concatenate([[0], np.cumsum(nk)]).astype(np.int32)
    qo_h = np.concatenate([[0], np.cumsum(nq)]).astype(np.int32)
    N, T = int(kv_h[-1]), int(qo_h[-1])
    S = P + N + 64
    perm = torch.randperm(S, generator=g, device="cuda").to(torch.int32)
    parent = None
    if case["tree"]:
        parent = torch.tensor(_parents(case, nq)[0], dtype=torch.int32).cuda()
    return dict(q=_normal(g, T, H, D), pool=_pool(g, S, case["fp8"]), fp8=case["fp8"], scale=0.0125 if case["fp8"] else 0.0,
                shared=perm[:P].contiguous(), kv_indices=perm[P:P + N].contiguous(), kv_h=kv_h, qo_h=qo_h,
                kv_indptr=torch.from_numpy(kv_h).cuda(), qo_indptr=torch.from_numpy(qo_h).cuda(), parent=parent,
                out=torch.empty((T, H, DV), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((T, H), dtype=torch.float32, device="cuda"), n_max=int(max(nk)), q_max=int(max(nq)))


def _prepare_sample(case, g):
    R, V = case["rows"], case["vocab"]
    # a language model's logits: a broad bulk, and a few tokens well above it
    x = torch.randn((R, V), generator=g, device="cuda") * 2.0
    likely = torch.randint(0, V, (R, 24), generator=g, device="cuda")
    x.scatter_add_(1, likely, 4.0 + 9.0 * torch.rand((R, 24), generator=g, device="cuda"))
    if case["masked"]:  # tokens that a grammar forbids
        x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.3, -math.inf)
    rand = lambda lo, hi: lo + (hi - lo) * torch.rand((R,), generator=g, device="cuda")  # noqa: E731
    f = case["filters"]
    s = dict(logits=x if case["fp32"] else x.to(torch.bfloat16), u=torch.rand((R,), generator=g, device="cuda"),
             temperature=rand(0.5, 1.3), top_k=None, top_p=None, min_p=None, token=torch.empty((R,), dtype=torch.int32, device="cuda"))
    if f in ("top_k", "all"):
        s["top_k"] = torch.randint(1, 101, (R,), generator=g, device="cuda", dtype=torch.int32)
    if f in ("top_p", "all"):
        s["top_p"] = rand(0.7, 0.99)
    if f in ("min_p", "all"):
        s["min_p"] = rand(0.0, 0.1)
    if f == "all":  # each request has settings of its own: greedy, or a filter left off
        s["temperature"][rand(0, 1) < 0.2] = 0.0
        s["top_k"][rand(0, 1) < 0.3] = 0
        s["top_p"][rand(0, 1) < 0.3] = 1.0
        s["min_p"][rand(0, 1) < 0.3] = 0.0
    return s


# ------------------------------------------------------------------ the framework's calls
def _own_append(s):
    from speculative_decoding_mla_gb300 import binding
    return binding.prepare_verify_attn_mla_append(s["latent"], s["k_rope"], s["positions"], s["slots"], s["table"], s["pool"],
                                                  q_rope=s["q_rope"], q=s["q"], kv_scale=s["scale"], interleaved=s["interleaved"])


def _own_shared(s):
    from speculative_decoding_mla_gb300 import binding
    n = binding.verify_attn_mla_shared_workspace_size(s["shared"].numel(), s["qo_h"], s["kv_h"], s["q"].shape[1])
    s["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    return binding.prepare_verify_attn_mla_shared(s["q"], s["pool"], s["shared"], s["kv_indptr"], s["kv_indices"], s["qo_indptr"],
                                                  s["kv_h"], s["qo_h"], s["out"], s["lse"], s["workspace"], SM_SCALE,
                                                  kv_scale=s["scale"], parent=s["parent"])


def _own_sample(s):
    from speculative_decoding_mla_gb300 import binding
    return binding.prepare_verify_attn_mla_sample(s["logits"], s["u"], s["token"], temperature=s["temperature"], top_k=s["top_k"],
                                                  top_p=s["top_p"], min_p=s["min_p"])


def run(state):
    op = state["op"]
    if own:
        state["call"]()
    else:
        {"append": _plain_append, "shared": _plain_shared, "sample": _plain_sample}[op](state)
    if op == "append":
        pool = state["pool"].view(torch.float8_e4m3fn) if state["fp8"] else state["pool"]
        return {"pool": pool, "q": state["q"]} if state["q"] is not None else {"pool": pool}
    if op == "shared":
        return {"out": state["out"], "lse": state["lse"]}
    return {"token": state["token"]}


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :DR // 2], x[..., DR // 2:])
    a, b = a * cos - b * sin, a * sin + b * cos
    return torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)


def _plain_append(s):
    keep = s["slots"] >= 0
    # a padded token stands in as a copy of the first real one, so that nothing else is written
    at = torch.where(keep, torch.arange(keep.numel(), device="cuda"), keep.to(torch.int32).argmax())
    cs = s["table"][s["positions"].long()]
    cos, sin = cs[:, :DR // 2], cs[:, DR // 2:]
    row = torch.cat([s["latent"].float(), _rotate(s["k_rope"].float(), cos, sin, s["interleaved"])], 1)
    if s["fp8"]:
        row = (row / s["scale_t"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        row = row.to(torch.bfloat16)
    s["pool"][s["slots"].long()[at]] = row[at]
    if s["q"] is not None:
        r = _rotate(s["q_rope"].float(), cos[:, None], sin[:, None], s["interleaved"]).to(torch.bfloat16)
        s["q"][..., DV:] = torch.where(keep[:, None, None], r, s["q"][..., DV:])


def _rows(s, slots):
    """Pool rows in 32 bits; a code's value is its e4m3 value times the scale, rounded to bf16."""
    x = s["pool"][slots.long()]
    return (x.view(torch.float8_e4m3fn).float() * s["scale"]).to(torch.bfloat16).float() if s["fp8"] else x.float()


def _plain_shared(s):
    q = s["q"].float()
    T, H, _ = q.shape
    n_max, q_max = s["n_max"], s["q_max"]
    kv0, qo0 = s["kv_indptr"].long(), s["qo_indptr"].long()
    n, nq = (kv0[1:] - kv0[:-1])[:, None], (qo0[1:] - qo0[:-1])[:, None]
    B = n.shape[0]
    # each sequence's own rows and queries, padded to the longest
    j, i = torch.arange(n_max, device="cuda")[None], torch.arange(q_max, device="cuda")[None]
    own_rows = _rows(s, s["kv_indices"][(kv0[:-1, None] + j).clamp(max=max(0, s["kv_indices"].numel() - 1))])
    q_at = (qo0[:-1, None] + i).clamp(max=T - 1)
    # drafts that draft i sees: itself and the chain of its parents (of all earlier drafts, without a tree)
    if s["parent"] is None:
        sees = (i[0][:, None] >= i[0][None, :])[None].expand(B, q_max, q_max)
    else:
        up = torch.where(i < nq, s["parent"][q_at].long(), -1)
        near = torch.eye(q_max, device="cuda") + (up[..., None] == i[0]).float()
        twice = lambda m: ((m @ m) > 0).float()  # noqa: E731
        sees = twice(twice(twice(twice(twice(twice(near)))))) > 0
    prefix = (n - nq)[:, :, None]
    draft = (j[:, None] - prefix).clamp(0, q_max - 1).expand(B, q_max, n_max)
    visible = (j[:, None] < prefix) | ((j < n)[:, None] & torch.gather(sees, 2, draft))  # [B, q_max, n_max]
    so = (q[q_at].reshape(B, q_max * H, D) @ own_rows.transpose(1, 2)).reshape(B, q_max, H, n_max) * SM_SCALE
    so = so.masked_fill(~visible[:, :, None], -math.inf)
    seq = torch.searchsorted(qo0[1:].contiguous(), torch.arange(T, device="cuda"), right=True)
    at = (seq, torch.arange(T, device="cuda") - qo0[seq])
    rows = _rows(s, s["shared"])
    ss = (q.reshape(T * H, D) @ rows.t()).reshape(T, H, -1) * SM_SCALE
    m = torch.maximum(ss.amax(-1), so.amax(-1)[at])
    mp = torch.zeros((B, q_max, H), device="cuda").index_put(at, m)
    ps, po = (ss - m[..., None]).exp_(), (so - mp[..., None]).exp_()
    total = ps.sum(-1) + po.sum(-1)[at]
    o = (ps.reshape(T * H, -1) @ rows[:, :DV]).reshape(T, H, DV)
    o += (po.reshape(B, q_max * H, n_max) @ own_rows[..., :DV]).reshape(B, q_max, H, DV)[at]
    s["out"].copy_(o / total[..., None])
    s["lse"].copy_(m + total.log())


def _plain_sample(s):
    x = s["logits"].double()
    V = x.shape[1]
    t = s["temperature"].double()[:, None]
    greedy = t == 0
    order = x.sort(dim=1, descending=True, stable=True)  # ties: the lowest index first
    w = torch.where(greedy, (order.values == order.values[:, :1]).double(), ((order.values - order.values[:, :1]) / torch.where(greedy, 1.0, t)).exp())
    place = torch.arange(V, device="cuda")[None]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        w = w.masked_fill((k > 0) & (place >= k), 0.0)
    most = w[:, :1]
    mass = w.cumsum(1)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cat([torch.zeros_like(most), mass[:, :-1]], 1)
        w = w.masked_fill((p < 1) & (before >= p * mass[:, -1:]), 0.0)
    if s["min_p"] is not None:
        w = w.masked_fill(w < s["min_p"].double()[:, None] * most, 0.0)
    w = w.masked_fill(greedy & (place > 0), 0.0)
    kept = torch.zeros_like(w).scatter_(1, order.indices, w).cumsum(1)  # in the order of the tokens
    past = (kept <= s["u"].double()[:, None] * kept[:, -1:]).sum(1)
    last = (kept < kept[:, -1:]).sum(1)
    s["token"].copy_(torch.minimum(past, last))


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "append":
        T = case["tokens"] - case["pad"]
        H = case["heads"]
        row = D if case["fp8"] else 2 * D
        return {"bytes": T * (2 * D + row + 4 * DR + 8 + 2 * 2 * DR * H), "flops": T * (3 * DR * (1 + H) + (D if case["fp8"] else 0))}
    if case["op"] == "shared":
        nk, nq = _lengths(case)
        H, P, T = case["heads"], case["prefix"], sum(nq)
        depth = _parents(case, nq)[1]
        keys = sum(q * (P + n - q) for n, q in zip(nk, nq)) + sum(d + 1 for d in depth)
        rows = P + sum(n for n, q in zip(nk, nq) if q)
        return {"bytes": rows * ((D if case["fp8"] else 2 * D) + 4) + T * H * (2 * D + 2 * DV + 4), "flops": 2 * (D + DV) * H * keys}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * (4 if case["fp32"] else 2) + 24 * case["rows"], "flops": 4 * n}


# ------------------------------------------------------------------ 64-bit results from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "shared": _exact_shared, "sample": _exact_sample}[case["op"]](case, s)


def _turn(x, angles, interleaved):
    """Pairs as complex numbers, turned by the table's (cos, sin)."""
    c = torch.complex(angles[..., :32].double(), angles[..., 32:].double())
    x = x.double()
    z = torch.complex(x[..., 0::2], x[..., 1::2]) if interleaved else torch.complex(x[..., :32], x[..., 32:])
    z = z * c
    return torch.view_as_real(z).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)


def _exact_append(case, s):
    if case["fp8"]:  # the values that the codes stand for, in units of the scale
        pool = s["pool"].view(torch.float8_e4m3fn).double()
    else:
        pool = s["pool"].double()
    n = case["tokens"] - case["pad"]
    angles = s["table"][s["positions"][:n].long()]
    rows = torch.cat([s["latent"][:n].double(), _turn(s["k_rope"][:n], angles, case["interleaved"])], 1)
    pool[s["slots"][:n].long()] = (rows / float(s["scale_t"])).clamp(-448, 448) if case["fp8"] else rows
    if s["q"] is None:
        return {"pool": pool}
    q = s["q"].double()
    q[:n, :, DV:] = _turn(s["q_rope"][:n], angles[:, None], case["interleaved"])
    return {"pool": pool, "q": q}


def _exact_shared(case, s):
    nk, nq = _lengths(case)
    keys = case["heads"] * sum(q * (case["prefix"] + n) for n, q in zip(nk, nq))
    if keys * 2 * (D + DV) > 6e12:
        return None
    parents = _parents(case, nq)[0]
    pool = s["pool"]
    if case["fp8"]:
        pool = (pool.view(torch.float8_e4m3fn).float() * s["scale"]).to(torch.bfloat16)
    out, lse = [], []
    for b, (n, q) in enumerate(zip(nk, nq)):
        t0, k0 = int(s["qo_h"][b]), int(s["kv_h"][b])
        rows = pool[torch.cat([s["shared"], s["kv_indices"][k0:k0 + n]]).long()].double()
        first = rows.shape[0] - q
        for i in range(q):
            seen, at = [], i
            while at >= 0:
                seen.append(at)
                at = parents[t0 + at] if case["tree"] else at - 1
            use = torch.cat([rows[:first], rows[[first + k for k in seen]]])
            z = (s["q"][t0 + i].double() @ use.t()) * SM_SCALE
            l = torch.logsumexp(z, 1)
            out.append((z - l[:, None]).exp() @ use[:, :DV])
            lse.append(l)
    return {"out": torch.stack(out), "lse": torch.stack(lse)}


def _exact_sample(case, s):
    if case["rows"] * case["vocab"] > 70e6:
        return None
    host = lambda k: None if s[k] is None else s[k].double().cpu().numpy()  # noqa: E731
    x, u, temp, top_k, top_p, min_p = (host(k) for k in ("logits", "u", "temperature", "top_k", "top_p", "min_p"))
    token = np.zeros(case["rows"], np.int32)
    for r in range(case["rows"]):
        if temp[r] == 0:
            token[r] = int(np.argmax(x[r]))
            continue
        w = np.exp((x[r] - x[r].max()) / temp[r])
        keep = np.ones(x.shape[1], bool)
        cut = top_k is not None and 0 < top_k[r] < x.shape[1]
        nucleus = top_p is not None and top_p[r] < 1
        if cut or nucleus:
            order = np.argsort(-x[r], kind="stable")
            if cut:
                order, rest = order[:int(top_k[r])], order[int(top_k[r]):]
                keep[rest] = False
            if nucleus:
                mass = np.cumsum(w[order])
                keep[order[1 + int(np.searchsorted(mass, top_p[r] * mass[-1], side="left")):]] = False
        if min_p is not None:
            keep &= w >= min_p[r]
        c = np.cumsum(np.where(keep, w, 0.0))
        token[r] = min(int(np.searchsorted(c, u[r] * c[-1], side="right")), int(np.searchsorted(c, c[-1], side="left")))
    return {"token": torch.from_numpy(token)}
