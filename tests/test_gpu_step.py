"""A whole speculative step of the pieces as they would be used together: the step's draft rows are appended
(position rotation on the way) behind a shared prefix and each sequence's own rows, the queries are rotated in
the same launch, the verify attention runs on the shared prefix, a stand-in output projection makes logits, the
target's tokens are sampled, and the draft trees are accepted against them.  Each stage is checked against its
plain form on the values that it really got.

Tolerances as derived in test_gpu_append.py and test_gpu_shared.py; tokens, paths and lengths are equal."""
import numpy as np
import pytest

import oracle
from speculative_decoding_mla_gb300 import synth
from tests.test_gpu_append import _near_bf16, _rot
from tests.test_gpu_sample import reference as sample_reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("captured", [False, True])
def test_append_verify_sample_accept(fp8, captured):
    import torch
    from speculative_decoding_mla_gb300 import build as vbuild
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding as B
    torch.manual_seed(3)
    H, P, V, R = 16, 900, 5000, 2000
    drafts, own = [5, 1, 8, 0, 3], [40, 130, 7, 20, 0]
    Bn, T = len(drafts), sum(drafts)
    kvh = np.concatenate([[0], np.cumsum([d + o for d, o in zip(drafts, own)])]).astype(np.int32)
    qoh = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
    N = int(kvh[-1])
    dev = lambda a, t=np.int32: torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    parent = np.concatenate([synth.tree_parents(5, d, 4, b) for b, d in enumerate(drafts) if d]).astype(np.int32)
    depth = np.zeros(T, np.int64)
    for b in range(Bn):
        for i in range(drafts[b]):
            p = parent[qoh[b] + i]
            depth[qoh[b] + i] = 0 if p < 0 else depth[qoh[b] + p] + 1
    perm = torch.randperm(R)[:P + N].to(torch.int32).cuda()
    shared, kvi = perm[:P].contiguous(), perm[P:].contiguous()
    scale = 0.0125 if fp8 else 0.0
    pool = torch.randn(R, 576, device="cuda") * 0.5
    pool = (pool / scale).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else pool.to(torch.bfloat16)
    # the drafts' rows: positions behind the prefix and the sequence's own tokens, slots the last of each sequence
    seq = np.repeat(np.arange(Bn), drafts)
    positions = dev(P + np.array(own)[seq] + depth)
    slots = kvi[dev(np.concatenate([np.arange(kvh[b + 1] - drafts[b], kvh[b + 1]) for b in range(Bn)]), ).long()].contiguous()
    kv = torch.randn(T, 576, device="cuda").to(torch.bfloat16) * 0.5
    angle = torch.arange(4096, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    table = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
    q = torch.randn(T, H, 576, device="cuda").to(torch.bfloat16)
    q_rope = torch.randn(T, H, 64, device="cuda").to(torch.bfloat16)
    out = torch.empty(T, H, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(T, H, device="cuda")
    ws = torch.empty(B.verify_attn_mla_shared_workspace_size(P, qoh, kvh, H), dtype=torch.uint8, device="cuda")
    head = (torch.randn(H * 512, V, device="cuda") * 0.3).to(torch.bfloat16)  # stands in for the rest of the model
    logits = torch.empty(T, V, dtype=torch.bfloat16, device="cuda")
    u = torch.rand(T, device="cuda")
    temp = torch.full((T,), 0.8, device="cuda")
    top_p = torch.full((T,), 0.9, device="cuda")
    target = torch.empty(T, dtype=torch.int32, device="cuda")
    root = torch.zeros(Bn, dtype=torch.int32, device="cuda")
    draft = torch.zeros(T, dtype=torch.int32, device="cuda")
    acc, nxt = torch.empty(Bn, dtype=torch.int32, device="cuda"), torch.empty(Bn, dtype=torch.int32, device="cuda")
    path = torch.empty(T, dtype=torch.int32, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    kvp, qop, par = dev(kvh), dev(qoh), dev(parent)
    root_t = dev(np.arange(Bn) + 7)

    def step():
        B.verify_attn_mla_append(kv[:, :512], kv[:, 512:], positions, slots, table, pool, q_rope=q_rope, q=q, kv_scale=scale, status_word=st)
        B.verify_attn_mla_shared(q, pool, shared, kvp, kvi, qop, kvh, qoh, out, lse, ws, synth.SM_SCALE, kv_scale=scale, parent=par)
        torch.matmul(out.view(T, H * 512), head, out=logits)
        B.verify_attn_mla_sample(logits, u, target, temperature=temp, top_p=top_p, status_word=st)
        # drafts that the target agrees with here and there: every second node proposes the target's token
        root.copy_(root_t)
        up = torch.where(par >= 0, target[(torch.where(par >= 0, par, 0) + qop[seq_t]).long()], root[seq_t])
        draft.copy_(torch.where(torch.arange(T, device="cuda") % 3 != 2, up, up + 1))
        B.verify_attn_mla_tree_accept(qop, par, draft, target, root, acc, path, nxt, st)

    seq_t = dev(seq).long()
    q0 = q.clone()
    step()
    if captured:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        kv.copy_(torch.randn_like(kv) * 0.5)
        u.copy_(torch.rand(T, device="cuda"))
        g.replay()
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0] and B.verify_attn_mla_check(ws) == 0
    # append
    cs = table.double().cpu().numpy()[positions.cpu().numpy()]
    want, mag = _rot(q_rope.double().cpu().numpy(), cs[:, None], True)
    assert _near_bf16(q.double().cpu().numpy()[..., 512:], want, mag).all()
    assert torch.equal(q[..., :512].contiguous().view(torch.int16), q0[..., :512].contiguous().view(torch.int16))
    values = (pool.view(torch.float8_e4m3fn).float() * scale).to(torch.bfloat16) if fp8 else pool
    rows = values[slots.long()].double().cpu().numpy()
    want, mag = _rot(kv[:, 512:].double().cpu().numpy(), cs, True)
    want = np.concatenate([kv[:, :512].double().cpu().numpy(), want], 1)
    mag = np.concatenate([abs(want[:, :512]), mag], 1)
    if fp8:  # a code and its bf16 value: 2^-4 and 2^-8, half a step of the smallest codes
        assert (abs(rows - np.clip(want, -448 * scale, 448 * scale)) <= (2.0 ** -4 + 2.0 ** -7) * mag + 2.0 ** -9 * scale).all()
    else:
        assert _near_bf16(rows, want, mag).all()
    # verify, on what the pool and q now hold
    vals = values.double().cpu().numpy()
    qn, words = q.double().cpu().numpy(), oracle.tree_masks(parent, qoh)
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    sh, ki = shared.cpu().numpy(), kvi.cpu().numpy()
    for b in range(Bn):
        r = vals[np.concatenate([sh, ki[kvh[b]:kvh[b + 1]]])]
        for i in range(drafts[b]):
            t = qoh[b] + i
            see = np.concatenate([np.ones(len(r) - drafts[b], bool), [(int(words[t]) >> k) & 1 == 1 for k in range(drafts[b])]]).astype(bool)
            s = (qn[t] @ r[see].T) * synth.SM_SCALE
            m = s.max(1, keepdims=True)
            e = np.exp(s - m)
            p = e / e.sum(1, keepdims=True)
            want, mag = p @ r[see][:, :512], p @ abs(r[see][:, :512])
            slack = (2.0 ** -8 + 2.0 ** -9 + 2.0 ** -12) * mag
            assert (abs(o[t] - want) <= slack + 2.0 ** -8 * (abs(want) + slack)).all()
            assert abs(l[t] - (m + np.log(e.sum(1, keepdims=True)))[:, 0]).max() < 1e-3
    # sample and accept
    tok = sample_reference(logits.float().cpu().numpy(), u.cpu().numpy(), temp.cpu().numpy(), top_p=top_p.cpu().numpy())
    assert np.array_equal(target.cpu().numpy(), tok)
    al, ap, nt, bad = oracle.tree_accept(qoh, parent, draft.cpu().numpy(), tok, root.cpu().numpy())
    assert not bad.any() and al.max() >= 2
    assert np.array_equal(acc.cpu().numpy(), al) and np.array_equal(path.cpu().numpy(), ap) and np.array_equal(nxt.cpu().numpy(), nt)
