"""Refusals of a step's calls over the scaled pool (tables, append, attention, beams), none of which needs a GPU: the C
ABI's argument errors (the pointers are never read) and the binding's checks."""
import ctypes

import numpy as np
import pytest

from speculative_decoding_mla_gb300 import build as vbuild


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


P = 1 << 20  # an aligned address that is never dereferenced
APPEND = dict(latent=P, ls=576, k_rope=P + 1024, ks=576, q_rope=P, qt=64 * 16, qh=64, pos=P, slots=P, table=P, rows=128, pairs=1,
              tokens=4, heads=16, pool=P, pool_slots=64, scales=P, block=16, q=P, status=None, stream=None)
ATTEND = dict(q=P, pool=P, slots=64, scales=P, block=16, kvp=P, kvi=P, qop=P, mask=None, parent=P, batch=2, heads=16, max_q=6,
              max_kv=20, sm_scale=0.1, out=P, lse=P, ws=P, wsb=1 << 30, stream=None)
TABLES = dict(cached=P, added=P, batch=2, block=16, table=P, stride=9, width=8, free=P, free_size=40, count=P, left=P, scratch=P,
              max_q=6, max_kv=20, kvp=P, qop=P, kvi=P, pos=P, slots=P, status=None, stream=None)
SELECT = dict(logits=P, fp32=0, stride=1000, requests=3, beams=4, keep=4, vocab=1000, score=P, finished=None, pad=0, parent=P,
              token=P, new_score=P, ws=P, wsb=1 << 30, stream=None)
REORDER = dict(src=P, ss=64, dst=P, ds=64, words=60, requests=3, beams=4, keep=4, parent=P, length=P, new_length=P, status=None,
               stream=None)
ENTRIES = dict(append_scaled=APPEND, scaled=ATTEND, step_tables=TABLES, beam_select=SELECT, beam_reorder=REORDER)

BAD = {
    "append_scaled": [
        *[({k: None}, "NULL") for k in ("latent", "k_rope", "pos", "slots", "table", "pool", "scales", "q_rope", "q")],
        *[(dict(block=b), "SHAPE") for b in (0, -1, 3, 12, 256, 1 << 30)],
        (dict(pool_slots=63), "SHAPE"), (dict(block=128), "SHAPE"), (dict(tokens=-1), "SHAPE"), (dict(tokens=1 << 31), "SHAPE"),
        (dict(heads=129), "SHAPE"), (dict(heads=-1), "SHAPE"), (dict(pool_slots=1 << 31, block=1), "SHAPE"), (dict(ls=504), "SHAPE"),
        (dict(scales=P + 2), "ALIGN"), (dict(pool=P + 8), "ALIGN"), (dict(latent=P + 2), "ALIGN"), (dict(ks=577), "ALIGN"),
        (dict(slots=P + 1), "ALIGN"), (dict(status=P + 3), "ALIGN"),
    ],
    "scaled": [
        *[({k: None}, "NULL") for k in ("q", "pool", "scales", "kvp", "kvi", "qop", "out", "lse", "ws")],
        *[(dict(block=b), "SHAPE") for b in (0, -16, 24, 256)],
        (dict(slots=65), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(slots=-16), "SHAPE"), (dict(slots=1 << 31), "SHAPE"),
        (dict(batch=-1), "SHAPE"), (dict(batch=513), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(heads=129), "SHAPE"),
        (dict(max_q=129), "SHAPE"), (dict(max_q=-1), "SHAPE"), (dict(max_kv=-1), "SHAPE"), (dict(max_kv=1 << 31), "SHAPE"),
        *[(dict(sm_scale=v), "SHAPE") for v in (0.0, -1.0, float("inf"), float("nan"))],
        *[({k: P + 2}, "ALIGN") for k in ("kvp", "kvi", "qop", "parent", "scales", "lse")],
        (dict(q=P + 8), "ALIGN"), (dict(out=P + 2), "ALIGN"), (dict(pool=P + 8), "ALIGN"), (dict(mask=P + 4), "ALIGN"),
        (dict(ws=P + 128), "ALIGN"),
    ],
    "step_tables": [
        *[({k: None}, "NULL") for k in ("cached", "added", "table", "free", "count", "left", "scratch", "kvp", "qop", "kvi", "pos", "slots")],
        *[(dict(block=b), "SHAPE") for b in (0, 6, 256)],
        (dict(batch=-1), "SHAPE"), (dict(batch=513), "SHAPE"), (dict(stride=7), "SHAPE"), (dict(width=-1), "SHAPE"),
        (dict(width=1 << 31, stride=1 << 31), "SHAPE"), (dict(stride=1 << 40), "SHAPE"), (dict(free_size=-1), "SHAPE"),
        (dict(free_size=1 << 31), "SHAPE"), (dict(max_q=1 << 31), "SHAPE"), (dict(max_kv=-1), "SHAPE"), (dict(max_q=-1), "SHAPE"),
        *[({k: P + 2}, "ALIGN") for k in ("cached", "added", "table", "free", "count", "left", "scratch", "kvp", "qop", "kvi", "pos",
                                          "slots", "status")],
    ],
    "beam_select": [
        *[({k: None}, "NULL") for k in ("logits", "score", "parent", "token", "new_score", "ws")],
        (dict(requests=-1), "SHAPE"), (dict(requests=65536), "SHAPE"), (dict(beams=0), "SHAPE"), (dict(beams=17), "SHAPE"),
        (dict(keep=0), "SHAPE"), (dict(keep=33), "SHAPE"), (dict(vocab=0), "SHAPE"), (dict(vocab=262145, stride=300000), "SHAPE"),
        (dict(stride=999), "SHAPE"), (dict(stride=1 << 40), "SHAPE"), (dict(pad=-1), "SHAPE"), (dict(pad=1000), "SHAPE"),
        (dict(logits=P + 1), "ALIGN"), (dict(fp32=1, logits=P + 2), "ALIGN"), (dict(ws=P + 16), "ALIGN"),
        *[({k: P + 2}, "ALIGN") for k in ("score", "finished", "parent", "token", "new_score")],
    ],
    "beam_reorder": [
        *[({k: None}, "NULL") for k in ("src", "dst", "parent", "length")],
        (dict(requests=-1), "SHAPE"), (dict(requests=65536), "SHAPE"), (dict(beams=0), "SHAPE"), (dict(beams=17), "SHAPE"),
        (dict(keep=0), "SHAPE"), (dict(keep=33), "SHAPE"), (dict(words=-1), "SHAPE"), (dict(ss=59), "SHAPE"), (dict(ds=59), "SHAPE"),
        (dict(ss=1 << 40), "SHAPE"), (dict(words=1 << 31, ss=1 << 31, ds=1 << 31), "SHAPE"),
        *[({k: P + 2}, "ALIGN") for k in ("src", "dst", "parent", "length", "new_length", "status")],
    ],
}


@pytest.mark.parametrize("entry,bad,want", [(e, b, w) for e, l in BAD.items() for b, w in l])
def test_argument_errors(B, entry, bad, want):
    a = {**ENTRIES[entry], **bad}
    assert getattr(B.lib(), "verify_attn_mla_" + entry)(*a.values()) == getattr(B, f"VMLA_ERR_{want}")


def test_nothing_to_do(B):
    lib = B.lib()
    assert lib.verify_attn_mla_append_scaled(*{**APPEND, "tokens": 0, "latent": None, "scales": None}.values()) == B.VMLA_OK
    assert lib.verify_attn_mla_beam_select(*{**SELECT, "requests": 0, "logits": None}.values()) == B.VMLA_OK
    assert lib.verify_attn_mla_beam_reorder(*{**REORDER, "requests": 0, "parent": None}.values()) == B.VMLA_OK


def test_sizes(B):
    n = ctypes.c_size_t(0)
    lib = B.lib()
    size = lib.verify_attn_mla_scaled_workspace_size
    assert size(2, 16, 6, 20, None) == B.VMLA_ERR_NULL
    for bad in ((-1, 16, 0, 0), (513, 16, 0, 0), (2, 0, 6, 20), (2, 129, 6, 20), (2, 16, 129, 20), (2, 16, 6, 1 << 31)):
        assert size(*bad, ctypes.byref(n)) == B.VMLA_ERR_SHAPE
    beams = lib.verify_attn_mla_beam_select_workspace_size
    assert beams(8, 100, 4, None) == B.VMLA_ERR_NULL
    for bad in ((-1, 100, 4), (65535 * 16 + 1, 100, 4), (8, 0, 4), (8, 262145, 4), (8, 100, 0), (8, 100, 33)):
        assert beams(*bad, ctypes.byref(n)) == B.VMLA_ERR_SHAPE
    lib.verify_attn_mla_status_string.restype = ctypes.c_char_p
    assert b"room" in lib.verify_attn_mla_status_string(B.VMLA_ERR_FULL)


def test_binding_checks(B):
    import torch
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pool, scales = torch.zeros(64, 576, dtype=torch.uint8), torch.zeros(4)
    q, out, lse = torch.zeros(6, 2, 576, dtype=torch.bfloat16), torch.zeros(6, 2, 512, dtype=torch.bfloat16), torch.zeros(6, 2)
    ws = torch.zeros(256, dtype=torch.uint8)
    attend = dict(q=q, kv_pool=pool, kv_scales=scales, kv_indptr=i32(3), kv_indices=i32(9), qo_indptr=i32(3), out=out, lse=lse,
                  workspace=ws, sm_scale=0.1, block_tokens=16)
    for bad, word in ((dict(block_tokens=0), "block_tokens"), (dict(block_tokens=24), "block_tokens"), (dict(kv_scales=torch.zeros(5)), "kv_scales"),
                      (dict(kv_scales=scales.double()), "kv_scales"), (dict(kv_pool=pool[:, :570]), "kv_pool"), (dict(q=q[0]), "q"),
                      (dict(out=out[:5]), "out"), (dict(lse=lse[:, :1]), "lse"), (dict(qo_indptr=i32(4)), "qo_indptr"),
                      (dict(parent=i32(5)), "parent"), (dict(draft_mask=torch.zeros(7, dtype=torch.int64)), "draft_mask"), ({}, "kv_scales|q|cuda|device")):
        with pytest.raises(ValueError, match=word):
            B.verify_attn_mla_scaled(**{**attend, **bad})
    with pytest.raises(ValueError, match="block_tokens"):
        B.verify_attn_mla_append_scaled(q[:, 0, :512], q[:, 0, 512:], i32(6), i32(6), torch.zeros(9, 64), pool, scales, block_tokens=5)
    tables = dict(cached=i32(2), added=i32(2), block_table=i32(2, 8), free_blocks=i32(9), free_count=i32(1), free_left=i32(1), scratch=i32(1),
                  kv_indptr=i32(3), qo_indptr=i32(3), kv_indices=i32(30), positions=i32(6), slots=i32(6))
    for bad, word in ((dict(added=i32(3)), "added"), (dict(block_table=i32(3, 8)), "block_table"), (dict(kv_indptr=i32(2)), "kv_indptr"),
                      (dict(positions=i32(5)), "positions"), (dict(free_count=i32(2)), "free_count"), (dict(status_word=i32(1)), "status_word")):
        with pytest.raises(ValueError, match=word):
            B.verify_attn_mla_step_tables(**{**tables, **bad})
    x = torch.zeros(8, 100)
    select = dict(logits=x, score=torch.zeros(8), parent=i32(2, 4), token=i32(2, 4), new_score=torch.zeros(2, 4), workspace=ws, beams=4)
    for bad, word in ((dict(beams=3), "beams"), (dict(beams=0), "beams"), (dict(logits=x.half()), "logits"), (dict(logits=x[0]), "logits"),
                      (dict(parent=i32(3, 4)), "parent"), (dict(token=i32(2, 5)), "token"), (dict(score=torch.zeros(7)), "score"),
                      (dict(finished=i32(9)), "finished")):
        with pytest.raises(ValueError, match=word):
            B.verify_attn_mla_beam_select(**{**select, **bad})
    reorder = dict(src=i32(8, 20), dst=i32(8, 20), parent=i32(2, 4), beams=4)
    for bad, word in ((dict(src=i32(7, 20)), "src"), (dict(dst=i32(8, 19)), "dst"), (dict(length=i32(7)), "length"), (dict(parent=i32(8)), "parent"),
                      (dict(new_length=i32(7)), "new_length"), (dict(status_word=i32(1)), "status_word"), ({}, "src"),
                      (dict(dst=np.zeros((8, 20), np.int32)), "src|dst")):
        with pytest.raises(ValueError, match=word):
            B.verify_attn_mla_beam_reorder(**{**reorder, **bad})
