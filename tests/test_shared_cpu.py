"""Refusals of the shared-prefix verify call, none of which needs a GPU."""
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
KVH, QOH = np.array([0, 8, 20], np.int32), np.array([0, 2, 6], np.int32)
GOOD = dict(q=P, pool=P, slots=64, scale=0.0, shared=P, rows=10, kvp=P, kvi=P, qop=P, mask=None, parent=None, kvh=KVH,
            qoh=QOH, batch=2, heads=16, sm_scale=0.1, splits=0, out=P, lse=P, ws=P, wsb=1 << 30, stream=None)


def _call(B, **kw):
    a = {**GOOD, **kw}
    for k in ("kvh", "qoh"):
        a[k] = a[k].ctypes.data if a[k] is not None else None
    return B.lib().verify_attn_mla_shared(*[a[k] for k in GOOD])


@pytest.mark.parametrize("bad,want", [
    *[({k: None}, "NULL") for k in ("q", "pool", "shared", "kvp", "kvi", "qop", "out", "lse", "ws", "kvh", "qoh")],
    (dict(rows=-1), "SHAPE"), (dict(rows=(1 << 31) - 10), "SHAPE"), (dict(slots=-1), "SHAPE"), (dict(slots=0), "SHAPE"),
    (dict(batch=-1), "SHAPE"), (dict(heads=0), "SHAPE"), (dict(heads=129), "SHAPE"), (dict(splits=65), "SHAPE"),
    (dict(splits=-2), "SHAPE"), (dict(sm_scale=0.0), "SHAPE"), (dict(sm_scale=float("nan")), "SHAPE"),
    (dict(scale=-0.5), "SHAPE"), (dict(scale=float("inf")), "SHAPE"), (dict(scale=float("nan")), "SHAPE"),
    (dict(kvh=np.array([0, 1, 20], np.int32)), "SHAPE"),       # fewer own rows than drafts
    (dict(kvh=np.array([1, 8, 20], np.int32)), "SHAPE"), (dict(qoh=np.array([0, 6, 2], np.int32)), "SHAPE"),
    (dict(kvh=np.array([0, 100, 200], np.int32), qoh=np.array([0, 65, 66], np.int32)), "SHAPE"),  # 65 drafts
    (dict(q=P + 8), "ALIGN"), (dict(pool=P + 2), "ALIGN"), (dict(out=P + 8), "ALIGN"), (dict(lse=P + 2), "ALIGN"),
    (dict(ws=P + 16), "ALIGN"), (dict(mask=P + 4), "ALIGN"), (dict(parent=P + 2), "ALIGN"), (dict(shared=P + 2), "ALIGN"),
    (dict(kvi=P + 1), "ALIGN"),
])
def test_argument_errors(B, bad, want):
    assert _call(B, **bad) == getattr(B, f"VMLA_ERR_{want}")


def test_batch_bound(B):
    n = 512  # one entry of the plan stands for the shared rows
    kvh, qoh = np.arange(n + 1, dtype=np.int32), np.arange(n + 1, dtype=np.int32)
    assert _call(B, batch=n, kvh=kvh, qoh=qoh) == B.VMLA_ERR_SHAPE
    size = ctypes.c_size_t(0)
    f = B.lib().verify_attn_mla_shared_workspace_size
    assert f(n, 16, 10, qoh.ctypes.data, kvh.ctypes.data, 0, ctypes.byref(size)) == B.VMLA_ERR_SHAPE
    assert f(2, 16, 10, QOH.ctypes.data, KVH.ctypes.data, 0, None) == B.VMLA_ERR_NULL
    assert f(2, 16, -1, QOH.ctypes.data, KVH.ctypes.data, 0, ctypes.byref(size)) == B.VMLA_ERR_SHAPE


def test_binding_checks(B):
    import torch
    q = torch.zeros(6, 16, 576, dtype=torch.bfloat16)
    idx = torch.zeros(20, dtype=torch.int32)
    pool = torch.zeros(64, 576, dtype=torch.bfloat16)
    out, lse, ws = torch.zeros(6, 16, 512, dtype=torch.bfloat16), torch.zeros(6, 16), torch.zeros(256, dtype=torch.uint8)
    ptr = torch.zeros(3, dtype=torch.int32)
    good = [q, pool, idx[:10], ptr, idx, ptr, KVH, QOH, out, lse, ws, 0.1]
    for at, bad in ((0, q[:5]), (2, idx.view(4, 5)), (3, ptr[:2]), (4, idx[:19]), (6, KVH[:2]), (8, out[..., :511]), (9, lse[:, :15])):
        a = list(good)
        a[at] = bad
        with pytest.raises(ValueError):
            B.verify_attn_mla_shared(*a)
    with pytest.raises(ValueError, match="device memory"):
        B.verify_attn_mla_shared(*good)
    with pytest.raises(ValueError, match="parent"):
        B.verify_attn_mla_shared(*good, parent=idx)
