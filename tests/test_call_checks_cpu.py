"""Refusals that keep a call from reading what it was not given; none of them needs a GPU."""
import ctypes

import numpy as np
import pytest

from speculative_decoding_mla_gb300 import build as vbuild
from tests.test_shared_cpu import KVH, QOH
from tests.test_shared_cpu import _call as _shared


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31, 2 ** 32 + 5, 2 ** 62, 2 ** 63 - 10, 2 ** 63 - 1])
def test_shared_rows_past_every_integer(B, rows):
    """The sum of shared and own rows is not taken before the shared ones are known to fit."""
    assert _shared(B, rows=rows) == B.VMLA_ERR_SHAPE
    size = ctypes.c_size_t(0)
    f = B.lib().verify_attn_mla_shared_workspace_size
    assert f(2, 16, rows, QOH.ctypes.data, KVH.ctypes.data, 0, ctypes.byref(size)) == B.VMLA_ERR_SHAPE


P = 1 << 20  # an aligned address that is never dereferenced
RUN = dict(q=P, pool=P, slots=64, kvp=P, kvi=P, qop=P, mask=None, parent=P, kvh=KVH, qoh=QOH, batch=2, heads=16,
           sm_scale=0.1, splits=0, out=P, lse=P, ws=P, wsb=1 << 30, stream=None)
RUNS = {k if k != "kvi" else "base": v for k, v in RUN.items()}
FP8 = dict(q=P, pool=P, slots=64, scale=0.5, **{k: v for k, v in RUN.items() if k not in ("q", "pool", "slots")})
DPLAN = dict(q=P, pool=P, slots=64, kvp=P, kvi=P, qop=P, mask=None, parent=P, batch=2, heads=16, max_q=6, max_kv=20,
             sm_scale=0.1, splits=0, out=P, lse=P, ws=P, wsb=1 << 30, stream=None)
DEFRAG = dict(pool=P, slots=64, kvp=P, kvi=P, kvh=KVH, batch=2, dst=P, dst_slots=64, base=P, status=P, stream=None)
MASK = dict(parent=P, qop=P, batch=2, total_q=6, out=P, status=P, stream=None)
# the int32 arrays that the kernels of an entry point read
READ = {"verify_attn_mla": (RUN, ("kvi", "qop", "parent")), "verify_attn_mla_simt": (RUN, ("kvi", "qop", "parent")),
        "verify_attn_mla_fp8": (FP8, ("kvi", "qop", "parent")), "verify_attn_mla_runs": (RUNS, ("kvp", "base", "qop", "parent")),
        "verify_attn_mla_device_plan": (DPLAN, ("kvp", "kvi", "qop", "parent")),
        "verify_attn_mla_defrag": (DEFRAG, ("kvp", "kvi", "base", "status")),
        "verify_attn_mla_tree_mask": (MASK, ("parent", "qop", "status"))}


@pytest.mark.parametrize("entry,array", [(e, a) for e, (_, arrays) in READ.items() for a in arrays])
def test_int32_arrays_are_aligned(B, entry, array):
    """A kernel's load of four bytes faults on any other address."""
    def call(**kw):
        a = {**READ[entry][0], **kw}
        return getattr(B.lib(), entry)(*[v.ctypes.data if isinstance(v, np.ndarray) else v for v in a.values()])
    for off in (1, 2, 3):
        assert call(**{array: P + off}) == B.VMLA_ERR_ALIGN


@pytest.mark.parametrize("off", [1, 2, 3])
def test_int32_arrays_of_the_shared_call_are_aligned(B, off):
    for array in ("shared", "kvi", "qop", "parent"):
        assert _shared(B, **{array: P + off}) == B.VMLA_ERR_ALIGN


def test_host_offsets_of_different_lengths(B):
    """Every call takes the batch from one of the two host arrays and reads as many entries of the other."""
    import torch
    qo, kv = QOH, KVH
    sizes = [lambda q, k: B.verify_attn_mla_workspace_size(q, k, 16), lambda q, k: B.verify_attn_mla_plan(0, q, k, 16),
             lambda q, k: B.verify_attn_mla_runs_workspace_size(q, k, 16),
             lambda q, k: B.verify_attn_mla_host_buffer_size(q, k, 16),
             lambda q, k: B.verify_attn_mla_shared_workspace_size(10, q, k, 16)]
    for f in sizes:
        for bad in (kv[:2], kv[:1], kv[:0]):
            with pytest.raises(ValueError, match="entries"):
                f(qo, bad)
    q, pool = torch.zeros(6, 16, 576, dtype=torch.bfloat16), torch.zeros(64, 576, dtype=torch.bfloat16)
    idx, ptr = torch.zeros(20, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    out, lse, ws = torch.zeros(6, 16, 512, dtype=torch.bfloat16), torch.zeros(6, 16), torch.zeros(256, dtype=torch.uint8)
    for bad in (qo[:2], qo[:0]):
        for f in (B.verify_attn_mla, B.verify_attn_mla_simt):
            with pytest.raises(ValueError, match="entries"):
                f(q, pool, ptr, idx, ptr, kv, bad, out, lse, ws, 0.1)
        with pytest.raises(ValueError, match="entries"):
            B.verify_attn_mla_fp8(q, pool, 0.5, ptr, idx, ptr, kv, bad, out, lse, ws, 0.1)
        with pytest.raises(ValueError, match="entries"):
            B.verify_attn_mla_simt_static(q, pool, ptr, idx, ptr, kv, bad, out, lse, 0.1)
        with pytest.raises(ValueError, match="entries"):
            B.verify_attn_mla_runs(q, pool, ptr, ptr, ptr, kv, bad, out, lse, ws, 0.1)
        with pytest.raises(ValueError, match="entries"):
            B.verify_attn_mla_host(q, pool, kv, idx, bad, out, lse, ws, 0.1)
        with pytest.raises(ValueError, match="entries"):
            B.verify_attn_mla_shared(q, pool, idx[:10], ptr, idx, ptr, kv, bad, out, lse, ws, 0.1)
