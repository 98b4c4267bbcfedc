"""Refusals of the latent-pool append, none of which needs a GPU: the C ABI's argument errors (the
pointers are never read) and the binding's checks."""
import numpy as np
import pytest

from speculative_decoding_mla_gb300 import build as vbuild


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


P = 1 << 20  # a 16-byte aligned address that is never dereferenced
GOOD = dict(latent=P, ls=576, k_rope=P + 1024, ks=576, q_rope=P, qt=64 * 16, qh=64, pos=P, slots=P, table=P, rows=128,
            pairs=1, tokens=4, heads=16, pool=P, pool_slots=64, scale=0.0, q=P, status=None, stream=None)


def _call(B, **kw):
    a = {**GOOD, **kw}
    return B.lib().verify_attn_mla_append(*[a[k] for k in GOOD])


@pytest.mark.parametrize("bad,want", [
    (dict(latent=None), "NULL"), (dict(k_rope=None), "NULL"), (dict(pos=None), "NULL"), (dict(slots=None), "NULL"),
    (dict(table=None), "NULL"), (dict(pool=None), "NULL"), (dict(q_rope=None), "NULL"), (dict(q=None), "NULL"),
    (dict(tokens=-1), "SHAPE"), (dict(tokens=1 << 31), "SHAPE"), (dict(heads=-1), "SHAPE"), (dict(heads=129), "SHAPE"),
    (dict(pool_slots=-1), "SHAPE"), (dict(pool_slots=1 << 31), "SHAPE"), (dict(rows=-1), "SHAPE"),
    (dict(scale=-1.0), "SHAPE"), (dict(scale=float("inf")), "SHAPE"), (dict(scale=float("nan")), "SHAPE"),
    (dict(ls=504), "SHAPE"), (dict(ks=56), "SHAPE"), (dict(qt=56), "SHAPE"), (dict(qh=56), "SHAPE"),
    (dict(ls=0), "SHAPE"), (dict(qh=-64), "SHAPE"), (dict(ls=1 << 40), "SHAPE"),
    (dict(latent=P + 2), "ALIGN"), (dict(k_rope=P + 8), "ALIGN"), (dict(table=P + 4), "ALIGN"), (dict(pool=P + 8), "ALIGN"),
    (dict(q=P + 2), "ALIGN"), (dict(q_rope=P + 8), "ALIGN"), (dict(pos=P + 2), "ALIGN"), (dict(slots=P + 1), "ALIGN"),
    (dict(status=P + 2), "ALIGN"), (dict(ls=577), "ALIGN"), (dict(ks=580), "ALIGN"), (dict(qt=68 * 16 + 4), "ALIGN"),
    (dict(qh=68), "ALIGN"),
])
def test_argument_errors(B, bad, want):
    assert _call(B, **bad) == getattr(B, f"VMLA_ERR_{want}")


def test_nothing_to_do_and_no_queries(B):
    assert _call(B, tokens=0, latent=None, q=None) == B.VMLA_OK
    # without heads the query arguments are not looked at; the call gets as far as asking for a device
    import torch
    if not torch.cuda.is_available():
        assert _call(B, heads=0, q=None, q_rope=None, qt=0, qh=0) == B.VMLA_ERR_DEVICE


def test_binding_checks(B):
    torch = pytest.importorskip("torch")
    cpu = torch.zeros(4, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="latent"):
        B.verify_attn_mla_append(cpu, cpu[:, :64], None, None, None, None)
    with pytest.raises(ValueError, match="together"):
        B.verify_attn_mla_append(cpu, cpu, None, None, None, None, q_rope=cpu)
    with pytest.raises(ValueError, match="latent"):
        B.verify_attn_mla_append(np.zeros((4, 512), np.uint16), None, None, None, None, None)
