"""Refusals of the sampling call, none of which needs a GPU."""
import numpy as np
import pytest

from speculative_decoding_mla_gb300 import build as vbuild


@pytest.fixture(scope="module")
def B():
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return binding


P = 1 << 20  # an aligned address that is never dereferenced
GOOD = dict(logits=P, fp32=0, stride=1000, rows=4, vocab=1000, temperature=P, top_k=P, top_p=P, min_p=P, uniform=P,
            token=P, status=None, stream=None)


def _call(B, **kw):
    a = {**GOOD, **kw}
    return B.lib().verify_attn_mla_sample(*[a[k] for k in GOOD])


@pytest.mark.parametrize("bad,want", [
    (dict(logits=None), "NULL"), (dict(uniform=None), "NULL"), (dict(token=None), "NULL"),
    (dict(rows=-1), "SHAPE"), (dict(rows=1 << 30), "SHAPE"), (dict(vocab=0), "SHAPE"), (dict(vocab=-5), "SHAPE"),
    (dict(vocab=262145, stride=1 << 20), "SHAPE"), (dict(stride=999), "SHAPE"), (dict(stride=-1000), "SHAPE"),
    (dict(stride=1 << 40), "SHAPE"),
    (dict(logits=P + 1), "ALIGN"), (dict(logits=P + 2, fp32=1), "ALIGN"), (dict(temperature=P + 2), "ALIGN"),
    (dict(top_k=P + 1), "ALIGN"), (dict(top_p=P + 2), "ALIGN"), (dict(min_p=P + 2), "ALIGN"),
    (dict(uniform=P + 2), "ALIGN"), (dict(token=P + 2), "ALIGN"), (dict(status=P + 2), "ALIGN"),
])
def test_argument_errors(B, bad, want):
    assert _call(B, **bad) == getattr(B, f"VMLA_ERR_{want}")


def test_nothing_to_do(B):
    assert _call(B, rows=0, logits=None, token=None) == B.VMLA_OK
    assert B.status_string(B.VMLA_ERR_PARAM) != "unknown status"


def test_binding_checks(B):
    import torch
    x, u, t = torch.zeros(4, 50), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    for a, k in (((x.double(), u, t), {}), ((x.to(torch.float16), u, t), {}), ((x.to(torch.int32), u, t), {}),
                 ((x[0], u, t), {}), ((x, u[:3], t), {}), ((x, u, t[:3]), {}), ((x, u, t), dict(top_k=t[:1])),
                 ((x, u, t), dict(temperature=x)), ((x, u, t), dict(status_word=t[:1])),
                 ((np.zeros((4, 50), np.float32), u, t), {})):
        with pytest.raises(ValueError):
            B.verify_attn_mla_sample(*a, **k)
    with pytest.raises(ValueError, match="device memory"):
        B.verify_attn_mla_sample(x, u, t)
