"""The append of long prompts: 32 heads to a warp, which calls of more than 16 heads take once tokens x ceil(heads / 32)
reach 64 for every SM.  Tolerances as derived in tests/test_gpu_append.py."""
import numpy as np
import pytest

from tests.test_gpu_append import _call, _case, _f64, _mods, _near_bf16, _rot

pytestmark = pytest.mark.gpu


def _tokens(heads):
    """The fewest tokens of the wide form, and a few more (not a multiple of a block's four warps)."""
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    parts = -(-heads // 32)
    tokens = -(-64 * sms // parts) + 3
    assert heads > 16 and tokens * parts >= 64 * sms
    return tokens


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("H,in_place,fp8", [(17, False, True), (24, True, False), (33, False, False), (33, True, True), (128, True, False)])
def test_wide_form(H, in_place, fp8, interleaved):
    torch, binding = _mods()
    T = _tokens(H)
    c = _case(T, H, T + 50, seed=H)
    scale = 0.0125 if fp8 else 0.0
    if fp8:
        c["pool"] = torch.full((T + 50, 576), 0x11, dtype=torch.uint8, device="cuda")
    good = torch.ones(T, dtype=torch.bool, device="cuda")
    good[-7:] = False                 # a padded batch
    c["slots"][-7:] = -1
    for at, key, bad in ((5, "slots", T + 50), (T // 2, "positions", 4096), (T - 9, "positions", -1)):
        c[key][at] = bad
        good[at] = False
    unrotated = c["q_rope"].clone()
    if in_place:
        c["q"][..., 512:] = c["q_rope"]
        c["q_rope"] = c["q"][..., 512:]
    pool0, q0 = c["pool"].clone(), c["q"].clone()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    _call(binding, c, interleaved=interleaved, kv_scale=scale, status_word=st)
    torch.cuda.synchronize()
    assert int(st[0]) == binding.VMLA_ERR_INDEX and int(st[1]) in (5, T // 2, T - 9)
    assert torch.equal(c["q"][~good].view(torch.int16), q0[~good].view(torch.int16))
    assert torch.equal(c["q"][..., :512].contiguous().view(torch.int16), q0[..., :512].contiguous().view(torch.int16))
    slots = c["slots"][good].long()
    rest = torch.ones(T + 50, dtype=torch.bool, device="cuda")
    rest[slots] = False
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal(c["pool"][rest].view(bits), pool0[rest].view(bits))
    cs = _f64(c["table"])[c["positions"][good].cpu().numpy()]
    for h in range(H):
        want, mag = _rot(_f64(unrotated[good][:, h]), cs, interleaved)
        assert _near_bf16(_f64(c["q"][good][:, h, 512:]), want, mag).all(), h
    if fp8:  # the cache rows are the same in the narrow form, which is tested against the formula
        d = {**c, "pool": pool0, "q": None, "q_rope": None}
        _call(binding, d, interleaved=interleaved, kv_scale=scale, status_word=st)
        assert torch.equal(c["pool"], d["pool"])
    else:
        assert torch.equal(c["pool"][slots][:, :512].view(torch.int16), c["latent"][good].contiguous().view(torch.int16))
        want, mag = _rot(_f64(c["k_rope"][good]), cs, interleaved)
        assert _near_bf16(_f64(c["pool"][slots][:, 512:]), want, mag).all()


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("scale", [1.0, 0.0125, 0.37])
def test_rotated_codes_come_from_unrounded_values(scale, interleaved):
    """A rotated column's code is that of its fp32 value / scale, without a rounding to bf16 between: the fp32 value is
    within 2 x 2^-24 of the products' magnitudes and its quotient within 2^-24, so the code lies between those of the two
    ends of that interval (which are mostly one code)."""
    torch, binding = _mods()
    c = _case(700, 0, 700, seed=3, sigma=2.0)
    c["pool"] = torch.zeros((700, 576), dtype=torch.uint8, device="cuda")
    _call(binding, c, interleaved=interleaved, kv_scale=scale)
    torch.cuda.synchronize()
    s32 = float(np.float32(scale))
    got = _f64(c["pool"].view(torch.float8_e4m3fn)[c["slots"].long()][:, 512:].float())
    want, mag = _rot(_f64(c["k_rope"]), _f64(c["table"])[c["positions"].cpu().numpy()], interleaved)
    slack = (2 * mag + 2 * abs(want)) * 2.0 ** -24 / s32
    code = lambda v: _f64(torch.from_numpy(np.clip(v, -448, 448)).float().to(torch.float8_e4m3fn).float())  # noqa: E731
    lo, hi = code(want / s32 - slack), code(want / s32 + slack)
    assert ((lo <= got) & (got <= hi)).all()
    assert (lo == hi).mean() > 0.99
