"""The latent-pool append on the GPU against its definition in 64 bits.

Tolerances, fixed before the first run.  A rotated value is x = a c - b d (or a d + b c) of bf16 a, b and
fp32 c, d: two products and a sum in fp32 are off by at most 2 x 2^-24 (|a c| + |b d|) (one product rounded,
the other inside a fused multiply-add, and the sum rounded; |x| <= |a c| + |b d|).  Storing rounds to bf16,
off by at most 2^-8 of the stored value's magnitude; dividing by the scale is off by 2^-24, an e4m3 code by at
most 2^-4 of the value or half a step (2^-10) of the smallest codes.  Latent columns in bf16 are copied: equal
bits."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

BF16, FP32, E4M3 = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4


def _mods():
    import torch
    from speculative_decoding_mla_gb300 import build as vbuild
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return torch, binding


def _case(T, H, slots, context=4096, seed=0, fused=True, sigma=1.0):
    torch, _ = _mods()
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = lambda *s: (torch.randn(s, generator=g, device="cuda") * sigma).to(torch.bfloat16)  # noqa: E731
    kv = n(T, 576)
    c = dict(latent=kv[:, :512] if fused else kv[:, :512].contiguous(), k_rope=kv[:, 512:] if fused else kv[:, 512:].contiguous(),
             slots=torch.randperm(slots, generator=g, device="cuda")[:T].to(torch.int32),
             positions=torch.randint(0, context, (T,), generator=g, device="cuda", dtype=torch.int32),
             table=torch.randn((context, 64), generator=g, device="cuda"), pool=n(slots, 576),
             q=n(T, H, 576) if H else None, q_rope=n(T, H, 64) if H else None)
    return c


def _call(binding, c, **k):
    binding.verify_attn_mla_append(c["latent"], c["k_rope"], c["positions"], c["slots"], c["table"], c["pool"],
                                   q_rope=c["q_rope"], q=c["q"], **k)


def _f64(t):
    return t.double().cpu().numpy()


def _rot(x, cs, interleaved):
    """(rotated, sum of the products' magnitudes), 64 bits."""
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    cos, sin = cs[..., :32], cs[..., 32:]
    r = (a * cos - b * sin, a * sin + b * cos)
    m = (abs(a * cos) + abs(b * sin), abs(a * sin) + abs(b * cos))
    join = (lambda p: np.stack(p, -1).reshape(x.shape)) if interleaved else (lambda p: np.concatenate(p, -1))
    return join(r), join(m)


def _near_bf16(got, want, mag):
    slack = 2 * FP32 * mag
    return abs(got - want) <= BF16 * (abs(want) + slack) + slack


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,H,fused", [(1, 64, True), (1, 0, True), (3, 1, False), (17, 24, True), (130, 33, True), (700, 128, False)])
def test_rows_and_queries(T, H, fused, interleaved):
    torch, binding = _mods()
    c = _case(T, H, 1000, seed=T + H, fused=fused)
    pool0, q0 = c["pool"].clone(), None if not H else c["q"].clone()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    _call(binding, c, interleaved=interleaved, status_word=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0]
    cs = _f64(c["table"])[c["positions"].cpu().numpy()]
    slots = c["slots"].long()
    assert torch.equal(c["pool"][slots][:, :512].view(torch.int16), c["latent"].contiguous().view(torch.int16))
    want, mag = _rot(_f64(c["k_rope"]), cs, interleaved)
    assert _near_bf16(_f64(c["pool"][slots][:, 512:]), want, mag).all()
    rest = torch.ones(1000, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert torch.equal(c["pool"][rest].view(torch.int16), pool0[rest].view(torch.int16))
    if H:
        want, mag = _rot(_f64(c["q_rope"]), cs[:, None], interleaved)
        assert _near_bf16(_f64(c["q"][..., 512:]), want, mag).all()
        assert torch.equal(c["q"][..., :512].contiguous().view(torch.int16), q0[..., :512].contiguous().view(torch.int16))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("T,scale", [(1, 0.0125), (37, 0.003), (515, 2.0)])
def test_e4m3_pool(T, scale, interleaved):
    torch, binding = _mods()
    c = _case(T, 8, 900, seed=T, sigma=3.0)
    c["pool"] = torch.full((900, 576), 0x11, dtype=torch.uint8, device="cuda")
    _call(binding, c, interleaved=interleaved, kv_scale=scale)
    torch.cuda.synchronize()
    slots = c["slots"].long()
    s32 = float(np.float32(scale))
    got = _f64(c["pool"].view(torch.float8_e4m3fn)[slots].float())
    cs = _f64(c["table"])[c["positions"].cpu().numpy()]
    rot, mag = _rot(_f64(c["k_rope"]), cs, interleaved)
    want = np.concatenate([_f64(c["latent"]), rot], 1) / s32
    slack = np.concatenate([np.zeros((T, 512)), 2 * FP32 * mag / s32], 1) + FP32 * abs(want)
    sat = np.clip(want, -448, 448)
    assert np.isfinite(got).all()
    assert (abs(got - sat) <= E4M3 * (abs(sat) + slack) + slack + 2.0 ** -10).all()
    assert (abs(want) > 448).any() == (scale < 1)  # the small scales reach the saturated codes (448 x 0.0125 = 5.6)
    rest = torch.ones(900, dtype=torch.bool, device="cuda")
    rest[slots] = False
    assert (c["pool"][rest] == 0x11).all()


def test_e4m3_rounds_to_the_nearest_code():
    """Latent values of scale 1 against torch's own conversion of each value (exact in bf16)."""
    torch, binding = _mods()
    c = _case(64, 0, 64, seed=5, sigma=20.0)
    c["pool"] = torch.zeros((64, 576), dtype=torch.uint8, device="cuda")
    _call(binding, c, kv_scale=1.0)
    want = c["latent"].float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(c["pool"][c["slots"].long()][:, :512], want)


def test_padding_and_bad_entries():
    torch, binding = _mods()
    c = _case(40, 16, 64, context=100, seed=9)
    good = torch.ones(40, dtype=torch.bool, device="cuda")
    for at, what in ((3, "pad"), (39, "pad"), (7, "slot"), (8, "negative"), (20, "position"), (21, "below")):
        good[at] = False
        if what in ("pad", "slot", "negative"):
            c["slots"][at] = {"pad": -1, "slot": 64, "negative": -2}[what]
        else:
            c["positions"][at] = 100 if what == "position" else -1
    c["positions"][3] = 1 << 30  # a padded token's position is not looked at
    pool0, q0 = c["pool"].clone(), c["q"].clone()
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    _call(binding, c, status_word=st)
    torch.cuda.synchronize()
    assert int(st[0]) == binding.VMLA_ERR_INDEX and int(st[1]) in (7, 8, 20, 21)
    written = torch.zeros(64, dtype=torch.bool, device="cuda")
    written[c["slots"][good].long()] = True
    assert torch.equal(c["pool"][~written].view(torch.int16), pool0[~written].view(torch.int16))
    assert torch.equal(c["q"][~good].view(torch.int16), q0[~good].view(torch.int16))
    cs = _f64(c["table"])[c["positions"][good].cpu().numpy()]
    want, mag = _rot(_f64(c["k_rope"][good]), cs, True)
    assert _near_bf16(_f64(c["pool"][c["slots"][good].long()][:, 512:]), want, mag).all()
    want, mag = _rot(_f64(c["q_rope"][good]), cs[:, None], True)
    assert _near_bf16(_f64(c["q"][good][..., 512:]), want, mag).all()
    # only padding: no error, nothing written
    c["slots"].fill_(-1)
    pool0 = c["pool"].clone()
    st.zero_()
    _call(binding, c, status_word=st)
    torch.cuda.synchronize()
    assert st.tolist() == [0, 0] and torch.equal(c["pool"].view(torch.int16), pool0.view(torch.int16))


def test_queries_in_place():
    """q_rope as q's own last columns gives the same bits as a separate array."""
    torch, binding = _mods()
    for inter in (True, False):
        c = _case(50, 40, 64, seed=3)
        c["q"][..., 512:] = c["q_rope"]
        d = {**c, "q": c["q"].clone(), "pool": c["pool"].clone()}
        _call(binding, c, interleaved=inter)
        d["q_rope"] = d["q"][..., 512:]
        _call(binding, d, interleaved=inter)
        torch.cuda.synchronize()
        assert torch.equal(c["q"].view(torch.int16), d["q"].view(torch.int16))


def test_strided_queries_heads_first():
    """q_rope [H, T, 64] seen as [T, H, 64], and a projection's columns with a gap between heads."""
    torch, binding = _mods()
    c = _case(33, 12, 64, seed=4)
    ref = {**c, "q": c["q"].clone(), "pool": c["pool"].clone()}
    _call(binding, ref)
    for alt in (c["q_rope"].transpose(0, 1).contiguous().transpose(0, 1),
                torch.nn.functional.pad(c["q_rope"], (128, 0))[..., 128:]):
        assert not alt.is_contiguous()
        d = {**c, "q": c["q"].clone(), "pool": c["pool"].clone(), "q_rope": alt}
        _call(binding, d)
        torch.cuda.synchronize()
        assert torch.equal(d["q"].view(torch.int16), ref["q"].view(torch.int16))


def test_far_slots_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the last slots' rows land there."""
    torch, binding = _mods()
    slots = 4_000_000  # 4.6 GB
    c = _case(5, 0, 64, seed=6)
    c["pool"] = torch.zeros((slots, 576), dtype=torch.bfloat16, device="cuda")
    c["slots"] = torch.tensor([slots - 1, slots - 2, 3_800_000, 1, 0], dtype=torch.int32, device="cuda")
    _call(binding, c)
    torch.cuda.synchronize()
    assert torch.equal(c["pool"][c["slots"].long()][:, :512].view(torch.int16), c["latent"].contiguous().view(torch.int16))
    assert int((c["pool"][:, 0] != 0).sum()) <= 5


def test_captured_and_on_another_stream():
    torch, binding = _mods()
    c = _case(20, 16, 256, seed=8)
    ref = {**c, "q": c["q"].clone(), "pool": c["pool"].clone()}
    _call(binding, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    _call(binding, {**c, "pool": c["pool"].clone(), "q": c["q"].clone()})
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        _call(binding, c)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c["pool"].view(torch.int16), ref["pool"].view(torch.int16))
    assert torch.equal(c["q"].view(torch.int16), ref["q"].view(torch.int16))
    # new positions and slots are read at the replay
    c["positions"].copy_(c["positions"].flip(0))
    c["slots"].copy_(c["slots"].flip(0))
    ref = {**c, "q": ref["q"], "pool": c["pool"].clone()}
    graph.replay()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        _call(binding, ref)
    torch.cuda.synchronize()
    assert torch.equal(c["pool"].view(torch.int16), ref["pool"].view(torch.int16))
    assert torch.equal(c["q"].view(torch.int16), ref["q"].view(torch.int16))


def test_rows_feed_the_verify_call():
    """Appended bf16 and e4m3 rows are what the verify calls read: same bits as on a pool written by torch."""
    torch, binding = _mods()
    from speculative_decoding_mla_gb300 import device, synth
    case = synth.make_case("append_feed", [300, 90], [4, 1], num_heads=16, pool_slots=512, seed=3)
    dc = device.to_device(case)
    out0, lse0, _ = device.run(dc)
    table = torch.zeros((8, 64), device="cuda")
    table[:, :32] = 1.0  # no turn: the rows are stored as they are
    idx = dc.kv_indices.long()
    pool = torch.zeros_like(dc.kv_pool)
    rows = dc.kv_pool[idx].contiguous()
    pos = torch.zeros(idx.numel(), dtype=torch.int32, device="cuda")
    binding.verify_attn_mla_append(rows[:, :512], rows[:, 512:], pos, dc.kv_indices, table, pool)
    dc.kv_pool = pool
    out1, lse1, ws = device.run(dc)
    assert binding.verify_attn_mla_check(ws) == 0
    assert torch.equal(out0.view(torch.int16), out1.view(torch.int16)) and torch.equal(lse0, lse1)


def test_binding_refuses_mismatched_arrays():
    torch, binding = _mods()
    c = _case(4, 8, 64)
    for key, bad in (("latent", c["latent"][:, :504]), ("k_rope", c["k_rope"][:3]), ("positions", c["positions"][:2]),
                     ("slots", c["slots"].long()), ("table", c["table"][:, :32].contiguous()), ("pool", c["pool"][:, :512]),
                     ("q", c["q"][..., :512].contiguous()), ("q_rope", c["q_rope"].float()), ("latent", c["latent"].t())):
        with pytest.raises(ValueError):
            _call(binding, {**c, key: bad})
    with pytest.raises(ValueError):
        _call(binding, c, status_word=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        _call(binding, c, kv_scale=0.1)  # an e4m3 pool has one-byte elements


@pytest.mark.parametrize("scale", [1.0, 0.1, 3.0, 0.0333333, 1e-4, 7.7e3, 2.0 ** -60, 2.0 ** 60, 1e-25, 1e-38, 1e25, 3e38])
def test_e4m3_quotients_are_rounded_as_a_division_rounds(scale):
    """Every bf16 pattern but NaN, divided in float32 (one rounding) and converted (another): the same codes, also for
    zeros' signs, infinities, subnormal values and scales at the ends of the range."""
    torch, binding = _mods()
    c = _case(128, 0, 128, seed=6)
    every = torch.arange(65536, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(128, 512)
    c["latent"] = torch.where(every.isnan(), torch.zeros_like(every), every).contiguous()
    c["pool"] = torch.zeros((128, 576), dtype=torch.uint8, device="cuda")
    _call(binding, c, kv_scale=scale)
    s32 = np.float32(scale)
    with np.errstate(over="ignore", under="ignore"):
        q = c["latent"].float().cpu().numpy() / s32
    want = torch.from_numpy(np.clip(q, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(c["pool"][c["slots"].long()][:, :512].cpu(), want)
