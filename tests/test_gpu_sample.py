"""Sampling on the GPU against its definition in 64 bits: tokens are whole numbers and have to be equal.

A weight of the kernel is good to 2^-37, a 64-bit reference to 2^-52, so the two can differ only where u times
the mass (or p times the mass) falls within about 2^-37 of one of the running sums: once in some 10^6 rows of
10^5 tokens.  Where a test puts it exactly on a border, the weights are equal and both sides' sums exact."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _mods():
    import torch
    from speculative_decoding_mla_gb300 import build as vbuild
    vbuild.build()
    from speculative_decoding_mla_gb300 import binding
    return torch, binding


def reference(x, u, temp=None, top_k=None, top_p=None, min_p=None):
    """The definition, row by row, in 64 bits (numpy)."""
    R, V = x.shape
    out = np.full(R, -1, np.int32)
    for r in range(R):
        z = np.where(np.isnan(x[r]), -np.inf, x[r].astype(np.float64))
        t = 1.0 if temp is None else float(temp[r])
        m = z.max()
        if m == -np.inf:
            continue
        if t == 0:
            out[r] = int(np.argmax(z))
            continue
        if m == np.inf:
            z, m = np.where(z == np.inf, 0.0, -np.inf), 0.0
        w = np.exp((z - m) / t)
        w[w < 2.0 ** -46] = 0.0
        order = np.argsort(-z, kind="stable")
        n = V
        if top_k is not None and 0 < top_k[r] < V:
            n = int(top_k[r])
        if top_p is not None and top_p[r] < 1:
            c = np.cumsum(w[order[:n]])
            n = min(n, 1 + int(np.searchsorted(c, float(top_p[r]) * c[-1], side="left")))
        keep = np.zeros(V, bool)
        keep[order[:n]] = True
        if min_p is not None:
            keep &= w >= float(min_p[r])
        c = np.cumsum(np.where(keep, w, 0.0))
        out[r] = min(int(np.searchsorted(c, float(u[r]) * c[-1], side="right")), int(np.searchsorted(c, c[-1], side="left")))
    return out


def draw(x, u, fp32=None, status=None, **k):
    """Tokens of the kernel for host arrays (or a device tensor of logits)."""
    torch, binding = _mods()
    if isinstance(x, np.ndarray):
        x = torch.from_numpy(x.astype(np.float32)).cuda()
        x = x if fp32 else x.to(torch.bfloat16)
    dev = lambda a, t: None if a is None else torch.from_numpy(np.ascontiguousarray(a, t)).cuda()  # noqa: E731
    tok = torch.full((x.shape[0],), -7, dtype=torch.int32, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    binding.verify_attn_mla_sample(x, dev(u, np.float32), tok, temperature=dev(k.get("temp"), np.float32),
                                   top_k=dev(k.get("top_k"), np.int32), top_p=dev(k.get("top_p"), np.float32),
                                   min_p=dev(k.get("min_p"), np.float32), status_word=st)
    torch.cuda.synchronize()
    if status is None:
        assert st.tolist() == [0, 0]
    else:
        status.extend(st.tolist())
    return tok.cpu().numpy()


def host(x, fp32):
    """Logits as the kernel sees them, in fp32."""
    import torch
    t = torch.from_numpy(x.astype(np.float32))
    return (t if fp32 else t.to(torch.bfloat16)).float().numpy()


def settings(rng, R, V):
    f32 = lambda a: np.asarray(a, np.float32)  # noqa: E731
    temp = f32(rng.uniform(0.3, 2.0, R))
    temp[rng.random(R) < 0.15] = 0
    return dict(temp=temp, top_k=np.where(rng.random(R) < 0.4, 0, rng.integers(1, 2 * V + 2, R) if V < 60 else rng.integers(1, 200, R)).astype(np.int32),
                top_p=f32(np.where(rng.random(R) < 0.4, 1, rng.uniform(0.05, 1, R))), min_p=f32(np.where(rng.random(R) < 0.4, 0, rng.uniform(0, 0.3, R))))


def logits(rng, R, V, sigma=2.5):
    x = rng.normal(0, sigma, (R, V))
    for r in range(R):
        at = rng.integers(0, V, max(1, V // 200) if V < 4000 else 20)
        x[r, at] += rng.uniform(3, 12, len(at))
    return x


FILTERS = [(), ("top_k",), ("top_p",), ("min_p",), ("top_k", "top_p"), ("top_k", "top_p", "min_p")]


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 50, 1000, 4095, 4096, 4097, 8200, 33000])
def test_every_filter(V, fp32):
    rng = np.random.default_rng(V + fp32)
    R = 40 if V <= 8200 else 24
    for on in FILTERS:
        x, s, u = logits(rng, R, V), settings(rng, R, V), rng.random(R).astype(np.float32)
        k = {n: s[n] for n in ("temp",) + on}
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), on


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R,V", [(200, 131072), (9, 262144), (1, 200003), (400, 20011)])
def test_large_vocabularies(R, V, fp32):
    rng = np.random.default_rng(R)
    for on in (("top_k", "top_p", "min_p"), ("top_p",), ()):
        x, s, u = rng.normal(0, 2, (R, V)).astype(np.float32), settings(rng, R, V), rng.random(R).astype(np.float32)
        x[:, ::5003] += 9
        k = {n: s[n] for n in ("temp",) + on}
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), on


def test_without_settings_the_temperature_is_one():
    rng = np.random.default_rng(3)
    x, u = logits(rng, 30, 5000), rng.random(30).astype(np.float32)
    assert np.array_equal(draw(x, u, True), reference(host(x, True), u))


@pytest.mark.parametrize("fp32", [False, True])
def test_ties_at_every_cut(fp32):
    """Logits of a few whole values: cuts fall among equal tokens, of which the lowest indexes stay."""
    rng = np.random.default_rng(8)
    for V, values in ((300, 4), (5000, 3), (40000, 2), (70000, 6)):
        R = 30
        x = rng.integers(-values, 1, (R, V)).astype(np.float64)
        s = settings(rng, R, V)
        s["top_k"] = rng.integers(1, V, R).astype(np.int32)
        for on in FILTERS[1:]:
            u = rng.random(R).astype(np.float32)
            k = {n: s[n] for n in ("temp",) + on}
            assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), (V, on)


def test_equal_logits_on_the_borders():
    """All weights equal: sums are whole multiples, and u or p on a border decides as defined on both sides."""
    for V in (8, 64, 4096, 65536):
        R = 64
        x = np.full((R, V), -3.25)
        u = (np.arange(R) / R).astype(np.float32)
        assert np.array_equal(draw(x, u, True), (u * V).astype(np.int32))
        p = ((1 + np.arange(R)) / R).astype(np.float32)
        ones = np.full(R, 1.0, np.float32)  # the last kept token
        want = np.maximum(np.ceil(p * V), 1).astype(np.int32) - 1
        assert np.array_equal(draw(x, ones, True, top_p=p), want)
        k = np.minimum(V, 1 + np.arange(R)).astype(np.int32)
        assert np.array_equal(draw(x, ones, False, top_k=k), k - 1)


@pytest.mark.parametrize("fp32", [False, True])
def test_forbidden_and_odd_logits(fp32):
    rng = np.random.default_rng(12)
    R, V = 24, 3001
    x = logits(rng, R, V)
    x[rng.random((R, V)) < 0.5] = -np.inf
    x[rng.random((R, V)) < 0.1] = np.nan
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, 2999] = -50.0       # one token left
    x[3, [5, 77, 2000]] = np.inf
    x[4, :] = np.inf
    x[5, 9] = np.inf
    x[6] = np.where(rng.random(V) < 0.5, 0.0, -0.0)
    x[7] = -3.38e38
    x[7, 100] = 3.38e38
    x[8] *= 1e30
    x[9] = np.where(np.isnan(x[9]), np.nan, np.finfo(np.float32).min if fp32 else -3.38e38)
    s = settings(rng, R, V)
    for on in FILTERS:
        u = rng.random(R).astype(np.float32)
        k = {n: s[n] for n in ("temp",) + on}
        got, want = draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)
        assert np.array_equal(got, want), (on, np.argwhere(got != want))
        assert (got[:2] == -1).all() and got[2] == 2999 and got[5] == 9


@pytest.mark.parametrize("fp32", [False, True])
def test_far_logits_and_temperatures(fp32):
    """Values whose differences do not fit one float, and the extreme temperatures."""
    rng = np.random.default_rng(5)
    R, V = 32, 2500
    x = logits(rng, R, V, 1.0)
    x[:8] = x[:8] * 1e-4 + 1000.0 * (rng.random((8, V)) < 0.5)
    x[8:16] = x[8:16] * 1e-6 + 7.0
    x[16:24] -= 500.0
    temp = np.exp2(rng.uniform(-6, 6, R)).astype(np.float32)
    temp[::8] = 2.0 ** -20
    temp[1::8] = 2.0 ** 20
    for on in FILTERS:
        s = settings(rng, R, V)
        k = {n: s[n] for n in on}
        k["temp"] = temp
        u = rng.random(R).astype(np.float32)
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), on


@pytest.mark.parametrize("fp32", [False, True])
def test_rising_and_falling_rows(fp32):
    """Rows whose values rise or fall by hundreds along the way (weights of 2^1000 to the first ones), and rows
    that start with forbidden tokens or with values far below all others."""
    rng = np.random.default_rng(11)
    R, V = 24, 40000
    x = logits(rng, R, V)
    ramp = np.linspace(0, 3000, V)
    x[:4] += ramp
    x[4:8] -= ramp
    x[8:12] += 400.0 * (np.arange(V) // 5000)
    x[12:16, :30000] = -np.inf
    x[16:20, :30000] = -1e30 if fp32 else -3.3e38
    x[20:22, 100:] = np.nan
    u = rng.random(R).astype(np.float32)
    for temp in (None, np.full(R, 0.7, np.float32), np.exp2(rng.uniform(-9, 9, R)).astype(np.float32), np.zeros(R, np.float32)):
        k = {} if temp is None else {"temp": temp}
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k))


@pytest.mark.parametrize("rows", [63, 64, 200])
def test_undecided_rows_of_flat_logits(rows):
    """131,072 nearly equal weights: single-precision sums leave one row of ten to exact ones."""
    rng = np.random.default_rng(rows)
    x = rng.normal(0, 0.01, (rows, 131072))
    u = rng.random(rows).astype(np.float32)
    assert np.array_equal(draw(x, u, True), reference(host(x, True), u))
    s = settings(rng, rows, 131072)
    k = {n: s[n] for n in ("temp", "top_p")}
    assert np.array_equal(draw(x, u, False, **k), reference(host(x, False), u, **k))


def test_settings_at_their_ends():
    rng = np.random.default_rng(6)
    R, V = 16, 6000
    x = logits(rng, R, V)
    u = rng.random(R).astype(np.float32)
    full = lambda v, t=np.float32: np.full(R, v, t)  # noqa: E731
    best = host(x, True).argmax(1)
    assert np.array_equal(draw(x, u, True, top_k=full(1, np.int32)), best)
    assert np.array_equal(draw(x, u, True, top_p=full(1e-6)), best)
    assert np.array_equal(draw(x, u, True, min_p=full(1.0)), best)
    assert np.array_equal(draw(x, u, True, temp=full(0.0), top_k=full(5, np.int32)), best)
    plain = draw(x, u, True)
    for k in (dict(top_k=full(0, np.int32)), dict(top_k=full(-3, np.int32)), dict(top_k=full(V, np.int32)),
              dict(top_k=full(2 ** 31 - 1, np.int32)), dict(top_p=full(1.0)), dict(min_p=full(0.0)), dict(temp=full(1.0))):
        assert np.array_equal(draw(x, u, True, **k), plain), k
    for k in (dict(top_k=full(V - 1, np.int32)), dict(top_p=full(1 - 2.0 ** -24)), dict(top_p=full(0.99999)), dict(min_p=full(1e-9))):
        assert np.array_equal(draw(x, u, True, **k), reference(host(x, True), u, **k)), k


def test_rows_at_every_alignment_and_stride():
    torch, binding = _mods()
    rng = np.random.default_rng(7)
    for fp32 in (False, True):
        for V, stride in ((1001, 1001), (4096, 4099), (5000, 5008)):
            R = 17
            x = logits(rng, R, V)
            u, s = rng.random(R).astype(np.float32), settings(rng, R, V)
            buf = torch.full((R * stride + 16,), 100.0, device="cuda").to(torch.float32 if fp32 else torch.bfloat16)
            for off in (0, 1, 3, 8):
                view = buf[off:off + R * stride].view(R, stride)[:, :V]
                buf.fill_(100.0)  # what lies between the rows would win if it were read
                view.copy_(torch.from_numpy(x))
                assert np.array_equal(draw(view, u, **s), reference(host(x, fp32), u, **s)), (V, stride, off)


def test_bad_settings():
    _, binding = _mods()
    rng = np.random.default_rng(2)
    R, V = 12, 500
    x, u = logits(rng, R, V), rng.random(R).astype(np.float32)
    good = reference(host(x, True), u)
    nan = float("nan")
    for name, bads in (("temp", (-1.0, nan, np.inf, 1e-7, 2e6)), ("top_p", (0.0, -0.1, 1.5, nan)), ("min_p", (-0.1, 1.01, nan)),
                       ("u", (-0.01, 1.01, nan, np.inf))):
        for bad in bads:
            k = {} if name == "u" else {name: np.full(R, 0.0 if name == "min_p" else 1.0, np.float32)}
            v = u.copy()
            (v if name == "u" else k[name])[5] = bad
            st = []
            got = draw(x, v, True, status=st, **k)
            assert st == [np.int32(binding.VMLA_ERR_PARAM), 5], (name, bad)
            assert got[5] == -1 and np.array_equal(np.delete(got, 5), np.delete(good, 5))


def test_captured_two_streams_and_repeated():
    torch, binding = _mods()
    rng = np.random.default_rng(4)
    R, V = 20, 30000
    x, u = logits(rng, R, V), rng.random(R).astype(np.float32)
    k = {n: v for n, v in settings(rng, R, V).items()}
    d = torch.from_numpy(x.astype(np.float32)).cuda()
    ud = torch.from_numpy(u).cuda()
    dev = {n: torch.from_numpy(v).cuda() for n, v in k.items()}
    names = dict(temperature=dev["temp"], top_k=dev["top_k"], top_p=dev["top_p"], min_p=dev["min_p"])
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    call = binding.prepare_verify_attn_mla_sample(d, ud, tok, **names)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        binding.verify_attn_mla_sample(d, ud, tok, **names)
    x2, u2 = logits(rng, R, V), rng.random(R).astype(np.float32)
    d.copy_(torch.from_numpy(x2))
    ud.copy_(torch.from_numpy(u2))
    g.replay()
    torch.cuda.synchronize()
    want = reference(host(x2, True), u2, **k)
    assert np.array_equal(tok.cpu().numpy(), want)
    toks = [torch.zeros(R, dtype=torch.int32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for t, s in zip(toks, streams):
            binding.verify_attn_mla_sample(d, ud, t, stream=s, **names)
    torch.cuda.synchronize()
    for t in toks:
        assert np.array_equal(t.cpu().numpy(), want)


@pytest.mark.parametrize("fp32", [False, True])
@pytest.mark.parametrize("R", [160, 12])
def test_rows_whose_first_logits_mislead(R, fp32):
    """Bins are counted from the largest of the logits that a warp loads first: rows whose maximum is far above those, rows
    with nothing but -inf (or NaN, or large negative numbers) there, rows of values next to zero and of one value."""
    rng = np.random.default_rng(R + fp32)
    V = 100003
    x = rng.normal(0, 2, (R, V)).astype(np.float32)
    for r in range(R):
        at = rng.integers(0, V, 30)
        kind = r % 8
        if kind == 0:
            x[r, at] = rng.uniform(30, 60, 30)
        elif kind == 1:
            keep = x[r, at].copy()
            x[r] = -np.inf
            x[r, at] = keep
        elif kind == 2:
            x[r, :-5000] = np.where(rng.random(V - 5000) < 0.5, np.nan, -np.inf)
        elif kind == 3:
            x[r] = -1e30
            x[r, at] = rng.normal(0, 2, 30)
        elif kind == 4:
            x[r] = rng.uniform(-2.0 ** -10, 2.0 ** -10, V)
        elif kind == 5:
            x[r] = rng.uniform(-2.0 ** -9, 2.0 ** -9, V)
        elif kind == 6:
            x[r, -300:] += 25
        else:
            x[r] = -7.25
            x[r, at[0]] = rng.uniform(-7, 7)
    for on in (("top_p",), ("top_k", "top_p", "min_p"), ("top_k",)):
        s, u = settings(rng, R, V), rng.random(R).astype(np.float32)
        s["top_k"] = np.where(rng.random(R) < 0.5, rng.integers(1, 200, R), rng.integers(1, V, R)).astype(np.int32)
        k = {n: s[n] for n in on}
        assert np.array_equal(draw(x, u, fp32, **k), reference(host(x, fp32), u, **k)), on


@pytest.mark.parametrize("R", [150, 3])
def test_cuts_away_from_the_bins_middles(R):
    """Values at the ends of their bins, so that the bins' middle values place top-p's cut some bins above or below the
    bin that it is in: widths are w = 2^-4 at 8 to 16, T = w; a token at 8 + 20 w, many just below 8 + 19 w (or above
    8 + 18 w), more just above 8 + 15 w (or below 8 + 16 w)."""
    rng = np.random.default_rng(R)
    V, w = 60000, 2.0 ** -4
    for low_then_high in (True, False):
        n_b, n_c = (1000, 50000) if low_then_high else (2000, 20000)
        x = np.full((R, V), -30.0, np.float32)
        for r in range(R):
            at, jitter = rng.permutation(V), rng.uniform(0.001, 0.02, V) * w
            x[r, at[0]] = 8 + 20 * w
            x[r, at[1:1 + n_b]] = (8 + 19 * w - jitter[:n_b]) if low_then_high else 8 + 18 * w + jitter[:n_b]
            c = at[1 + n_b:1 + n_b + n_c]
            x[r, c] = (8 + 15 * w + jitter[:n_c]) if low_then_high else 8 + 16 * w - jitter[:n_c]
        p = rng.uniform(0.49, 0.51, R) if low_then_high else rng.uniform(0.5, 0.6, R)
        k = dict(temp=np.full(R, w, np.float32), top_p=p.astype(np.float32))
        u = rng.random(R).astype(np.float32)
        assert np.array_equal(draw(x, u, True, **k), reference(x, u, **k)), low_then_high
        k["top_k"] = rng.integers(n_b + 10000, V, R).astype(np.int32)
        assert np.array_equal(draw(x, u, True, **k), reference(x, u, **k)), low_then_high
