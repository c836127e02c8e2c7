"""token_logprobs and token_logprobs_backward against their definitions in 64 bits.

Tolerances, from the operations' roundings (u = 2^-24): an exponent t = (z - m) s log2(e)
carries at most 3 u |t|, exp2 another 2^-22, and the sum of the terms that matter has
|t| < 40, so every term of R is within 40 * 3 u + 2^-22 < 8e-6 of its value, relatively; the
accumulation of positive terms adds less than 2e-6 (at most 32 additions a thread, then
trees).  So R, and with it log_sum = log1p(R) and the entropy (a sum of positive terms, each
a multiple of such a term), are within REL = 1e-5 relatively; log p adds the roundings of x
and of one subtraction.  A gradient's factor p has log2 p with the same error again, so its
terms are within 2 REL of their sizes, plus the one rounding to the output's type.
"""
import math

import pytest
import torch

import embedding_weight_grad_gb300 as ewg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
REL = 1e-5
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def make(n, V, dtype, seed=0, pad=0, std=3.0, lift=12.0):
    """Logits whose token is anything from unlikely to near certain."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.randn(n, V, generator=g, device=DEV) * std
    t = torch.randint(V, (n,), generator=g, device=DEV)
    z[torch.arange(n, device=DEV), t] += torch.rand(n, generator=g, device=DEV) * lift
    buf = torch.full((n, V + pad), float("nan"), dtype=dtype, device=DEV)
    buf[:, :V] = z.to(dtype)
    return buf[:, :V], t


def reference(z, t, scale):
    """logprobs, entropy, R, log_sum, row_max and all log p of rows with a finite logit, in 64 bits."""
    z = z.double()
    m = z.amax(1)
    x = (z - m[:, None]) * scale
    e = x.exp().scatter(1, z.argmax(1, keepdim=True), 0.0)
    R = e.sum(1)
    log_sum = R.log1p()
    logp = x - log_sum[:, None]
    xe = torch.where(e > 0, e * x, 0.0).sum(1)
    return logp.gather(1, t.clamp_min(0).long()[:, None])[:, 0], log_sum - xe / (1 + R), R, log_sum, m, logp


def check_forward(z, t, scale, top, r):
    logp, entropy, R, log_sum, m, all_logp = reference(z, t, scale)
    share = R / (1 + R)

    def near(got, want, tol, what):
        worst = ((got.double() - want).abs() - tol).max().item()
        assert worst <= 0, (what, worst)
    assert torch.equal(r.row_max.double(), m)
    near(r.log_sum, log_sum, REL * share + 4 * U * log_sum, "log_sum")
    near(r.entropy, entropy, 1.5 * REL * entropy + 1e-38, "entropy")
    near(r.logprobs, logp, REL * share + 6 * U * logp.abs(), "logprobs")
    if top:
        best, ids = order(z, top)
        assert torch.equal(r.top_ids, ids)
        want = all_logp.gather(1, ids.clamp_min(0))
        near(torch.where(ids >= 0, r.top_logprobs, 0.0), torch.where(ids >= 0, want, 0.0),
             REL * share[:, None] + torch.where(ids >= 0, 6 * U * want.abs(), 0.0), "top")
        assert bool((r.top_logprobs[ids < 0] == -math.inf).all())


def order(z, top):
    """The `top` largest by a stable sort (equal logits by lower id); id -1 past the finite ones."""
    v, ids = torch.sort(z.double() + 0.0, dim=1, descending=True, stable=True)
    v, ids = v[:, :top], ids[:, :top]
    return v, torch.where(v > -math.inf, ids, -1)


def check_backward(z, t, scale, G, E, got):
    """Rows with a token and a finite logit."""
    logp, entropy, R, log_sum, m, all_logp = reference(z, t, scale)
    p = all_logp.exp()
    q = p.scatter(1, t.long()[:, None], logp.expm1()[:, None])
    plogp = torch.where(p > 0, p * all_logp, 0.0)
    want = -G.double()[:, None] * q
    size = G.double().abs()[:, None] * q.abs()
    if E is not None:
        want = want - E.double()[:, None] * (plogp + p * entropy[:, None])
        size = size + E.double().abs()[:, None] * (plogp.abs() + p * entropy[:, None])
    tol = scale * (2 * REL * size) + 1e-37
    if got.dtype == BF16:
        tol = tol + scale * want.abs() * 2.0 ** -8
    worst = ((got.double() - scale * want).abs() - tol).max().item()
    assert worst <= 0, worst


def both(z, t, scale=1.0, top=0, entropy=True, seed=3):
    r = ewg.token_logprobs(z, t, scale=scale, top=top, check=True)
    check_forward(z, t, scale, top, r)
    g = torch.Generator(device=DEV).manual_seed(seed)
    G = torch.randn(t.shape, generator=g, device=DEV)
    E = torch.randn(t.shape, generator=g, device=DEV) if entropy else None
    got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, entropy=r.entropy,
                                      grad_entropy=E, scale=scale, check=True)
    check_backward(z, t, scale, G, E, got)
    return r, got


SIZES = [(1, 1), (1, 2), (3, 7), (5, 31), (2, 33), (9, 63), (33, 257), (300, 1000), (17, 2047), (7, 4099),
         (200, 12345), (160, 16400), (3, 50257), (1, 129280), (2, 129283), (700, 300), (1, 256000)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,V", SIZES)
def test_sizes(n, V, dtype):
    z, t = make(n, V, dtype, seed=n + V)
    both(z, t, top=min(V, 5))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,V,top", [(2500, 1111, 4), (2432, 4101, 3), (2432, 8200, 3), (160, 8300, 7), (160, 33001, 7),
                                     (151, 33001, 7), (76, 66000, 2), (38, 140001, 9), (2432, 102403, 0), (2432, 30003, 1),
                                     (2432, 102403, 1)])
def test_many_rows(n, V, top, dtype):
    """Rows enough to fill the device: other shares of a row for a thread."""
    z, t = make(n, V, dtype, seed=n + V, pad=V % 2)
    r = ewg.token_logprobs(z, t, scale=0.9, top=top)
    for i in range(0, n, 256):                   # the 64-bit reference in pieces
        part = ewg.TokenLogprobs(*(x if x is None else x[i:i + 256] for x in r))
        check_forward(z[i:i + 256], t[i:i + 256], 0.9, top, part)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad", [0, 1, 3])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 15, 33, 64, 100, 255, 257, 300, 511, 512, 513, 1000, 1024, 1031, 1500,
                               2047, 2048, 2056])
def test_short_rows(V, pad, dtype):
    """Rows held in registers, several to a warp."""
    for n in (1, 3, 333):
        for std, lift in ((3.0, 12.0), (0.1, 0.0), (3.0, 40.0)):
            z, t = make(n, V, dtype, seed=n + V, pad=pad, std=std, lift=lift)
            both(z, t, scale=0.8)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [3, 50, 200, 400, 513, 1001, 2003])
def test_short_rows_of_every_kind(V, dtype):
    """Without alternatives short rows go another way than with them: results agree to the
    tolerance of either, NaN and infinities alike."""
    z, t = make(96, V, dtype, seed=V, pad=1)
    n = torch.arange(96, device=DEV)
    t[n % 8 == 1] = -1
    t[n % 8 == 2] = V + 3
    z[n % 8 == 3] = -math.inf
    z[4::8, 1:] = -math.inf                          # one token left
    z[5::8, 0] = z[5::8].amax(1)                     # the maximum twice, once at the row's edge
    z[6::8, V - 1] = 50.0
    z[6::8, V // 2] = 50.0
    z[7, V // 2] = math.nan
    z[15, 0] = math.inf
    z[23] = torch.finfo(dtype).min                   # a mask of the lowest value everywhere
    z[31, 1:] = torch.finfo(dtype).min
    a, b = ewg.token_logprobs(z, t, scale=1.3), ewg.token_logprobs(z, t, scale=1.3, top=1)
    for x, y in zip(a[:4], b[:4]):
        torch.testing.assert_close(x, y, rtol=2 * REL, atol=1e-37, equal_nan=True)
    assert torch.equal(a.row_max.nan_to_num(7.0), b.row_max.nan_to_num(7.0))


@pytest.mark.parametrize("n,V,top", [(36000, 65000, 2), (2400000, 1001, 0), (17, 140000000, 3)])
def test_offsets_beyond_32_bits(n, V, top):
    """More than 2^31 logits: the last rows of a large array, forward and in place backward."""
    z = torch.full((n, V), -3.0, dtype=BF16, device=DEV)
    last = 3
    part, t_part = make(last, V, BF16, seed=V)
    z[-last:] = part
    t = torch.zeros(n, dtype=torch.int64, device=DEV)
    t[-last:] = t_part
    r = ewg.token_logprobs(z, t, top=top, check=True)
    tail = ewg.TokenLogprobs(*(x if x is None else x[-last:] for x in r))
    check_forward(part, t_part, 1.0, top, tail)
    G = torch.ones(n, device=DEV)
    got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, out=z, check=True)
    check_backward(part, t_part, 1.0, G[-last:], None, got[-last:])


@pytest.mark.parametrize("low", [-0.37, -1.7, -6.1])
@pytest.mark.parametrize("n,V", [(2, 40), (2432, 4096), (2432, 200000), (1, 200000), (2, 1000000)])
def test_equal_terms(n, V, low):
    """All terms of R but the target's are equal, so that roundings of a running sum may all fall
    to one side: a thread adds at most 4 a vector, 400 of them at most, each with u of the
    sum.  Relative errors: 400 u = 2.4e-5 and REL of the terms."""
    z = torch.full((n, V), low, device=DEV, dtype=BF16)
    z[:, V // 2] = 1.0
    t = torch.full((n,), V // 3, device=DEV)
    r = ewg.token_logprobs(z, t)
    x = z[0, 0].double() - 1.0
    R = (V - 1) * x.exp()
    log_sum = R.log1p()
    entropy = log_sum - R * x / (1 + R)
    tol = (400 * U + REL) * R / (1 + R)
    assert bool(((r.log_sum - log_sum).abs() <= tol + 4 * U * log_sum).all())
    assert bool(((r.logprobs - (x - log_sum)).abs() <= tol + 6 * U * (x - log_sum).abs()).all())
    assert bool(((r.entropy - entropy).abs() <= tol * (1 - x) + 4 * U * (log_sum + x.abs())).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad", [1, 2, 3, 5, 8, 40])
def test_row_strides(dtype, pad):
    """Rows of a wider buffer (NaN between them): every alignment of a row."""
    for n, V in [(9, 1001), (5, 20011)]:
        z, t = make(n, V, dtype, seed=pad, pad=pad)
        r, got = both(z, t, scale=0.7, top=3)
        # a gradient of another alignment than the logits: the same numbers
        for gpad in (0, 1, 4):
            out = torch.full((n, V + gpad), 7.0, dtype=dtype, device=DEV)
            G = torch.ones(n, device=DEV)
            a = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, scale=0.7)
            b = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, scale=0.7, out=out[:, :V])
            assert torch.equal(a, b)
            assert bool((out[:, V:] == 7.0).all())


@pytest.mark.parametrize("top", [1, 2, 20, 32])
@pytest.mark.parametrize("n,V", [(40, 33), (6, 5000), (2, 70000), (170, 9000)])
@pytest.mark.parametrize("kind", ["equal", "ties", "rising", "falling", "zeros of both signs"])
def test_alternatives_order(top, n, V, kind):
    g = torch.Generator(device=DEV).manual_seed(V)
    z = {"equal": lambda: torch.full((n, V), 1.5, device=DEV),
         "ties": lambda: torch.randint(-3, 4, (n, V), generator=g, device=DEV).float(),
         "rising": lambda: torch.arange(V, device=DEV).float().expand(n, V) * 2.0 ** -6,
         "falling": lambda: -torch.arange(V, device=DEV).float().expand(n, V) * 2.0 ** -6,
         "zeros of both signs": lambda: torch.where(torch.rand(n, V, generator=g, device=DEV) < 0.5, 0.0, -0.0)}[kind]()
    for dtype in (BF16, FP32):
        zz = z.to(dtype).contiguous()
        t = torch.randint(V, (n,), generator=g, device=DEV)
        check_forward(zz, t, 1.0, top, ewg.token_logprobs(zz, t, top=top, check=True))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("V", [50, 3001, 30000, 140000])
def test_masks(dtype, V):
    """Tokens that cannot occur, masked with -inf and with the type's lowest value."""
    z, t = make(12, V, dtype, seed=V)
    z = z.clone()
    g = torch.Generator(device=DEV).manual_seed(1)
    keep = torch.rand(12, V, generator=g, device=DEV) < 0.1
    keep.scatter_(1, t[:, None], True)
    z[:6] = torch.where(keep[:6], z[:6], -math.inf)
    z[6:] = torch.where(keep[6:], z[6:], torch.finfo(dtype).min)
    z[0] = -math.inf
    z[0, t[0]] = 2.0                                     # one token is left: certain
    z[6] = torch.finfo(dtype).min                        # all at the lowest value: uniform
    r, got = both(z, t, top=8)
    assert r.logprobs[0] == 0 and r.entropy[0] == 0
    assert int((r.top_ids[0] >= 0).sum()) == 1
    assert bool((got[0] == 0).all())
    assert abs(r.entropy[6].item() - math.log(V)) < 1e-5 * math.log(V)


@pytest.mark.parametrize("V", [40, 5000, 130000])
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_rows_without_anything(dtype, V):
    """A row of -inf only, and padding rows whose logits are NaN."""
    z, t = make(5, V, dtype)
    z = z.clone()
    z[1] = -math.inf
    z[3] = math.nan
    t[3] = -100
    r = ewg.token_logprobs(z, t, top=4, check=True)
    assert r.logprobs[1] == -math.inf and r.row_max[1] == -math.inf
    assert r.entropy[1] == 0 and r.log_sum[1] == 0
    assert r.logprobs[3] == 0 and r.entropy[3] == 0 and r.row_max[3] == 0 and r.log_sum[3] == 0
    for row in (1, 3):
        assert bool((r.top_ids[row] == -1).all()) and bool((r.top_logprobs[row] == -math.inf).all())
    ones = torch.ones(5, device=DEV)
    got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, ones, entropy=r.entropy,
                                      grad_entropy=ones, check=True)
    assert bool((got[1] == 0).all()) and bool((got[3] == 0).all())
    rest = [0, 2, 4]
    check_forward(z[rest], t[rest], 1.0, 4, type(r)(*(x[rest] for x in r)))
    check_backward(z[rest], t[rest], 1.0, ones[rest], ones[rest], got[rest])


@pytest.mark.parametrize("V", [40, 5000, 130000])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nan_and_infinity_show(V, bad):
    for where in (0, V // 2, V - 1):
        z, t = make(2, V, FP32)
        z = z.clone()
        z[0, where] = bad
        r = ewg.token_logprobs(z, t, top=2, check=True)
        assert math.isnan(r.logprobs[0]) and math.isnan(r.entropy[0]) and math.isnan(r.log_sum[0])
        got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, torch.ones(2, device=DEV))
        assert bool(got[0].isnan().any())
        check_forward(z[1:], t[1:], 1.0, 2, type(r)(*(x[1:] for x in r)))


@pytest.mark.parametrize("V", [64, 2000, 40000, 200000])
def test_near_certain_rows_keep_their_digits(V):
    """One logit 10 to 60 above the others: log p, entropy and gradient of about exp(-10) to exp(-60)."""
    for where in (0, 1, V // 3, V - 1):
        g = torch.Generator(device=DEV).manual_seed(where)
        z = torch.randn(6, V, generator=g, device=DEV)
        z[:, where] = torch.tensor([14.0, 20.0, 25.0, 33.0, 50.0, 70.0], device=DEV)
        t = torch.full((6,), where, device=DEV)
        both(z, t)
        t[:] = (where + 1) % V
        both(z, t)


@pytest.mark.parametrize("scale", [0.01, 0.5, 1.0, 2.5])
def test_scale_and_large_offsets(scale):
    z, t = make(20, 4000, FP32, seed=5)
    both(z, t, scale=scale, top=2)
    # a power-of-two offset far above the spread: the same row, shifted exactly
    zb = (z * 64).round() / 64
    a, b = ewg.token_logprobs(zb, t, scale=scale), ewg.token_logprobs(zb + 4096.0, t, scale=scale)
    assert torch.equal(a.logprobs, b.logprobs) and torch.equal(a.entropy, b.entropy)


def test_shapes_and_target_types():
    z, t = make(6, 777, BF16, seed=9)
    r = ewg.token_logprobs(z, t, top=3)
    r3 = ewg.token_logprobs(z.view(2, 3, 777), t.view(2, 3).int(), top=3)
    assert r3.logprobs.shape == (2, 3) and r3.top_ids.shape == (2, 3, 3)
    for a, b in zip(r, r3):
        assert torch.equal(a, b.reshape(a.shape))
    r1 = ewg.token_logprobs(z[2], t[2], top=3)           # a single row: a scalar target
    assert r1.logprobs.shape == () and torch.equal(r1.top_ids, r.top_ids[2])
    G = torch.ones(2, 3, device=DEV)
    g3 = ewg.token_logprobs_backward(z.view(2, 3, 777), t.view(2, 3).int(), r3.row_max, r3.log_sum, G)
    g = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G.view(6))
    assert g3.shape == (2, 3, 777) and torch.equal(g3.view(6, 777), g)
    g1 = ewg.token_logprobs_backward(z[2], t[2], r1.row_max, r1.log_sum, torch.ones((), device=DEV))
    assert g1.shape == (777,) and torch.equal(g1, g[2])


def test_no_rows():
    z = torch.empty(0, 100, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    r = ewg.token_logprobs(z, t, top=2, check=True)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 2)
    e = torch.empty(0, device=DEV)
    assert ewg.token_logprobs_backward(z, t, e, e, e, check=True).shape == (0, 100)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad", [0, 3])
def test_backward_in_place(dtype, pad):
    z, t = make(50, 5003, dtype, pad=pad)
    r = ewg.token_logprobs(z, t)
    G = torch.randn(50, device=DEV)
    want = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G)
    got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, out=z)
    assert got.data_ptr() == z.data_ptr() and torch.equal(z, want)


def test_backward_against_differences():
    """Central differences of the 64-bit definition (truncation ~h^2 = 1e-10)."""
    z, t = make(4, 300, FP32, seed=2, lift=4.0)
    G, E = torch.randn(4, device=DEV), torch.randn(4, device=DEV)
    r = ewg.token_logprobs(z, t, scale=1.25)
    got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, entropy=r.entropy, grad_entropy=E, scale=1.25)

    def loss(x):
        logp, entropy, *_ = reference(x, t, 1.25)
        return G.double() * logp + E.double() * entropy
    h = 1e-5
    for v in torch.cat([t, torch.arange(0, 300, 41, device=DEV)]).tolist():
        step = torch.zeros(4, 300, dtype=torch.float64, device=DEV)
        step[:, v] = h
        diff = (loss(z.double() + step) - loss(z.double() - step)) / (2 * h)
        assert ((got[:, v].double() - diff).abs() <= 4 * REL * (G.abs() + 8 * E.abs())).all()


@pytest.mark.parametrize("n,V", [(5, 100), (600, 100), (5000, 64), (3, 60000)])
@pytest.mark.parametrize("tdt", [torch.int32, torch.int64])
def test_targets_outside_the_vocabulary(n, V, tdt):
    z, t = make(n, V, FP32)
    t = t.to(tdt)
    good = ewg.token_logprobs(z, t, top=1)
    t2 = t.clone()
    t2[n - 2] = V
    ws = ewg.status_workspace()
    r = ewg.token_logprobs(z, t2, top=1, workspace=ws)
    assert ewg.read_status(ws) == ewg.ERR_ID_OUT_OF_RANGE
    assert math.isnan(r.logprobs[n - 2])
    rest = torch.arange(n, device=DEV) != n - 2
    assert torch.equal(r.logprobs[rest], good.logprobs[rest]) and torch.equal(r.entropy, good.entropy)
    G = torch.ones(n, device=DEV)
    got = ewg.token_logprobs_backward(z, t2, r.row_max, r.log_sum, G, workspace=ws)
    assert ewg.read_status(ws) == ewg.ERR_ID_OUT_OF_RANGE
    assert bool((got[n - 2] == 0).all())
    with pytest.raises(ewg.EwgError) as err:
        ewg.token_logprobs(z, t2, check=True)
    assert err.value.code == ewg.ERR_ID_OUT_OF_RANGE
    ewg.token_logprobs(z, t, workspace=ws)               # the next call's status is its own
    assert ewg.read_status(ws) == ewg.OK


def test_streams_and_graph():
    """Calls on another stream than the current one, and a captured call replayed on new logits."""
    z, t = make(64, 20000, BF16, seed=11)
    want = ewg.token_logprobs(z, t, top=4)
    G = torch.randn(64, device=DEV)
    want_g = ewg.token_logprobs_backward(z, t, want.row_max, want.log_sum, G)
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    with torch.cuda.stream(s):
        r = ewg.token_logprobs(z, t, top=4)
        g = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G)
    s.synchronize()
    for a, b in zip(want, r):
        assert torch.equal(a, b)
    assert torch.equal(g, want_g)
    src = torch.zeros_like(z)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = ewg.token_logprobs(src, t, top=4)
        g = ewg.token_logprobs_backward(src, t, r.row_max, r.log_sum, G)
    src.copy_(z)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, r):
        assert torch.equal(a, b)
    assert torch.equal(g, want_g)


def test_refusals():
    z, t = make(8, 100, FP32)
    r = ewg.token_logprobs(z, t)
    G = torch.ones(8, device=DEV)

    def no(call):
        with pytest.raises((ValueError, ewg.EwgError)):
            call()
    no(lambda: ewg.token_logprobs(z.half(), t))
    no(lambda: ewg.token_logprobs(z, t.short()))
    no(lambda: ewg.token_logprobs(z, t.float()))
    no(lambda: ewg.token_logprobs(z.cpu(), t.cpu()))
    no(lambda: ewg.token_logprobs(z, t[:4]))
    no(lambda: ewg.token_logprobs(z.t(), torch.zeros(100, dtype=torch.int64, device=DEV)))
    no(lambda: ewg.token_logprobs(z[:1].expand(8, 100), t))
    no(lambda: ewg.token_logprobs(z, torch.zeros(16, dtype=torch.int64, device=DEV)[::2]))
    no(lambda: ewg.token_logprobs(torch.empty(8, 0, device=DEV), t))
    for scale in (0.0, -1.0, math.inf, math.nan):
        no(lambda: ewg.token_logprobs(z, t, scale=scale))
    no(lambda: ewg.token_logprobs(z, t, top=33))
    no(lambda: ewg.token_logprobs(z, t, top=-1))
    no(lambda: ewg.token_logprobs(z[:, :3], t.clamp(max=2), top=4))
    no(lambda: ewg.token_logprobs(z, t, workspace=torch.empty(16, dtype=torch.uint8, device=DEV)))
    back = lambda *a, **k: ewg.token_logprobs_backward(z, t, *a, **k)
    no(lambda: back(r.row_max, r.log_sum, G.double()))
    no(lambda: back(r.row_max[:4], r.log_sum, G))
    no(lambda: back(r.row_max, r.log_sum, G, grad_entropy=G))
    no(lambda: back(r.row_max, r.log_sum, G, out=torch.empty(8, 100, dtype=BF16, device=DEV)))
    no(lambda: back(r.row_max, r.log_sum, G, out=torch.empty(8, 99, device=DEV)))
    buf = torch.zeros(9 * 100, device=DEV)
    no(lambda: ewg.token_logprobs_backward(buf[:800].view(8, 100), t, r.row_max, r.log_sum, G,
                                           out=buf[100:].view(8, 100)))      # partly the logits
    flat = torch.zeros(8 * 100 + 8, device=DEV)
    no(lambda: ewg.token_logprobs_backward(flat[:800].view(8, 100), t, r.row_max, r.log_sum, flat[796:804],
                                           out=flat[:800].view(8, 100)))     # over a gradient


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,V,top", [(8, 100, 0), (9, 1001, 0), (9, 1001, 3), (2432, 4101, 2), (9, 5003, 3), (160, 16401, 0),
                                     (9, 33001, 4), (160, 102403, 1), (1, 140001, 2), (80, 1100003, 0)])
def test_infinity_shows_at_every_alignment(n, V, top, dtype):
    """A row with +inf has NaN results wherever it stands: in the row's whole vectors or in
    the elements outside them, whether it is the row's token or not."""
    for pad, where in ((0, 0), (1, 0), (1, V - 1), (2, V - 1), (3, 1), (1, V // 2)):
        z, t = make(n, V, dtype, seed=V + where, pad=pad)
        rows = torch.arange(min(n, 16), device=DEV)
        bad = rows[rows % 2 == 0]
        z[bad, where] = math.inf
        t[bad] = torch.where(bad % 4 == 0, where, (where + 7) % V)
        r = ewg.token_logprobs(z, t, scale=0.9, top=top)
        for x in (r.logprobs, r.entropy, r.log_sum):
            assert bool(x[bad].isnan().all()), (pad, where)
        assert bool((r.row_max[bad] == math.inf).all())
        for E in (None, torch.ones(n, device=DEV)):
            got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, torch.ones(n, device=DEV), entropy=r.entropy,
                                              grad_entropy=E, scale=0.9)
            assert bool(got[bad].isnan().all()), (pad, where)
        good = rows[rows % 2 == 1]
        if len(good):
            check_forward(z[good], t[good], 0.9, top, type(r)(*(x if x is None else x[good] for x in r)))


@pytest.mark.parametrize("V,top", [(100, 0), (1001, 1), (50000, 2)])
@pytest.mark.parametrize("scale", [2.3e38, 2.4e38, 3.4e38])
def test_largest_scales(scale, V, top):
    """A scale of nearly the largest number (times log2(e) it would not be one): all the weight is
    on the largest logit, shared where it occurs twice."""
    for dtype in (BF16, FP32):
        z = (torch.arange(V, device=DEV) % 17).float().neg().expand(2, V).contiguous()
        z[:, 17::17] = -20.0                             # 0 is left the only largest ...
        z[1, V - 1] = 0.0                                # ... and has company
        z, t = z.to(dtype), torch.zeros(2, dtype=torch.int64, device=DEV)
        r = ewg.token_logprobs(z, t, scale=scale, top=top)
        want = torch.tensor([0.0, math.log(2.0)], device=DEV)
        for x in (-r.logprobs, r.log_sum, r.entropy):
            assert bool(((x - want).abs() <= 4 * U).all()), x
        if top:
            assert torch.equal(r.top_ids[:, 0], t)
        got = ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, torch.full((2,), 2.0 ** -100, device=DEV),
                                          scale=scale)
        half = scale * 2.0 ** -101
        assert bool((got[0] == 0).all())
        assert abs(got[1, 0].item() - half) <= 2.0 ** -8 * half and abs(got[1, V - 1].item() + half) <= 2.0 ** -8 * half
        assert bool((got[1, 1:V - 1] == 0).all())


def test_autograd_is_told_of_logits_replaced():
    """A graph that saved the logits raises once the gradient has been written over them."""
    x = torch.randn(4, 50, device=DEV, requires_grad=True)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    G = torch.ones(4, device=DEV)
    z = x * 1.0
    saved = (z * z).sum()
    r = ewg.token_logprobs(z, t)
    assert not any(y.requires_grad for y in r if y is not None)
    version = z._version
    ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G)           # to a tensor of its own
    assert z._version == version
    ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, out=z)
    assert z._version > version
    with pytest.raises(RuntimeError, match="inplace"):
        saved.backward()
    with torch.inference_mode():                                          # tensors without a count
        z = torch.randn(4, 50, device=DEV)
        r = ewg.token_logprobs(z, t)
        ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, out=z)


def test_as_an_autograd_function():
    """The two calls as the halves of a function: the gradient of log_softmax in 64 bits."""
    class Logprobs(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, targets):
            r = ewg.token_logprobs(logits, targets)
            ctx.save_for_backward(logits, targets, r.row_max, r.log_sum)
            return r.logprobs

        @staticmethod
        def backward(ctx, grad):
            logits, targets, row_max, log_sum = ctx.saved_tensors
            return ewg.token_logprobs_backward(logits, targets, row_max, log_sum, grad.contiguous()), None
    x, t = make(7, 333, FP32, seed=1)
    x.requires_grad_()
    w = torch.randn(7, device=DEV)
    (Logprobs.apply(x * 1.0, t) * w).sum().backward()
    check_backward(x.detach(), t, 1.0, w, None, x.grad)


def test_status_of_many_short_rows():
    """The status of 3 000 000 rows costs a part of the call, not a multiple (one block read all
    targets: 6 times), and tells of a single bad target, wherever it stands."""
    n, V = 3000000, 40
    z = torch.randn(n, V, device=DEV, dtype=BF16)
    t = torch.randint(V, (n,), device=DEV)
    ws = ewg.status_workspace()
    r = ewg.token_logprobs(z, t)
    G = torch.ones(n, device=DEV)
    out = torch.empty_like(z)
    for call in (lambda **how: ewg.token_logprobs(z, t, **how),
                 lambda **how: ewg.token_logprobs_backward(z, t, r.row_max, r.log_sum, G, out=out, **how)):
        def shortest(**how):
            times = []
            for _ in range(12):
                a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
                a.record()
                call(**how)
                b.record()
                b.synchronize()
                times.append(a.elapsed_time(b))
            return min(times)
        assert shortest(workspace=ws) < 2 * shortest()
        assert ewg.read_status(ws) == ewg.OK
        for at in (0, 65537, 1234567, n - 1):
            good = int(t[at])
            t[at] = V
            ws.fill_(0)
            call(workspace=ws)
            assert ewg.read_status(ws) == ewg.ERR_ID_OUT_OF_RANGE
            t[at] = good
        ws.fill_(255)
        call(workspace=ws)
        assert ewg.read_status(ws) == ewg.OK
