"""layer_norm and layer_norm_backward against their definitions in 64 bits.

Tolerances, from the operations' roundings (u = 2^-24).  K additions, one after the other or in
a tree, are off by at most K u times the sum of magnitudes; a thread adds at most H / 256 + 64
numbers before trees of at most 16 levels, so K = H / 256 + 80.

Forward, d = x - mean: a deviation is off by 2 u |d| and by the centre's error, K u avg|d|;
the variance (a sum of squares) by (K + 6) u relatively, rstd by half of that and 3 u; the product
with the weight and the bias add u each, the output's rounding half a step.

Backward (mean and rstd are inputs): n by 2 u, u = g w by u, avg(u) by (K + 2) u avg|u|, avg(u n) by
(K + 5) u avg|u n|; dx adds 4 u of its three terms, and half a step.  Sums over rows: at
most n / 16 + 352 additions of terms that are off by 4 u.
"""
import pytest
import torch

import embedding_weight_grad_gb300 as ewg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF16, FP32 = torch.bfloat16, torch.float32


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rows(n, H, dtype, seed=0, pad=0, offset=0.0, spread=1.0, lead=0):
    """Rows of a wider buffer, which starts `lead` elements in, NaN between them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    buf = torch.full((n * (H + pad) + lead,), float("nan"), dtype=dtype, device=DEV)[lead:].view(n, H + pad)
    x = buf[:, :H]
    x.copy_((torch.randn(n, H, generator=g, device=DEV) * spread + offset) * (1 + torch.arange(H, device=DEV) % 7))
    return x


def vectors(H, dtype, seed=1):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (1 + 0.5 * torch.randn(H, generator=g, device=DEV)).to(dtype), torch.randn(H, generator=g, device=DEV).to(dtype)


def near(got, want, tol, what):
    worst = ((got.double() - want).abs() - tol).max().item()
    assert worst <= 0, (what, worst)


def check_forward(x, w, b, eps, r):
    H = x.shape[-1]
    K = H / 256 + 80
    x64 = x.double()
    mean = x64.mean(-1, keepdim=True)
    d = x64 - mean
    var = d.square().mean(-1, keepdim=True)
    rstd = (var + eps).rsqrt()
    avg = d.abs().mean(-1, keepdim=True)
    w64 = 1.0 if w is None else w.double()
    want = d * rstd * w64 + (0.0 if b is None else b.double())
    near(r.mean, mean[..., 0], K * U * avg[..., 0] + 2 * U * mean[..., 0].abs(), "mean")
    near(r.rstd, rstd[..., 0], (K / 2 + 6) * U * rstd[..., 0], "rstd")
    part = (d * rstd * w64).abs()
    tol = (K / 2 + 12) * U * part + (K * U * avg * rstd * w64).abs() + 2 * U * want.abs()
    near(r.out, want, tol + (half_step(x.dtype) * (want.abs() + tol) if x.dtype == BF16 else 0), "out")


def check_backward(g, x, mean, rstd, w, got, before=None, after=None):
    """before, after: the main_grads (weight's, bias's; None: not wanted)."""
    n, H = x.shape
    K = H / 256 + 80
    g64, x64 = g.double(), x.double()
    r64 = rstd.double()[:, None]
    hat = (x64 - mean.double()[:, None]) * r64
    u = g64 * (1.0 if w is None else w.double())
    c1, c2 = u.mean(1, keepdim=True), (u * hat).mean(1, keepdim=True)
    a1, a2 = u.abs().mean(1, keepdim=True), (u * hat).abs().mean(1, keepdim=True)
    want = r64 * (u - c1 - hat * c2)
    tol = r64 * U * (4 * (u.abs() + c1.abs() + (hat * c2).abs()) + (K + 2) * a1 + hat.abs() * (K + 6) * a2) + U * want.abs()
    near(got, want, tol + (half_step(x.dtype) * (want.abs() + tol) if x.dtype == BF16 else 0), "grad_x")
    for k, term in enumerate((g64 * hat, g64)):
        if before is None or before[k] is None:
            continue
        total = before[k].double() + term.sum(0)
        tol = (n / 16 + 352) * U * term.abs().sum(0) + U * total.abs()
        near(after[k], total, tol + half_step(after[k].dtype) * (total.abs() + tol), ("main_grad", k))


def both(x, w, b, eps=1e-5, mg_dtype=FP32, seed=2, grad=None):
    r = ewg.layer_norm(x, w, b, eps=eps)
    check_forward(x, w, b, eps, r)
    gen = torch.Generator(device=DEV).manual_seed(seed)
    H = x.shape[-1]
    g = torch.randn(x.shape, generator=gen, device=DEV).to(x.dtype) if grad is None else grad
    mgs = [torch.randn(H, generator=gen, device=DEV).to(mg_dtype) for _ in range(2)]
    before = [m.clone() for m in mgs]
    got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=mgs[0], bias_main_grad=mgs[1])
    check_backward(g, x, r.mean, r.rstd, w, got, before, mgs)
    return r, g, got


SIZES = [(1, 1), (1, 2), (2, 3), (5, 8), (1, 31), (33, 32), (3, 33), (17, 100), (64, 128), (9, 250), (300, 256), (7, 257),
         (100, 511), (5, 512), (4097, 40), (3, 1000), (65, 1001), (200, 1024), (31, 1025), (2, 2047), (40, 2048), (3, 2056),
         (160, 4096), (7, 4099), (33, 5001), (320, 7168), (5, 8191), (154, 8192), (3, 8200), (2, 12288), (3, 16384),
         (2, 16391), (2, 20000), (3, 32768), (1, 33001), (2, 65536), (2, 65537), (1, 100000)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,H", SIZES)
def test_sizes(n, H, dtype):
    x = rows(n, H, dtype, seed=n + H)
    both(x, *vectors(H, dtype))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,H", [(2000, 8), (5000, 64), (3000, 264), (2500, 777), (2000, 1000), (1500, 2304), (1300, 5120),
                                 (700, 6151), (1216, 8192), (400, 24576)])
def test_many_rows(n, H, dtype):
    """Rows enough for every block to take several."""
    x = rows(n, H, dtype, seed=n + H)
    both(x, *vectors(H, FP32))


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (2, 2), (3, 5), (4, 4), (8, 0), (8, 8), (40, 16), (6, 2)])
@pytest.mark.parametrize("n,H", [(19, 96), (9, 1024), (5, 4104), (33, 7168), (3, 20008)])
def test_strides_and_alignment(n, H, pad, lead, dtype):
    x = rows(n, H, dtype, seed=pad, pad=pad, lead=lead)
    w, b = vectors(H, dtype)
    r, g, got = both(x, w, b, grad=rows(n, H, dtype, seed=9, pad=lead, lead=pad))
    # outputs elsewhere, rows of another stride: what lies between the rows is left alone
    out = torch.full((n, H + 5), 7.0, dtype=dtype, device=DEV)
    ro = ewg.layer_norm(x, w, b, out=out[:, :H])
    assert ro.out.data_ptr() == out.data_ptr() and bool((out[:, H:] == 7.0).all())
    check_forward(x, w, b, 1e-5, ro)
    out.fill_(7.0)
    ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, out=out[:, :H])
    assert bool((out[:, H:] == 7.0).all())
    check_backward(g, x, r.mean, r.rstd, w, out[:, :H])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad,lead", [(0, 0), (0, 1), (0, 3), (1, 0), (1, 7), (2, 2), (3, 5), (4, 4), (7, 1), (8, 6)])
@pytest.mark.parametrize("H", [1, 2, 3, 7, 8, 9, 15, 17, 63, 64, 65, 127, 250, 511, 513, 769, 1001, 1025, 2047, 4099, 7167, 8189,
                               8192])
def test_rows_of_one_alignment(H, pad, lead, dtype):
    """All arrays' rows begin at the same places in 16 bytes, whatever these are; what lies before, between and
    behind the rows is left alone."""
    w, b = vectors(H, FP32)
    mg0 = torch.ones(H, device=DEV)
    for n in (1, 3, 9, 41, 700 if H < 3000 else 160):
        x, g = rows(n, H, dtype, seed=H, pad=pad, lead=lead), rows(n, H, dtype, seed=9, pad=pad, lead=lead)

        def target():
            buf = torch.full((n * (H + pad) + lead + 16,), 7.0, dtype=dtype, device=DEV)
            return buf, buf[lead:lead + n * (H + pad)].view(n, H + pad)[:, :H]

        def check_guard(buf, y):
            y.fill_(7.0)
            assert bool((buf == 7.0).all())
        buf, out = target()
        r = ewg.layer_norm(x, w, b, out=out)
        check_forward(x, w, b, 1e-5, r)
        check_guard(buf, out)
        buf, out = target()
        mgs = [mg0.clone(), mg0.clone()]
        ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=mgs[0], bias_main_grad=mgs[1], out=out)
        check_backward(g, x, r.mean, r.rstd, w, out, [mg0, mg0], mgs)
        check_guard(buf, out)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vec_dtype", [BF16, FP32])
@pytest.mark.parametrize("mg_dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [120, 1001, 4096])
def test_types(H, mg_dtype, vec_dtype, dtype):
    x = rows(70, H, dtype, seed=H)
    both(x, *vectors(H, vec_dtype), mg_dtype=mg_dtype)


@pytest.mark.parametrize("H", [1, 64, 1001, 8192, 40000])
def test_without_weight_bias_or_main_grads(H):
    x = rows(37, H, BF16, seed=H)
    w, b = vectors(H, FP32)
    g = rows(37, H, BF16, seed=3)
    for ww, bb in ((None, None), (w, None), (None, b)):
        r = ewg.layer_norm(x, ww, bb)
        check_forward(x, ww, bb, 1e-5, r)
        for want_w, want_b in ((False, False), (True, False), (False, True)):
            mgs = [torch.ones(H, device=DEV) if k else None for k in (want_w, want_b)]
            before = [m if m is None else m.clone() for m in mgs]
            got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, ww, weight_main_grad=mgs[0], bias_main_grad=mgs[1])
            check_backward(g, x, r.mean, r.rstd, ww, got, before, mgs)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [24, 1000, 1001, 7168, 20000])
def test_in_place(H, dtype):
    x = rows(301, H, dtype, seed=H)
    w, b = vectors(H, dtype)
    r = ewg.layer_norm(x, w, b)
    again = x.clone()
    r2 = ewg.layer_norm(again, w, b, out=again)
    assert r2.out is again and torch.equal(again, r.out) and torch.equal(r2.mean, r.mean)
    g = rows(301, H, dtype, seed=5)
    mg = [torch.zeros(H, device=DEV) for _ in range(6)]
    got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=mg[0], bias_main_grad=mg[1])
    for k, target in ((2, "grad"), (4, "x")):
        gg, xx = g.clone(), x.clone()
        o = ewg.layer_norm_backward(gg, xx, r.mean, r.rstd, w, weight_main_grad=mg[k], bias_main_grad=mg[k + 1],
                                    out=gg if target == "grad" else xx)
        assert torch.equal(o, got) and torch.equal(mg[k], mg[0]) and torch.equal(mg[k + 1], mg[1])


@pytest.mark.parametrize("H", [40, 1001, 7168, 20000])
def test_rows_far_from_zero(H):
    """A mean a thousand times the deviation: the deviations keep their digits."""
    x = rows(40, H, FP32, seed=H, spread=1e-3, offset=1.0)
    w, b = vectors(H, FP32)
    check_forward(x / (1 + torch.arange(H, device=DEV) % 7), w, b, 1e-12, ewg.layer_norm(x / (1 + torch.arange(H, device=DEV) % 7), w, b, eps=1e-12))
    both(x, w, b)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("H", [1, 8, 100, 1001, 8192, 20000])
def test_equal_elements(H, dtype):
    """No deviation: the bias remains, but for the centre's error, K u of an error of u."""
    x = torch.full((3, H), 2.75, dtype=dtype, device=DEV)
    w, b = vectors(H, dtype)
    r = ewg.layer_norm(x, w, b)
    centre = (H / 256 + 80) * U * 2 * U * 2.75 * 1e-5 ** -0.5
    near(r.out, b.double(), centre * w.double().abs() + (2 * U * b.double().abs() if dtype == FP32 else 0), "out")
    assert bool((r.mean == 2.75).all())
    torch.testing.assert_close(r.rstd, torch.full((3,), 1e-5, device=DEV).rsqrt(), rtol=4 * U, atol=0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("H", [5, 256, 1001, 7168, 20000])
def test_nan_and_infinity_stay_in_their_row(H, bad):
    for dtype in (BF16, FP32):
        x = rows(6, H, dtype, seed=H)
        w, b = vectors(H, dtype)
        clean = ewg.layer_norm(x, w, b)
        x[2, H // 2] = bad
        r = ewg.layer_norm(x, w, b)
        assert bool(r.out[2].isnan().all()) and bool(r.rstd[2].isnan())
        keep = [0, 1, 3, 4, 5]
        assert torch.equal(r.out[keep], clean.out[keep]) and torch.equal(r.mean[keep], clean.mean[keep])
        g = rows(6, H, dtype, seed=4)
        got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w)
        assert bool(got[2].isnan().all())
        check_backward(g[keep], x[keep], r.mean[keep], r.rstd[keep], w, got[keep])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("n,H", [(2432, 4096), (2433, 2048), (2435, 2056), (3001, 2303), (2440, 2816), (4864, 4099), (2501, 5000),
                                 (5003, 7168), (2436, 8189), (2737, 8192)])
def test_wide_rows_in_number(n, H, pad, dtype):
    """Every block takes many batches, the last ones short; rows that hold no numbers are nobody else's matter."""
    x = rows(n, H, dtype, seed=H, pad=pad)
    w, b = vectors(H, dtype)
    r = ewg.layer_norm(x, w, b)
    check_forward(x, w, b, 1e-5, r)
    y = x.clone()
    r2 = ewg.layer_norm(y, w, b, out=y)
    if pad == 0:
        assert torch.equal(r2.out, r.out) and torch.equal(r2.mean, r.mean) and torch.equal(r2.rstd, r.rstd)
        assert torch.equal(ewg.layer_norm(x, w, b, stats=False).out, r.out)
    bad = torch.arange(5, n, 7, device=DEV)
    x[bad[0::3], 0] = float("nan")
    x[bad[1::3], H - 1] = float("inf")
    x[bad[2::3], H // 2] = -float("inf")
    r2 = ewg.layer_norm(x, w, b)
    assert bool(r2.out[bad].isnan().all()) and bool(r2.rstd[bad].isnan().all())
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(r2.out[keep], r.out[keep]) and torch.equal(r2.mean[keep], r.mean[keep])
    assert torch.equal(r2.rstd[keep], r.rstd[keep])


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("vec_dtype", [BF16, FP32])
@pytest.mark.parametrize("n,H", [(1001, 9000), (701, 12288), (701, 16384), (333, 24576), (307, 32768), (95, 65536), (401, 8193)])
def test_rows_of_more_than_8192_in_number(n, H, vec_dtype, dtype):
    """Every block and cluster takes several batches, in place too; rows that hold no numbers are nobody else's matter."""
    x = rows(n, H, dtype, seed=H)
    w, b = vectors(H, vec_dtype)
    r, g, got = both(x, w, b)
    y = x.clone()
    r2 = ewg.layer_norm(y, w, b, out=y)
    assert torch.equal(r2.out, r.out) and torch.equal(r2.mean, r.mean) and torch.equal(r2.rstd, r.rstd)
    for target in (0, 1):
        pair = [g.clone(), x.clone()]
        assert torch.equal(ewg.layer_norm_backward(*pair, r.mean, r.rstd, w, out=pair[target]), got)
    bad = torch.arange(3, n, 5, device=DEV)
    x[bad[0::3], 0] = float("nan")
    x[bad[1::3], H - 1] = float("inf")
    x[bad[2::3], H // 2] = -float("inf")
    r2 = ewg.layer_norm(x, w, b)
    assert bool(r2.out[bad].isnan().all()) and bool(r2.rstd[bad].isnan().all())
    got2 = ewg.layer_norm_backward(g, x, r2.mean, r2.rstd, w)
    assert bool(got2[bad].isnan().all())
    keep = torch.ones(n, dtype=torch.bool, device=DEV)
    keep[bad] = False
    for a, c in ((r2.out, r.out), (r2.mean, r.mean), (r2.rstd, r.rstd), (got2, got)):
        assert torch.equal(a[keep], c[keep])


@pytest.mark.parametrize("H", [16, 1024, 8192, 32768, 131072])
def test_the_ends_of_eps(H):
    """A row of equal elements whose mean is exact gives the bias at the least eps too."""
    x = torch.full((3, H), 2.0, device=DEV)
    w, b = vectors(H, FP32)
    for eps in (1e-320, 1e-46, 1e-40, 2.0 ** -127, 2.0 ** 127, 1e39, float("inf")):
        with pytest.raises(ewg.EwgError, match="eps"):
            ewg.layer_norm(x, w, b, eps=eps)
    for eps in (2.0 ** -126, 2.0 ** 126):
        r = ewg.layer_norm(x, w, b, eps=eps)
        assert torch.equal(r.out, b.expand(3, H)) and bool((r.rstd == eps ** -0.5).all())


@pytest.mark.parametrize("H", [16, 1001, 7168])
def test_small_and_large_numbers(H):
    """Sums of squares stay in range from 2^-60 to 2^50; eps takes over for the smallest."""
    w, b = vectors(H, FP32)
    for k in (-60, -20, 20, 50):
        x = rows(9, H, FP32, seed=H) * 2.0 ** k
        for eps in (1e-5, 1e-30):
            check_forward(x, w, b, eps, ewg.layer_norm(x, w, b, eps=eps))


@pytest.mark.parametrize("H", [24, 1001, 8192, 20000, 40000])
def test_without_stats(H):
    x = rows(33, H, BF16, seed=H)
    w, b = vectors(H, BF16)
    r = ewg.layer_norm(x, w, b, stats=False)
    assert r.mean is None and r.rstd is None and torch.equal(r.out, ewg.layer_norm(x, w, b).out)


def test_shapes():
    x = rows(12, 96, BF16)
    w, b = vectors(96, BF16)
    r = ewg.layer_norm(x, w, b)
    r3 = ewg.layer_norm(x.view(2, 6, 96), w, b)
    assert r3.out.shape == (2, 6, 96) and r3.mean.shape == (2, 6) and torch.equal(r3.out.view(12, 96), r.out)
    r1 = ewg.layer_norm(x[3], w, b)
    assert r1.mean.shape == () and torch.equal(r1.out, r.out[3])
    g = rows(12, 96, BF16, seed=4)
    a = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w)
    c = ewg.layer_norm_backward(g.view(2, 6, 96), x.view(2, 6, 96), r3.mean, r3.rstd, w)
    assert torch.equal(a, c.view(12, 96))
    assert ewg.layer_norm_backward(g[3], x[3], r1.mean, r1.rstd, w).shape == (96,)
    for shape in ((0, 96), (3, 0, 96)):                  # no rows: the main_grads stay
        e = torch.empty(shape, dtype=BF16, device=DEV)
        r0 = ewg.layer_norm(e, w, b)
        mg = torch.full((96,), 3.0, device=DEV)
        assert r0.out.shape == shape and r0.mean.shape == shape[:-1]
        assert ewg.layer_norm_backward(e, e, r0.mean, r0.rstd, w, weight_main_grad=mg).shape == shape
        assert bool((mg == 3.0).all())


@pytest.mark.parametrize("n,H", [(70000, 40000), (300000, 8192)])
def test_offsets_beyond_32_bits(n, H):
    """More than 2^31 elements: the last rows of a large array."""
    x = torch.zeros(n, H, dtype=BF16, device=DEV)
    x[-3:] = rows(3, H, BF16, seed=H)
    w, b = vectors(H, BF16)
    r = ewg.layer_norm(x, w, b, out=x.clone())
    tail = ewg.LayerNorm(*(t[-3:] for t in r))
    check_forward(x[-3:], w, b, 1e-5, tail)
    g = torch.zeros_like(x)
    g[-3:] = rows(3, H, BF16, seed=H + 1)
    mgs = [torch.zeros(H, device=DEV) for _ in range(2)]
    got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=mgs[0], bias_main_grad=mgs[1], out=r.out)
    check_backward(g[-3:], x[-3:], tail.mean, tail.rstd, w, got[-3:], [torch.zeros(H, device=DEV)] * 2, mgs)


@pytest.mark.parametrize("H", [33, 768, 4096])
def test_gradient_against_differences(H):
    """The gradient of sum(c * layer_norm(x)) by central differences of the definition in 64 bits, along
    random directions: what the differences miss is of the third order, h^2."""
    x = rows(6, H, FP32, seed=H)
    w, b = vectors(H, FP32)
    gen = torch.Generator(device=DEV).manual_seed(8)
    c = torch.randn(6, H, generator=gen, device=DEV)
    r = ewg.layer_norm(x, w, b)
    mgs = [torch.zeros(H, device=DEV) for _ in range(2)]
    dx = ewg.layer_norm_backward(c, x, r.mean, r.rstd, w, weight_main_grad=mgs[0], bias_main_grad=mgs[1])

    def value(x64, w64, b64):
        d = x64 - x64.mean(1, keepdim=True)
        return (c.double() * (d * (d.square().mean(1, keepdim=True) + 1e-5).rsqrt() * w64 + b64)).sum()
    args = [x.double(), w.double(), b.double()]
    h = 2.0 ** -13
    for k, grad in enumerate((dx, mgs[0], mgs[1])):
        for trial in range(3):
            v = torch.randn(args[k].shape, generator=gen, device=DEV).double()
            moved = [[a + s * h * v if i == k else a for i, a in enumerate(args)] for s in (1, -1)]
            slope = (value(*moved[0]) - value(*moved[1])) / (2 * h)
            size = (grad.double() * v).abs().sum()
            assert abs((grad.double() * v).sum() - slope) < 1e-5 * size


@pytest.mark.parametrize("n,H", [(3001, 2048), (3001, 1001), (700, 12000)])
def test_same_call_same_bits_and_streams(n, H):
    """Twice on each of two streams at once, and captured and replayed."""
    x, g = rows(n, H, BF16, seed=1), rows(n, H, BF16, seed=2)
    w, b = vectors(H, FP32)
    r = ewg.layer_norm(x, w, b)
    want = torch.zeros(2, H, device=DEV)
    dx = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=want[0], bias_main_grad=want[1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                mg = torch.zeros(2, H, device=DEV)
                rs = ewg.layer_norm(x, w, b)
                outs.append((rs, ewg.layer_norm_backward(g, x, rs.mean, rs.rstd, w, weight_main_grad=mg[0],
                                                         bias_main_grad=mg[1]), mg))
    torch.cuda.synchronize()
    for rs, d, mg in outs:
        assert all(torch.equal(p, q) for p, q in zip(rs, r)) and torch.equal(d, dx) and torch.equal(mg, want)
    graph = torch.cuda.CUDAGraph()
    mg = torch.zeros(2, H, device=DEV)
    out, ws = torch.empty_like(x), ewg.layer_norm_workspace(x.shape)
    with torch.cuda.graph(graph):
        rs = ewg.layer_norm(x, w, b)
        ewg.layer_norm_backward(g, x, rs.mean, rs.rstd, w, weight_main_grad=mg[0], bias_main_grad=mg[1], out=out,
                                workspace=ws)
    ws.fill_(0xff)                                   # a workspace needs no initialisation
    for _ in range(3):
        mg.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, dx) and torch.equal(mg, want) and torch.equal(rs.out, r.out)


def test_main_grads_accumulate():
    """Calls one after the other add to what is there."""
    x = rows(50, 300, BF16)
    w, b = vectors(300, FP32)
    r = ewg.layer_norm(x, w, b)
    g = rows(50, 300, BF16, seed=6)
    one, three = torch.zeros(300, device=DEV), torch.zeros(300, device=DEV)
    ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=one)
    for _ in range(3):
        ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=three)
    torch.testing.assert_close(three, 3 * one, rtol=4 * U, atol=0)


def test_autograd_is_told():
    x = rows(4, 64, FP32).clone()
    w, b = vectors(64, FP32)
    v = (x._version, w._version)
    r = ewg.layer_norm(x, w, b)
    assert (x._version, w._version) == v
    mg = torch.zeros(64, device=DEV)
    ewg.layer_norm_backward(x, x, r.mean, r.rstd, w, weight_main_grad=mg, out=r.out)
    assert mg._version == 1 and r.out._version == 1
    ewg.layer_norm(x, w, b, out=x)
    assert x._version == v[0] + 1


def test_refusals():
    x = rows(6, 64, BF16)
    w, b = vectors(64, BF16)
    r = ewg.layer_norm(x, w, b)
    back = lambda **k: ewg.layer_norm_backward(**{**dict(grad=x.clone(), x=x, mean=r.mean, rstd=r.rstd, weight=w), **k})
    mg = torch.zeros(64, device=DEV)
    for call in (lambda: ewg.layer_norm(x.half(), w, b), lambda: ewg.layer_norm(x, w.float(), b),
                 lambda: ewg.layer_norm(x, w[:32], b), lambda: ewg.layer_norm(x, w.expand(6, 64)),
                 lambda: ewg.layer_norm(x.t(), w[:6], b[:6]), lambda: ewg.layer_norm(x[:, ::2], w[::2], b[::2]),
                 lambda: ewg.layer_norm(x[:, :0]), lambda: ewg.layer_norm(x, w.cpu(), b.cpu()),
                 lambda: ewg.layer_norm(x, w, b, out=torch.empty(6, 64, device=DEV)),
                 lambda: ewg.layer_norm(x, w, b, out=x[:5]),
                 lambda: back(grad=x.float()), lambda: back(grad=x[:3]), lambda: back(mean=r.mean.double()),
                 lambda: back(mean=r.mean[:3]), lambda: back(weight_main_grad=mg, bias_main_grad=mg.bfloat16()),
                 lambda: back(weight_main_grad=mg[:32]), lambda: back(weight_main_grad=mg.int()),
                 lambda: back(rstd=r.rstd.cpu()), lambda: back(out=x[:, :32])):
        with pytest.raises(ValueError):
            call()
    two = torch.zeros(128, device=DEV)
    wide = torch.zeros(6, 128, dtype=BF16, device=DEV)
    for call in (lambda: ewg.layer_norm(x, w, b, eps=-1.0), lambda: ewg.layer_norm(x, w, b, eps=float("nan")),
                 lambda: ewg.layer_norm(wide[:, :64], w, b, out=wide[:, 32:96]),
                 lambda: ewg.layer_norm(x[:5], w, b, out=x[1:]), lambda: ewg.layer_norm(x[:1].expand(6, 64), w, b),
                 lambda: ewg.layer_norm(x, x[0], b, out=x),
                 lambda: back(weight_main_grad=two[:64], bias_main_grad=two[32:96]),
                 lambda: back(workspace=torch.empty(100, dtype=torch.uint8, device=DEV)),
                 lambda: back(weight_main_grad=w), lambda: back(workspace=ewg.layer_norm_workspace(x.shape)[1:])):
        with pytest.raises(ewg.EwgError):
            call()


# Rows that no block holds: a thread adds up 32 numbers at a time, 32 of these sums and then at most 64 of those, and
# the threads' sums meet in 13 additions: at most 142 in a row, however wide the row is.  K: with 1 / H and the product by it.
WIDE = 144
WIDEST = 1 << 24


@pytest.mark.parametrize("value", [8.1, 1.1, 3.3, -1.9])
@pytest.mark.parametrize("H", [32769, 1 << 20, (1 << 22) + 3, WIDEST - 1, WIDEST])
def test_equal_elements_of_very_wide_rows(H, value):
    """The first centre is off by e = K u of the value c.  The deviations are all c e, exactly, and their mean is off by K u
    of that, which leaves the mean its own rounding.  The variance is what the squares' mean (K u) and the mean's square
    (2 K u) are off, with two roundings: at most (3 K + 4) u (c e)^2."""
    x = torch.full((1, H), value, dtype=FP32, device=DEV)
    c, eps = x[0, 0].item(), 1e-10
    r = ewg.layer_norm(x, None, None, eps=eps)
    off = WIDE * U * abs(c)
    assert abs(r.mean.item() - c) <= U * abs(c) + 2 * WIDE * U * off, (r.mean.item() - c) / (U * abs(c))
    most = (3 * WIDE + 4) * U * off ** 2
    want = eps ** -0.5
    assert abs(r.rstd.item() - want) <= (most / (2 * eps) + 4 * U) * want
    # (the mean's rounding is no deviation: what it leaves of each element is the centre's rest, off by K u)
    assert r.out.abs().max().item() <= (2 * WIDE + 4) * U * off * want * (1 + 4 * U)


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,H,offset", [(1, WIDEST, 0.0), (2, (1 << 22) + 3, 0.0), (3, 65537, 0.0), (1, WIDEST, 1.0)])
def test_very_wide_rows(n, H, offset, dtype):
    """As check_forward and check_backward, with a K that does not grow with H, and a gradient whose mean is not 0.  The
    deviations are taken from a number near the mean, off it by K u avg|x|, in bf16 by half a step of the mean
    besides; what is added up are the deviations from that."""
    gen = torch.Generator(device=DEV).manual_seed(H)
    x = (offset + torch.randn(n, H, generator=gen, device=DEV) * 0.5).to(dtype)
    g = (1.1 + torch.randn(n, H, generator=gen, device=DEV) * 0.01).to(dtype)
    w = (1 + 0.1 * torch.randn(H, generator=gen, device=DEV))
    K, eps = WIDE, 1e-5
    x64, g64, w64 = x.double(), g.double(), w.double()
    mean = x64.mean(1, keepdim=True)
    d = x64 - mean
    near_mean = K * U * x64.abs().mean(1, keepdim=True) + (2.0 ** -8 * mean.abs() if dtype == BF16 else 0)
    avg = d.abs().mean(1, keepdim=True) + near_mean
    var = d.square().mean(1, keepdim=True)
    square = var + near_mean ** 2
    rstd = (var + eps).rsqrt()
    r = ewg.layer_norm(x, w, None, eps=eps)
    rest = (K + 2) * U * avg
    near(r.mean, mean[:, 0], (rest + 2 * U * mean.abs())[:, 0], "mean")
    var_tol = (K + 4) * U * square + 2 * near_mean * rest + rest ** 2 + 2 * U * var
    r_tol = (var_tol / (2 * (var + eps)) + 5 * U) * 1.01
    near(r.rstd, rstd[:, 0], (r_tol * rstd)[:, 0], "rstd")
    want = d * rstd * w64
    tol = rstd * w64.abs() * (rest + 3 * U * (d.abs() + near_mean)) + (r_tol + 3 * U) * want.abs()
    near(r.out, want, tol + (half_step(BF16) * (want.abs() + tol) if dtype == BF16 else 0), "out")
    mgs = [torch.ones(H, device=DEV) for _ in range(2)]
    got = ewg.layer_norm_backward(g, x, r.mean, r.rstd, w, weight_main_grad=mgs[0], bias_main_grad=mgs[1])
    r64 = r.rstd.double()[:, None]
    hat = (x64 - r.mean.double()[:, None]) * r64
    u = g64 * w64
    c1, c2 = u.mean(1, keepdim=True), (u * hat).mean(1, keepdim=True)
    a1, a2 = u.abs().mean(1, keepdim=True), (u * hat).abs().mean(1, keepdim=True)
    want = r64 * (u - c1 - hat * c2)
    tol = r64 * U * (4 * (u.abs() + c1.abs() + (hat * c2).abs()) + (K + 3) * a1 + hat.abs() * (K + 6) * a2) + U * want.abs()
    near(got, want, tol + (half_step(dtype) * (want.abs() + tol) if dtype == BF16 else 0), "grad_x")
    for mg, term in zip(mgs, (g64 * hat, g64)):
        total = 1 + term.sum(0)
        near(mg, total, (n + 8) * U * (term.abs().sum(0) + total.abs()), "main_grad")
