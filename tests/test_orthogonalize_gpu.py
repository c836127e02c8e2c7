"""orthogonalize_update against its definition in 64 bits.

Tolerance (2-norm of the error over that of the result): the one rounding to bf16 is at most
2^-9.  The fp16 operands of each step are rounded by at most 2^-11 of their off-diagonal
entries, 2^-11 / sqrt(3) in the root mean square, and enter through B, whose norm is below 3
with the default polynomial; the roundings are independent and the polynomial shrinks
perturbations of singular values near 1, so the last two or three steps' remain:
sqrt(3 steps * 3 operands) * 3 * 2^-11 / sqrt(3) * (off-diagonal share of about 1/2) < 2.5e-3.
Together below TOL = 4.5e-3.
"""
import math

import pytest
import torch

import embedding_weight_grad_gb300 as ewg

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
MUON = (3.4445, -4.7750, 2.0315)
TOL = 4.5e-3
BF16, FP32 = torch.bfloat16, torch.float32


def reference(G, steps=5, coefficients=MUON):
    a, b, c = coefficients
    X = G.double()
    tall = X.shape[-2] > X.shape[-1]
    X = X.mT if tall else X
    norm = X.norm(dim=(-2, -1), keepdim=True)
    X = X / torch.where(norm > 0, norm, 1.0)
    for _ in range(steps):
        A = X @ X.mT
        X = a * X + (b * A + c * A @ A) @ X
    return X.mT if tall else X


def randn(*shape, dtype=FP32, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * 1e-3).to(dtype)


def check(got, G, **how):
    want = reference(G, **how)
    assert got.shape == G.shape and got.dtype == BF16
    err = ((got.double() - want).norm(dim=(-2, -1)) / want.norm(dim=(-2, -1))).max().item()
    assert err < TOL, err


SIZES = [(1, 1), (1, 7), (7, 1), (2, 2), (3, 5), (8, 8), (31, 33), (64, 64), (65, 63), (127, 129), (128, 1000),
         (255, 257), (256, 256), (257, 256), (300, 300), (511, 513), (1, 5000), (5000, 3), (999, 1537), (1001, 640),
         (64, 20000), (20000, 40), (2000, 1100)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, dtype):
    G = randn(rows, cols, dtype=dtype, seed=rows + cols)
    check(ewg.orthogonalize_update(G, check=True), G)


SMALL = [(1, 1), (1, 9), (4, 2), (3, 3), (8, 13), (16, 16), (17, 40), (15, 1000), (32, 32), (33, 32), (28, 30), (32, 64),
         (31, 65), (32, 4097), (25, 777), (32, 70000),
         (48, 48), (40, 1001), (33, 4096), (4000, 47)]


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("kind", ["full", "transposed", "strided", "low rank", "one large"])
@pytest.mark.parametrize("rows,cols", SMALL)
def test_small_sides_are_only_rounded(rows, cols, kind, dtype):
    """A smaller side up to 32, or 48 beside one up to 4096, is computed in fp32 and rounded to bf16 once: 2^-8 of an element.  M
    reaches a^5 = 485 on directions without weight and carries some 8 * 2^-24 of that, the
    steps' own roundings come to less: 5e-4 of 1, about the largest singular value."""
    G = randn(3, rows, cols, dtype=dtype, seed=rows + cols)
    if kind == "transposed":
        G = randn(3, cols, rows, dtype=dtype, seed=rows).mT
    elif kind == "strided":
        G = randn(3, rows, cols + 3, dtype=dtype, seed=rows)[:, :, 1:cols + 1]
    elif kind == "low rank":
        k = min(2, rows, cols)
        G = ((randn(3, rows, k, seed=rows) * 1e3) @ randn(3, k, cols, seed=cols)).to(dtype)
    elif kind == "one large":
        G[:, rows // 2, cols // 2] = 3.0
    for steps in (1, 5):
        got, want = ewg.orthogonalize_update(G, steps=steps, check=True).double(), reference(G, steps=steps)
        worst = ((got - want).abs() - 2.0 ** -8 * want.abs()).max().item()
        assert worst <= 5e-4, worst


@pytest.mark.parametrize("batch,rows,cols", [(1, 40, 60), (3, 17, 300), (24, 128, 128), (200, 9, 5), (5, 300, 270),
                                             (7, 513, 260)])
def test_batches(batch, rows, cols):
    G = randn(batch, rows, cols, seed=batch)
    G *= torch.logspace(-6, 6, batch, device=DEV)[:, None, None]     # each matrix has its own norm
    X = ewg.orthogonalize_update(G, check=True)
    check(X, G)
    for z in (0, batch - 1):
        assert torch.equal(X[z], ewg.orthogonalize_update(G[z]))
    G4 = G.view(1, batch, rows, cols)
    assert torch.equal(ewg.orthogonalize_update(G4)[0], X)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_strides(dtype):
    """Rows of a wider buffer at odd offsets, matrices apart, transposed, and out the same way."""
    buf = torch.full((4, 101, 333), math.nan, dtype=dtype, device=DEV)
    G = buf[1:4, 1:91, 3:273]
    G.copy_(randn(3, 90, 270, dtype=dtype))
    want = ewg.orthogonalize_update(G.contiguous())
    check(want, G)
    assert torch.equal(ewg.orthogonalize_update(G), want)
    out = torch.full((3, 95, 275), 7.0, dtype=BF16, device=DEV)
    for at in (0, 1, 4):
        out.fill_(7.0)
        r = ewg.orthogonalize_update(G, out=out[:, 2:92, at:at + 270])
        assert torch.equal(r, want) and r.data_ptr() == out[:, 2:92, at:at + 270].data_ptr()
        assert int((out == 7.0).sum()) == out.numel() - want.numel()
    T = G.mT                                                     # tall, inner stride not 1
    assert torch.equal(ewg.orthogonalize_update(T), want.mT)
    tall = T.contiguous()
    assert torch.equal(ewg.orthogonalize_update(tall), want.mT)
    out.fill_(7.0)
    ewg.orthogonalize_update(T, out=out[:, 2:92, 1:271].mT)
    assert torch.equal(out[:, 2:92, 1:271], want)


@pytest.mark.parametrize("rows,cols", [(300, 500), (512, 512), (500, 130)])
@pytest.mark.parametrize("kind", ["rank one", "low rank", "low rank and noise", "decaying", "one outlier", "diagonal",
                                  "sparse", "orthogonal"])
def test_spectra(rows, cols, kind):
    """Updates whose singular values span many orders of magnitude."""
    g = torch.Generator(device=DEV).manual_seed(4)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    r = min(rows, cols)
    if kind == "rank one":
        G = n(rows, 1) @ n(1, cols)
    elif kind == "low rank":
        G = n(rows, 12) @ n(12, cols)
    elif kind == "low rank and noise":
        G = n(rows, 12) @ n(12, cols) + 0.05 * n(rows, cols)
    elif kind == "decaying":
        u, v = torch.linalg.qr(n(rows, r))[0], torch.linalg.qr(n(cols, r))[0]
        G = (u / (1 + torch.arange(r, device=DEV)) ** 1.5) @ v.mT
    elif kind == "one outlier":
        G = n(rows, cols)
        G[rows // 2, cols // 3] = 1e4
    elif kind == "diagonal":
        G = torch.zeros(rows, cols, device=DEV)
        G.diagonal().copy_(torch.rand(r, generator=g, device=DEV) + 0.01)
    elif kind == "sparse":
        G = n(rows, cols) * (torch.rand(rows, cols, generator=g, device=DEV) < 0.01)
    else:
        q = torch.linalg.qr(n(max(rows, cols), r))[0]
        G = q if rows >= cols else q.mT.contiguous()
    check(ewg.orthogonalize_update(G, check=True), G)


@pytest.mark.parametrize("rows,cols", [(5, 9), (200, 300), (300, 200)])
def test_the_scale_of_the_update_does_not_matter(rows, cols):
    G = randn(rows, cols)
    want = ewg.orthogonalize_update(G)
    for k in (-60, -20, 30, 100):
        assert torch.equal(ewg.orthogonalize_update(G * 2.0 ** k), want)


def test_zero_and_not_finite_matrices_of_a_batch():
    G = randn(5, 70, 300)
    G[1] = 0
    G[2, 69, 299] = math.nan
    G[3, 0, 0] = math.inf
    X = ewg.orthogonalize_update(G, check=True)
    assert bool((X[1] == 0).all())
    assert bool(X[2].isnan().all()) and bool(X[3].isnan().all())
    check(X[[0, 4]], G[[0, 4]])


@pytest.mark.parametrize("rows,cols", [(24, 1 << 20), (1 << 20, 48), (260, 100001)])
def test_longest_sides(rows, cols):
    G = randn(rows, cols, seed=rows)
    check(ewg.orthogonalize_update(G, check=True), G)


@pytest.mark.parametrize("kind", ["rising", "falling", "shuffled"])
@pytest.mark.parametrize("base", [1e-30, 1.0, 1e30])
@pytest.mark.parametrize("rows,cols", [(1, 400000), (2, 400001), (37, 20000), (300, 40)])
def test_norm_of_wide_ranges(rows, cols, base, kind):
    """One step with (1, 0, 0) is G / |G|.  Its magnitudes span 2^-24 to 1 across the elements, so
    more than 1/100 of them (N) carry the norm.  The factor that the result has of G is off by the
    mean of N independent roundings of 2^-9 / sqrt(3) at most: six times that and 2^-20."""
    x = torch.linspace(-24, 0, rows * cols, device=DEV)
    x = x.flip(0) if kind == "falling" else x[torch.randperm(x.numel(), device=DEV)] if kind == "shuffled" else x
    G = (torch.exp2(x) * torch.where(torch.rand_like(x) < 0.5, -base, base)).reshape(rows, cols)
    got = ewg.orthogonalize_update(G, steps=1, coefficients=(1.0, 0.0, 0.0), check=True).double()
    G = G.double() / base
    factor = ((got * G).sum() / (G * G).sum() * G.norm()).item()
    assert abs(factor - 1) < 6 * 2 ** -9 / math.sqrt(3 * G.numel() / 100) + 2 ** -20


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
def test_steps_and_coefficients(steps):
    G = randn(200, 333)
    check(ewg.orthogonalize_update(G, steps=steps, check=True), G, steps=steps)
    cubic = (1.5, -0.5, 0.0)                 # the classical iteration
    check(ewg.orthogonalize_update(G, steps=steps, coefficients=cubic), G, steps=steps, coefficients=cubic)


def test_cubic_steps_converge_to_an_orthogonal_matrix():
    G = randn(100, 700)
    X = ewg.orthogonalize_update(G, steps=20, coefficients=(1.5, -0.5, 0.0)).double()
    eye = torch.eye(100, dtype=torch.float64, device=DEV)
    assert (X @ X.mT - eye).norm().item() / 10 < 2 * TOL     # |eye| = 10; X X^T doubles X's error


def test_the_same_call_gives_the_same_bits():
    G = randn(2, 700, 900)
    ws = ewg.orthogonalize_workspace(G.shape)
    first = ewg.orthogonalize_update(G, workspace=ws)
    for fill in (0, 255):                    # whatever the workspace held
        ws.fill_(fill)
        assert torch.equal(ewg.orthogonalize_update(G, workspace=ws, check=True), first)


def test_streams_and_graph():
    Ga, Gb = randn(600, 1000, seed=1), randn(3, 300, 200, seed=2)
    wa, wb = ewg.orthogonalize_update(Ga), ewg.orthogonalize_update(Gb)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)
    got = []
    for _ in range(3):
        with torch.cuda.stream(sa):
            xa = ewg.orthogonalize_update(Ga)
        with torch.cuda.stream(sb):
            xb = ewg.orthogonalize_update(Gb)
        got.append((xa, xb))
    torch.cuda.synchronize()
    for xa, xb in got:
        assert torch.equal(xa, wa) and torch.equal(xb, wb)
    src, ws = torch.zeros_like(Ga), ewg.orthogonalize_workspace(Ga.shape)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x = ewg.orthogonalize_update(src, workspace=ws)
    src.copy_(Ga)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, wa) and ewg.read_status(ws) == ewg.OK


def test_empty_batch():
    assert ewg.orthogonalize_update(torch.empty(0, 4, 5, device=DEV)).shape == (0, 4, 5)


def test_refusals():
    G = randn(30, 40)

    def no(call):
        with pytest.raises((ValueError, ewg.EwgError)):
            call()
    no(lambda: ewg.orthogonalize_update(G.half()))
    no(lambda: ewg.orthogonalize_update(G.cpu()))
    no(lambda: ewg.orthogonalize_update(G[0]))
    no(lambda: ewg.orthogonalize_update(G[:, ::2]))
    no(lambda: ewg.orthogonalize_update(torch.empty(0, 5, device=DEV)))
    no(lambda: ewg.orthogonalize_update(G[:1].expand(30, 40)))
    no(lambda: ewg.orthogonalize_update(G[None].expand(3, 30, 40)))
    no(lambda: ewg.orthogonalize_update(G, steps=0))
    no(lambda: ewg.orthogonalize_update(G, steps=65))
    no(lambda: ewg.orthogonalize_update(G, coefficients=(1.0, math.nan, 0.0)))
    no(lambda: ewg.orthogonalize_update(G, out=torch.empty(30, 40, device=DEV)))
    no(lambda: ewg.orthogonalize_update(G, out=torch.empty(40, 30, dtype=BF16, device=DEV)))
    H = G.bfloat16()
    no(lambda: ewg.orthogonalize_update(H, out=H))               # out apart from grad
    ws = ewg.orthogonalize_workspace(G.shape)
    no(lambda: ewg.orthogonalize_update(G, workspace=ws[:-256]))
    no(lambda: ewg.orthogonalize_update(G, workspace=torch.empty(ws.numel() + 8, dtype=torch.uint8, device=DEV)[8:]))
    with pytest.raises(ewg.EwgError):
        ewg.orthogonalize_workspace((16385, 16385))
    assert ewg.lib().ewg_orthogonalize_workspace_bytes(1, 0, 5) == 0


@pytest.mark.parametrize("batch,rows,cols", [(1, 700, 512), (3, 300, 256), (30, 1100, 500), (4, 5000, 130)])
def test_tall_results_of_any_alignment(batch, rows, cols):
    """The rows of a tall result that are not aligned go out through the shared memory that the
    next copies come into: the bits of an aligned one, call after call."""
    G = randn(batch, rows, cols, seed=rows)
    want = ewg.orthogonalize_update(G)
    for at, wide in ((0, 1), (1, 7), (4, 12), (3, 5)):
        out = torch.full((batch, rows, cols + wide), 7.0, dtype=BF16, device=DEV)
        for _ in range(5):
            out.fill_(7.0)
            ewg.orthogonalize_update(G, out=out[:, :, at:at + cols], check=True)
            assert torch.equal(out[:, :, at:at + cols], want)
            assert int((out == 7.0).sum()) == out.numel() - want.numel()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("batch,rows,cols", [(1, 1, 1), (2, 1, 9), (1, 8, 13), (3, 32, 32), (2, 70, 300), (1, 256, 256),
                                             (2, 333, 200), (1, 40, 5000), (1, 600, 1001)])
def test_out_lies_as_it_likes(batch, rows, cols, dtype):
    """A row-major or a transposed gradient into a row-major or a transposed out, in any
    combination: the bits that the gradient has without one, and nothing written beside them."""
    G = randn(batch, rows, cols, dtype=dtype, seed=rows)
    for grad in (G, G.mT.contiguous().mT):
        want = ewg.orthogonalize_update(grad, check=True)
        for wide in (0, 1, 5, 8):
            plain = torch.full((batch, rows, cols + wide), 7.0, dtype=BF16, device=DEV)
            turned = torch.full((batch, cols, rows + wide), 7.0, dtype=BF16, device=DEV)
            for buf, out in ((plain, plain[:, :, wide // 2:wide // 2 + cols]),
                             (turned, turned[:, :, wide // 2:wide // 2 + rows].mT)):
                got = ewg.orthogonalize_update(grad, out=out, check=True)
                assert got.data_ptr() == out.data_ptr() and got.stride() == out.stride()
                assert torch.equal(out, want)
                assert int((buf == 7.0).sum()) == buf.numel() - want.numel()
    one = torch.empty(cols, rows, dtype=BF16, device=DEV).mT
    assert torch.equal(ewg.orthogonalize_update(G[0], out=one), ewg.orthogonalize_update(G[0]))


def test_out_with_gaps_in_rows_and_columns_is_refused():
    G = randn(2, 30, 40)
    with pytest.raises(ValueError):
        ewg.orthogonalize_update(G, out=torch.empty(2, 30, 80, dtype=BF16, device=DEV)[:, :, ::2])


def test_autograd_is_told_of_out_written():
    G = randn(40, 60)
    for out in (torch.zeros(40, 60, dtype=BF16, device=DEV), torch.zeros(60, 40, dtype=BF16, device=DEV).mT):
        for grad in (G, G.mT.contiguous().mT):
            version = out._version
            ewg.orthogonalize_update(grad, out=out)
            assert out._version > version


def spectra(kind, rows, cols, g):
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)
    k = min(rows, cols)
    if kind == "dense":
        return n(rows, cols)
    if kind == "rank one":
        return n(rows, 1) @ n(1, cols)
    if kind == "low rank":
        return n(rows, 5) @ n(5, cols)
    if kind == "low rank and noise":
        return n(rows, 12) @ n(12, cols) + 0.3 * n(rows, cols)
    if kind == "outlier":
        G = n(rows, cols)
        G[rows // 2, cols // 3] = 1e3
        return G
    if kind == "rows of many sizes":
        return n(rows, cols) * torch.logspace(0, -3, rows, device=DEV)[:, None]
    if kind == "rows without tokens":
        return n(rows, cols) * (torch.rand(rows, 1, generator=g, device=DEV) < 0.3)
    if kind == "identity":
        return torch.eye(max(rows, cols), device=DEV)[:rows, :cols].contiguous()
    if kind == "diagonal":
        return torch.eye(max(rows, cols), device=DEV)[:rows, :cols] * (torch.rand(rows, 1, generator=g, device=DEV) + 0.01)
    u, v = torch.linalg.qr(n(rows, k))[0], torch.linalg.qr(n(cols, k))[0]
    s = {"orthogonal": lambda i: 1.0 + 0 * i, "slow decay": lambda i: (1.0 + i) ** -0.5,
         "fast decay": lambda i: (1.0 + i) ** -2.0, "linear": lambda i: 1.0 - i / k}[kind](torch.arange(k, device=DEV))
    return (u * s) @ v.mT


DENSE = ["dense", "rank one", "low rank", "low rank and noise", "outlier", "rows of many sizes", "rows without tokens",
         "slow decay", "fast decay", "linear"]


def errors(rows, cols, kind, seeds):
    g = torch.Generator(device=DEV).manual_seed(100 * rows + cols)
    G = torch.stack([spectra(kind, rows, cols, g) for _ in range(seeds)]) * 1e-2
    got, want = ewg.orthogonalize_update(G, check=True).double(), reference(G)
    size = want.norm(dim=(-2, -1)).clamp_min(1e-300)
    return ((got - want).norm(dim=(-2, -1)) / size).max().item(), \
        ((want.to(BF16).double() - want).norm(dim=(-2, -1)) / size).max().item()


@pytest.mark.parametrize("rows,cols", [(33, 5000), (49, 49), (61, 50), (63, 200), (64, 64), (71, 72), (86, 73), (118, 117),
                                       (128, 1000), (200, 333), (256, 256), (300, 299), (513, 700), (1024, 1030)])
def test_the_promised_precision(rows, cols):
    """What include/ewg.h promises of five steps, by the kind of update and the smaller side."""
    dense = 3e-3 if min(rows, cols) < 256 else 2.4e-3
    for kind in DENSE:
        assert errors(rows, cols, kind, 3)[0] < dense, kind
    for kind, most in (("orthogonal", 4e-3), ("diagonal", 5e-3), ("identity", 9e-3)):
        assert errors(rows, cols, kind, 3)[0] < most, kind


@pytest.mark.parametrize("rows,cols", [(1, 1), (9, 1), (4, 2), (8, 13), (17, 40), (32, 32), (32, 70000), (48, 48),
                                       (1001, 40)])
def test_the_promised_precision_of_small_sides(rows, cols):
    """In fp32 M makes of its own rounding 8 * 2^-24 of a^5 = 485, 2.4e-4 of the largest singular
    value at most: d.  Where that moves an element to another bf16 number, the exact one was no
    further than d from the middle between them: the error is that of the exact result's rounding and
    2 d at most."""
    for kind in [*DENSE, "orthogonal", "diagonal", "identity"]:
        if kind in ("rows without tokens", "outlier") and min(rows, cols) < 4:
            continue                                     # (nothing may be left of it)
        error, rounding = errors(rows, cols, kind, 1)
        assert error < rounding + 5e-4, kind
