"""The embedding-head operators on the GPU against their fp64 forms: layer norm, linear and
balance loss, both directions, both point types.

Tolerances (derived, per element): u = 2^-24 is half an fp32 step relative to a value, and an
output of type t is off by at most eps_t / 2 of its value from its own rounding.  A sum of n
products accumulated in fp32 is off by at most about n u sum|terms| for any order with
rounding to nearest; twice that (and a few more) covers an accumulator that truncates.
"""
import math

import pytest
import torch

import head_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def fk(cuda_device):
    from exact_lloyd_means_b200 import fk as m
    return m


def half_step(t):
    return torch.finfo(t).eps / 2


def rnd(shape, dtype=torch.float32, seed=0, scale=1.0, shift=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(dtype)


def within(got, want, tol, what=""):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    if bool(bad.any()):
        worst = int((err / (tol + 1e-300)).nan_to_num(nan=1e300).argmax())
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} out of tolerance; worst at {worst}: got "
            f"{float(got.reshape(-1)[worst])}, want {float(want.reshape(-1)[worst])}, tolerance "
            f"{float((tol + 0 * want).reshape(-1)[worst])}")


# ------------------------------------------------------------------------------ layer norm

def ln_tol(X, gamma, beta, eps, dtype):
    """|mean error| <= n u mean|x| with n the longest chain of additions (every kernel sums a
    row over at least 16 lanes); rstd is off by half the relative error of var, which is that
    of n additions plus the square of the mean's error; y = (x - mean) rstd gamma + beta."""
    x = X.double()
    d = x.shape[1]
    n = d / 16 + 24
    y, mean, rstd = ref.layer_norm(X, gamma, beta, eps)
    em = n * U * x.abs().mean(1) + 2 * U * mean.abs()
    er = 0.5 * (n * U + (em * rstd) ** 2) + 4 * U
    ga = torch.ones(d, device=x.device, dtype=torch.float64) if gamma is None else \
        gamma.double().abs()
    be = 0 if beta is None else beta.double().abs()
    c = (x - mean[:, None]).abs()
    ey = ga * rstd[:, None] * (em[:, None] + c * (er[:, None] + 4 * U)) + 2 * U * be
    return half_step(dtype) * y.abs() + ey * (1 + half_step(dtype)), em, er * rstd


LN_SIZES = [(1, 1), (3, 2), (7, 17), (50, 768), (33, 100), (129, 129), (5, 1000), (20, 4096),
            (9, 5001), (2, 70000), (1030, 8), (4, 16384), (300, 256)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d", LN_SIZES)
def test_layer_norm(fk, N, d, dtype):
    t = TYPES[dtype]
    X = rnd((N, d), t, 1, shift=0.5)
    gamma, beta = rnd((d,), seed=2, shift=1.0), rnd((d,), seed=3)
    Y = torch.full_like(X, float("nan"))
    mean, rstd = (torch.full((N,), float("nan"), device="cuda") for _ in range(2))
    fk.fk_layer_norm(X, gamma, beta, Y, 1e-5, mean, rstd)
    y, m, r = ref.layer_norm(X, gamma, beta, 1e-5)
    ty, tm, tr = ln_tol(X, gamma, beta, 1e-5, t)
    within(Y, y, ty, "Y")
    within(mean, m, tm, "mean")
    within(rstd, r, tr, "rstd")
    # no parameters, no statistics, in place
    X2 = X.clone()
    fk.fk_layer_norm(X2, None, None, X2)
    y2 = ref.layer_norm(X, None, None, 1e-5)[0]
    within(X2, y2, ln_tol(X, None, None, 1e-5, t)[0], "in place")


@pytest.mark.parametrize("N,d", [(50001, 64), (45000, 256), (25003, 512), (20001, 760), (15000, 1024),
                                 (7001, 2000), (3333, 4096), (1999, 8192)])
def test_layer_norm_with_many_rows_a_block(fk, N, d):
    """Every block takes many turns of rows, the last ones without a row for some groups."""
    test_layer_norm(fk, N, d, "bf16")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_norm_rows_of_one_value_and_special_values(fk, dtype):
    t = TYPES[dtype]
    X = rnd((6, 40), t, 4)
    X[0] = 3.0  # no variance: h = 0
    X[1, 7] = float("inf")
    X[2, 3] = float("nan")
    X[3] = 0.0
    Y = torch.empty_like(X)
    rstd = torch.empty(6, device="cuda")
    fk.fk_layer_norm(X, None, None, Y, 1e-5, None, rstd)
    assert torch.all(Y[0] == 0) and torch.all(Y[3] == 0)
    assert abs(float(rstd[0]) - 1e-5 ** -0.5) < 1e-3
    assert bool(Y[1].isnan().all()) and bool(Y[2].isnan().all())  # as the formula gives
    within(Y[4:], ref.layer_norm(X[4:], None, None, 1e-5)[0],
           ln_tol(X[4:], None, None, 1e-5, t)[0])


def lnb_tols(dY, X, gamma, mean, rstd, dtype):
    dy, r = dY.double(), rstd.double()[:, None]
    N, d = dy.shape
    c = (X.double() - mean.double()[:, None]).abs()
    h = c * r
    eh = 3 * U * h  # one subtraction (of given values), one product
    w = dy.abs() * (1 if gamma is None else gamma.double().abs())
    n = d / 16 + 24
    e1 = n * U * w.mean(1, keepdim=True)
    e2 = (n + 4) * U * (w * h).mean(1, keepdim=True)
    b = (w * h).mean(1, keepdim=True)
    ex = r * (4 * U * (w + w.mean(1, keepdim=True) + h * b) + e1 + h * e2 + eh * b)
    dx, dg, db = ref.layer_norm_backward(dY, X, gamma, mean, rstd)
    nr = N / 8 + 64  # longest chain of additions down a column
    eg = nr * U * (dy.abs() * h).sum(0) + (dy.abs() * eh).sum(0) + U * dg.abs()
    eb = nr * U * dy.abs().sum(0)
    return half_step(dtype) * dx.abs() + ex * (1 + half_step(dtype)), eg, eb


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d", LN_SIZES + [(3001, 96), (700, 3), (2000, 2500)])
def test_layer_norm_backward(fk, N, d, dtype):
    t = TYPES[dtype]
    X, dY = rnd((N, d), t, 1, shift=0.5), rnd((N, d), t, 5)
    gamma = rnd((d,), seed=2, shift=1.0)
    _, m, r = ref.layer_norm(X, None, None, 1e-5)
    m, r = m.float(), r.float()
    ws = fk.layer_norm_backward_workspace(N, d, t)
    dX = torch.full_like(X, float("nan"))
    dg, db = (torch.full((d,), float("nan"), device="cuda") for _ in range(2))
    fk.fk_layer_norm_backward(dY, X, gamma, m, r, dX, dg, db, ws)
    want = ref.layer_norm_backward(dY, X, gamma, m, r)
    tol = lnb_tols(dY, X, gamma, m, r, t)
    for name, a, b, c in zip(("dX", "dgamma", "dbeta"), (dX, dg, db), want, tol):
        within(a, b, c, name)
    # each output alone, in place, without gamma; the same bits
    dg2, db2, dY2 = torch.empty_like(dg), torch.empty_like(db), dY.clone()
    fk.fk_layer_norm_backward(dY, X, gamma, m, r, None, dg2, None, ws)
    fk.fk_layer_norm_backward(dY, X, gamma, m, r, None, None, db2, ws)
    fk.fk_layer_norm_backward(dY2, X, gamma, m, r, dY2, None, None, ws)
    assert torch.equal(dg2, dg) and torch.equal(db2, db) and torch.equal(dY2, dX)
    fk.fk_layer_norm_backward(dY, X, None, m, r, dX, dg2, db2, ws)
    within(dX, ref.layer_norm_backward(dY, X, None, m, r)[0],
           lnb_tols(dY, X, None, m, r, t)[0], "dX without gamma")
    assert torch.equal(dg2, dg) and torch.equal(db2, db)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [1, 64])
def test_layer_norm_backward_of_rows_without_a_gradient(fk, d, dtype):
    """One column, or columns that all have the same w and no variance: w - mean(w) and h are
    exactly 0, and so is dX."""
    t = TYPES[dtype]
    X = rnd((70, 1), t, 1, shift=0.5).expand(70, d).contiguous()
    dY = rnd((70, 1), t, 2).expand(70, d).contiguous()
    gamma = torch.full((d,), 0.7, device="cuda")
    mean, rstd = X[:, 0].float().contiguous(), torch.full((70,), 1e-5 ** -0.5, device="cuda")
    for g in (None, gamma):
        dX = torch.full_like(X, float("nan"))
        fk.fk_layer_norm_backward(dY, X, g, mean, rstd, dX, None, None,
                                  fk.layer_norm_backward_workspace(70, d, t))
        assert torch.all(dX == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d", [3, 40, 129, 768, 1000, 1024, 5001, 9000])
def test_layer_norm_of_constant_rows(fk, d, dtype):
    """Rows of one value, in both directions.  A mean of d equal values is off by the roundings of
    its sum (d / 16 additions and 24 more) and of 1 / d: n u of the value.  Forward, x - mean is that
    and rstd at most 1 / sqrt(eps); backward, w - mean(w) is that, and h, formed from a mean that is
    the value itself, is 0."""
    t = TYPES[dtype]
    n = d / 16 + 24
    X = rnd((70, 1), t, 1, shift=0.5).expand(70, d).contiguous()
    Y, mean, rstd = torch.empty_like(X), *(torch.empty(70, device="cuda") for _ in range(2))
    fk.fk_layer_norm(X, None, None, Y, 1e-5, mean, rstd)
    x = X[:, :1].double()
    assert bool((Y.double().abs() <= 1.01 * n * U * x.abs() * 1e-5 ** -0.5).all())
    assert bool(((mean.double() - x[:, 0]).abs() <= n * U * x[:, 0].abs()).all())
    dY = rnd((70, 1), t, 2).expand(70, d).contiguous()
    gamma = torch.full((d,), 0.7, device="cuda")
    mean, rstd = X[:, 0].float().contiguous(), torch.full((70,), 1e-5 ** -0.5, device="cuda")
    for g in (None, gamma):
        dX = torch.full_like(X, float("nan"))
        fk.fk_layer_norm_backward(dY, X, g, mean, rstd, dX, None, None,
                                  fk.layer_norm_backward_workspace(70, d, t))
        w = dY[:, :1].double().abs() * (1.0 if g is None else 0.7)
        assert bool((dX.double().abs() <= 1.01 * (n + 4) * U * w * 1e-5 ** -0.5).all())


@pytest.mark.parametrize("N,d", [(2003, 1000), (1501, 1024), (1201, 1800), (900, 2048)])
def test_layer_norm_backward_of_wide_fp32_rows(fk, N, d):
    test_layer_norm_backward(fk, N, d, "f32")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d", [(70, 768), (33, 4096), (40, 129), (9, 9000)])
def test_layer_norm_backward_far_from_zero(fk, N, d, dtype):
    """A mean a thousand times the spread: h = (x - mean) rstd must not be formed as a
    difference of products."""
    t = TYPES[dtype]
    X, dY = rnd((N, d), t, 1, shift=1000.0), rnd((N, d), t, 5)
    _, m, r = ref.layer_norm(X, None, None, 1e-5)
    m, r = m.float(), r.float()
    dX = torch.empty_like(X)
    dg, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    fk.fk_layer_norm_backward(dY, X, None, m, r, dX, dg, db,
                              fk.layer_norm_backward_workspace(N, d, t))
    want, tol = ref.layer_norm_backward(dY, X, None, m, r), lnb_tols(dY, X, None, m, r, t)
    for name, a, b, c in zip(("dX", "dgamma", "dbeta"), (dX, dg, db), want, tol):
        within(a, b, c, name)


# ---------------------------------------------------------------------------------- linear

def act_err(z, y, ez, slope_max=1.13):
    """Error of act(z) for z off by ez: |act'| <= 1.13, and the function itself within a few
    units of |z| (the erf form subtracts near -1) and of its value."""
    return slope_max * ez + 10 * U * (z.abs() + y.abs())


def linear_tols(X, W, b, act, R, dtype):
    d = X.shape[1]
    y, z = ref.linear(X, W, b, act, R)
    mag = X.double().abs() @ W.double().abs().t()
    if b is not None:
        mag = mag + b.double().abs()
    ez = (2.2 * d + 16) * U * mag
    ey = ez if act == "none" else act_err(z, y if R is None else y - R.double(), ez)
    if R is not None:
        ey = ey + 2 * U * (y.abs() + R.double().abs())
    hs = half_step(dtype)
    return y, z, hs * y.abs() + ey * (1 + hs), hs * z.abs() + ez * (1 + hs)


LIN_SIZES = [(1, 1, 1), (1, 16, 16), (3, 5, 7), (2, 4096, 30), (5, 600, 33), (11, 333, 50),
             (16, 512, 70), (1, 768, 768), (8, 768, 129), (9, 64, 1000),
             (17, 100, 300), (50, 768, 256), (127, 129, 131), (128, 64, 256), (300, 257, 513),
             (257, 1000, 65), (1000, 72, 4), (4, 4096, 40), (64, 2048, 64), (130, 4104, 520),
             (1025, 320, 1100)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,m", LIN_SIZES)
def test_linear(fk, N, d, m, dtype):
    t = TYPES[dtype]
    X, W = rnd((N, d), t, 1), rnd((m, d), t, 2, d ** -0.5)
    b, R = rnd((m,), seed=3), rnd((N, m), t, 4)
    ws = fk.linear_workspace(N, d, m, t)
    for act, bias, res, save in (("none", b, None, False), ("gelu", b, R, True),
                                 ("relu", None, None, True), ("silu", b, R, False)):
        Y = torch.full((N, m), float("nan"), dtype=t, device="cuda")
        Z = torch.full_like(Y, float("nan")) if save else None
        fk.fk_linear(X, W, Y, ws, bias=bias, act=act, residual=res, Z=Z)
        y, z, ty, tz = linear_tols(X, W, bias, act, res, t)
        within(Y, y, ty, f"Y {act}")
        if save:
            within(Z, z, tz, f"Z {act}")
        if res is not None:  # in place on the residual
            Y2 = res.clone()
            fk.fk_linear(X, W, Y2, ws, bias=bias, act=act, residual=Y2)
            assert torch.equal(Y2, Y)
    assert fk.fk_get_device_error(ws) == fk.FK_OK


def linear_backward_tols(dY, X, W, act, Z, dtype):
    """G = dY act'(Z) is off by a few units and, as a bf16 operand, by half a bf16 step; each
    product then by the sum over |G| |operand| of that and of the accumulation."""
    N, m = dY.shape
    d = X.shape[1]
    hs = half_step(dtype)
    g = dY.double()
    eg = torch.zeros_like(g)
    if act != "none":
        z = Z.double()
        g = g * ref.slope(z, act)
        eg = dY.double().abs() * 16 * U * (1 + z.abs())
    eop = eg + (hs * g.abs() if dtype == torch.bfloat16 and act != "none" else 0)
    dx, dw, db = ref.linear_backward(dY, X, W, act, Z)
    aw, ax = W.double().abs(), X.double().abs()
    ex = eop @ aw + (2.2 * m + 16) * U * (g.abs() @ aw)
    ew = eop.t() @ ax + (2.2 * N + 16) * U * (g.abs().t() @ ax)
    eb = eg.sum(0) + (N / 8 + 64) * U * g.abs().sum(0)
    return (dx, dw, db), (hs * dx.abs() + ex * (1 + hs), hs * dw.abs() + ew * (1 + hs), eb)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,m", LIN_SIZES + [(5000, 96, 40), (20000, 8, 24), (4097, 300, 264)])
def test_linear_backward(fk, N, d, m, dtype):
    t = TYPES[dtype]
    X, W, dY = rnd((N, d), t, 1), rnd((m, d), t, 2, d ** -0.5), rnd((N, m), t, 5)
    Z = rnd((N, m), t, 6)
    ws = fk.linear_backward_workspace(N, d, m, t)
    for act in ("none", "relu", "gelu", "silu"):
        dX, dW = torch.full_like(X, float("nan")), torch.full_like(W, float("nan"))
        db = torch.full((m,), float("nan"), device="cuda")
        z = None if act == "none" else Z
        fk.fk_linear_backward(dY, X, W, ws, act=act, Z=z, dX=dX, dW=dW, dbias=db)
        want, tol = linear_backward_tols(dY, X, W, act, z, t)
        for name, a, b, c in zip(("dX", "dW", "dbias"), (dX, dW, db), want, tol):
            within(a, b, c, f"{name} {act}")
        # each output alone gives the same bits
        for name, full in (("dX", dX), ("dW", dW), ("dbias", db)):
            one = torch.full_like(full, float("nan"))
            fk.fk_linear_backward(dY, X, W, ws, act=act, Z=z, **{name: one})
            assert torch.equal(one, full), (name, act)
    assert fk.fk_get_device_error(ws) == fk.FK_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,m", [(20001, 64, 520), (21000, 40, 333), (9000, 200, 1032)])
def test_linear_with_many_tiles_a_block(fk, N, d, m, dtype):
    """Every block takes several tiles of a short depth."""
    test_linear(fk, N, d, m, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,d,m", [(1001, 300, 129), (2900, 136, 100), (6500, 40, 768)])
def test_linear_backward_with_many_parts_of_the_bias(fk, N, d, m, dtype):
    """The bias gradient's parts are summed with the cut products' or by themselves."""
    test_linear_backward(fk, N, d, m, dtype)


@pytest.mark.parametrize("N,d,m", [(135000, 40, 24), (131200, 128, 100)])
def test_linear_backward_bf16_over_very_many_rows(fk, N, d, m):
    """dW's depth is past what one accumulation takes."""
    test_linear_backward(fk, N, d, m, "bf16")


@pytest.mark.parametrize("depth", [64, 700, 4096, 40000])
def test_linear_fp32_error_does_not_grow_with_the_depth(fk, depth):
    """Sums of `depth` products of fp32 numbers, in both passes.  The accumulator of the tensor
    cores cuts at most 2^-23 of the sum at each of the 16 steps of a run of 256 (and of the few
    steps that lead up to it); the runs are added with rounding to nearest.  With the running
    sum averaging half its end, that is 16 2^-24 = 9.5e-7 if every cut were the largest; half
    of that on average, and the runs' own signs and the plain roundings well inside the rest."""
    N, m = 96, 80
    g = torch.Generator(device="cuda").manual_seed(depth)
    A = torch.randn((N, depth), generator=g, device="cuda")
    B = torch.randn((m, depth), generator=g, device="cuda")

    def off(got, want):
        return float((got.double() - want).norm() / want.norm())

    Y = torch.empty((N, m), device="cuda")
    fk.fk_linear(A, B, Y, fk.linear_workspace(N, depth, m))
    want = A.double() @ B.double().t()
    assert off(Y, want) <= 9.5e-7
    # dX over the outputs, dW over the rows
    dX = torch.empty((N, m), device="cuda")
    fk.fk_linear_backward(A, torch.zeros((N, m), device="cuda"), B.t().contiguous(),
                          fk.linear_backward_workspace(N, m, depth), dX=dX)
    assert off(dX, want) <= 9.5e-7
    dW = torch.empty((N, m), device="cuda")
    At, Bt = A.t().contiguous(), B.t().contiguous()
    fk.fk_linear_backward(At, Bt, torch.zeros((N, m), device="cuda"),
                          fk.linear_backward_workspace(depth, m, N), dW=dW)
    assert off(dW, want) <= 9.5e-7


def test_linear_fp32_of_positive_terms_over_a_very_long_depth(fk):
    """Whole tiles over 400,000 rows, where every cut and every rounding goes with the sum.  A
    run's cuts are at most 16 2^-24 = 9.5e-7 of it and half of that on average; a chain of r
    additions with rounding to nearest is off by 2^-24 sqrt(r) / 3 (each by u / sqrt(3) of the
    running sum, whose mean square is a third of its end), which for the 256 runs of 65,536 rows
    is 3.2e-7 and for all of 400,000 rows would be 7.9e-7."""
    N, d, m = 400_000, 2048, 1280
    X, dY = rnd((N, d), seed=1).abs_(), rnd((N, m), seed=2).abs_()
    dW = torch.empty((m, d), device="cuda")
    fk.fk_linear_backward(dY, X, dW.clone(), fk.linear_backward_workspace(N, d, m), dW=dW)
    want = dY[:, :64].double().t() @ X[:, :64].double()
    e = (dW[:64, :64].double() - want) / want
    assert float(e.square().mean().sqrt()) <= math.hypot(4.8e-7, 3.2e-7)


def test_linear_fp32_few_rows_of_a_very_long_depth(fk):
    """Few rows add up in chains of at most 2^13 a thread: 2^-24 sqrt(2^13) / 3 = 1.8e-6, over 128
    threads 1.6e-7; runs of 2^20 are joined one after the other (of 32: 1.1e-7)."""
    for N, d in ((2, 1 << 20), (1, (1 << 20) + 4), (16, (1 << 20) + 3), (2, 1 << 22), (3, (1 << 22) + 8), (2, 1 << 25), (1, (1 << 25) + 1)):
        X, W = rnd((N, d), seed=1).abs_(), rnd((5, d), seed=2).abs_()
        Y = torch.empty((N, 5), device="cuda")
        fk.fk_linear(X, W, Y, fk.linear_workspace(N, d, 5))
        want = X.double() @ W.double().t()
        e = (Y.double() - want) / want
        assert float(e.square().mean().sqrt()) <= math.hypot(4.8e-7, 3.2e-7), d


def test_linear_bf16_over_a_very_long_depth(fk):
    """A gradient over 300,000 rows: the depth is cut into parts, and the error stays that of
    one rounding to bf16 (2^-8 at most, a third of that on average)."""
    N, d, m = 300_001, 24, 40
    X, dY = rnd((N, d), torch.bfloat16, 1, shift=0.1), rnd((N, m), torch.bfloat16, 2, shift=0.1)
    W = rnd((m, d), torch.bfloat16, 3)
    dW = torch.empty_like(W)
    fk.fk_linear_backward(dY, X, W, fk.linear_backward_workspace(N, d, m, torch.bfloat16), dW=dW)
    want = dY.double().t() @ X.double()
    assert float(((dW.double() - want).abs() / want.abs()).max()) <= half_step(torch.bfloat16) * 1.1


def test_linear_fp32_keeps_every_bit_of_its_operands(fk):
    """One-term sums: the product of two fp32 numbers to fp32 accuracy, over a wide range of
    exponents."""
    N, m = 64, 48
    g = torch.Generator(device="cuda").manual_seed(8)
    X = torch.randn((N, 1), generator=g, device="cuda") * torch.exp(
        10 * torch.randn((N, 1), generator=g, device="cuda"))
    W = torch.randn((m, 1), generator=g, device="cuda") * torch.exp(
        10 * torch.randn((m, 1), generator=g, device="cuda"))
    Y = torch.empty((N, m), device="cuda")
    fk.fk_linear(X, W, Y, fk.linear_workspace(N, 1, m))
    want = X.double() @ W.double().t()
    # three bf16 pieces hold all 24 bits of each; the largest product left out is 2^-24 of the
    # whole (three such), each of six additions truncates at 2^-23, one rounding at the end
    within(Y, want, 16 * U * want.abs())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linear_special_values(fk, dtype):
    t = TYPES[dtype]
    X, W = rnd((40, 32), t, 1), rnd((24, 32), t, 2)
    X[3, 5], X[7, 0], W[9, 1] = float("nan"), float("inf"), float("-inf")
    Y = torch.empty((40, 24), dtype=t, device="cuda")
    fk.fk_linear(X, W, Y, fk.linear_workspace(40, 32, 24, t))
    bad = torch.zeros(40, 24, dtype=torch.bool, device="cuda")
    bad[3], bad[7], bad[:, 9] = True, True, True
    # a NaN or infinite operand leaves no finite result where it takes part, and no trace
    # anywhere else
    assert bool((~Y[bad].isfinite()).all()) and bool(Y[3].isnan().all())
    assert bool(Y[~bad].isfinite().all())


# --------------------------------------------------------------------------------- balance

def balance_tols(S, labels, counts, n, scale, coef, dtype):
    K = S.shape[1]
    x = (scale * S.double())
    x = torch.where(x.isfinite(), x.abs(), torch.zeros_like(x))
    # p = exp(x - max) / sum: the argument is off by a few u of |x|, exp by a few u, the sum of
    # K terms over at least 16 lanes by K / 16 u
    ep = U * (6 * x.max(1, keepdim=True).values + K / 16 + 32)
    loss, dS = ref.balance(S, labels, counts, n, scale, coef)
    f = counts.double() / (max(n, 1) * (labels.numel() // max(labels.shape[0], 1)))
    kept = ref._kept(labels, K)[2]
    xx = torch.where(kept[:, None], scale * S.double(), torch.zeros_like(x))
    p = torch.softmax(xx, 1).nan_to_num() * kept[:, None]
    t = (p * f).sum(1, keepdim=True)
    c = coef * scale * K / max(n, 1)
    e = abs(c) * p * (2 * ep + 8 * U) * (f + t)
    hs = half_step(dtype)
    el = abs(coef) * K / max(n, 1) * (2 * ep * t).sum() + 4 * U * loss.abs()
    return loss, dS, el, hs * dS.abs() + e * (1 + hs) + 1e-40


BAL_SIZES = [(1, 1, 1), (1, 2, 1), (5, 3, 2), (100, 8, 2), (257, 64, 2), (1000, 60, 3),
             (33, 129, 8), (500, 256, 4), (65, 1000, 1), (40, 2048, 2), (9, 4097, 1),
             (20, 8192, 8), (3, 70000, 1), (3000, 16, 1), (10, 40000, 300),
             (40000, 4096, 1), (6, 12288, 2), (7, 12256, 1), (30000, 6, 3)]


def make_labels(N, K, top, seed, pad):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lab = (torch.rand((N, top), generator=g, device="cuda") ** 2 * K).to(torch.int32).clamp(
        max=K - 1)
    drop = torch.rand((N, top), generator=g, device="cuda") < 0.2
    if top > 1:
        lab[drop] = -1  # single dropped selections
    lab[torch.rand((N,), generator=g, device="cuda") < pad] = -1
    return lab


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,K,top", BAL_SIZES)
def test_balance(fk, N, K, top, dtype):
    t = TYPES[dtype]
    for pad, scale, coef in ((0.0, 1.0, 1.0), (0.3, 2.5, 0.01), (1.1, 1.0, 1.0)):
        S = rnd((N, K), t, 7, 2.0)
        lab = make_labels(N, K, top, 3, pad)
        padded = ~ref._kept(lab, K)[2]
        S[padded] = float("nan")  # never looked at
        if K > 3:
            S[:, 1] = float("-inf")  # a masked cell
        counts = torch.full((K,), -5, dtype=torch.int32, device="cuda")
        rows = torch.full((1,), -5, dtype=torch.int32, device="cuda")
        fk.fk_balance_counts(lab if top > 1 else lab[:, 0].contiguous(), counts, rows)
        want_c, n = ref.balance_counts(lab, K)
        assert torch.equal(counts.long(), want_c) and int(rows) == n
        loss = torch.full((1,), float("nan"), device="cuda")
        dS = torch.full_like(S, float("nan"))
        ws = fk.balance_workspace(N, K, t)
        fk.fk_balance_loss(S, lab, counts, rows, loss, dS, ws, scale, coef)
        S0 = torch.where(padded[:, None], torch.zeros_like(S), S)
        wl, wd, tl, td = balance_tols(S0, lab, counts, n, scale, coef, t)
        within(loss, wl.reshape(1), tl, "loss")
        within(dS, wd, td, "dS")
        loss2, S2 = torch.empty_like(loss), S.clone()
        fk.fk_balance_loss(S2, lab, counts, rows, loss2, None, ws, scale, coef)
        assert torch.equal(loss2, loss)
        fk.fk_balance_loss(S2, lab, counts, rows, loss2, S2, ws, scale, coef)  # in place
        assert torch.equal(loss2, loss) and torch.equal(S2, dS)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [1, 3, 8, 64, 129, 4096, 9000])
def test_balance_of_an_even_selection_has_no_gradient(fk, K, dtype):
    """Every cell selected equally often: f_j - t_i is 0 for every score, and exactly so."""
    t = TYPES[dtype]
    S = rnd((2 * K, K), t, 3, 2.0) if K <= 129 else rnd((K, K), t, 3, 2.0)
    N = S.shape[0]
    lab = (torch.arange(N, dtype=torch.int32, device="cuda") % K).reshape(N, 1)
    counts = torch.empty(K, dtype=torch.int32, device="cuda")
    rows = torch.empty(1, dtype=torch.int32, device="cuda")
    fk.fk_balance_counts(lab, counts, rows)
    assert int(counts.min()) == int(counts.max()) == N // K
    loss, dS = torch.empty(1, device="cuda"), torch.full_like(S, 9.0)
    fk.fk_balance_loss(S, lab, counts, rows, loss, dS, fk.balance_workspace(N, K, t))
    assert torch.all(dS == 0)
    assert abs(float(loss) - 1.0) <= 4 * U  # K (1 / K) to a few roundings


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [5, 300, 5000])
def test_balance_rows_that_masks_leave_empty(fk, K, dtype):
    t = TYPES[dtype]
    S = rnd((6, K), t, 1)
    S[0] = float("-inf")
    S[1] = torch.finfo(t).min  # the type's lowest value everywhere: an even row
    S[2, 1:] = float("-inf")
    S[3, 0] = float("inf")
    S[4, 1] = float("nan")
    lab = torch.arange(6, dtype=torch.int32, device="cuda").reshape(6, 1) % K
    lab[5] = K + 7  # outside: selects nothing, so the row is padding
    counts = torch.empty(K, dtype=torch.int32, device="cuda")
    rows = torch.empty(1, dtype=torch.int32, device="cuda")
    fk.fk_balance_counts(lab, counts, rows)
    assert int(rows) == 5 and int(counts.sum()) == 5
    loss, dS = torch.empty(1, device="cuda"), torch.full_like(S, 9.0)
    ws = fk.balance_workspace(6, K, t)
    fk.fk_balance_loss(S, lab, counts, rows, loss, dS, ws)
    assert bool(dS[3].isnan().any()) and bool(dS[4].isnan().all()) and bool(loss.isnan())
    assert torch.all(dS[0] == 0) and torch.all(dS[5] == 0)
    f = counts.double() / 5
    even = K / 5 * (f - f.mean()) / K
    # p = 1/K to a few u (K / 16 additions), f and t likewise
    within(dS[1], even, half_step(t) * even.abs() + (K / 8 + 64) * U * (f + f.mean()) / 5, "even")
    # p = 1 at one cell: t = f_0 there, up to rounding
    assert float(dS[2].float().abs().max()) <= 8 * U * K / 5


def balance_difference_tols(S, labels, counts, n, scale, coef, dtype):
    """Bounds that know differences of scores only.  x = scale (s - max) is formed in four
    roundings (the difference, log2(e), its product with the scale, the product), so it is off by
    4 u |x|; a warp's maximum in between splits x in two parts of that kind.  2^x is within 4 u,
    twice where the warps' sums are joined; the sum of K terms over at least 16 lanes K / 16 u and
    its reciprocal a few.  A probability under 2^-126 may be 0, which takes up to 2^-125 from p and,
    as the shares add up to at most 1, from t.  An output is rounded to a multiple of its type's
    least subnormal, and two of its factors to one of fp32's."""
    K = S.shape[1]
    kept = (ref._kept(labels, K)[2] & (S > -math.inf).any(1))[:, None]  # rows that have any p
    x = torch.where(kept, scale * S.double(), torch.zeros((), dtype=torch.float64, device="cuda"))
    x = x - x.max(1, keepdim=True).values
    p = torch.softmax(x, 1) * kept
    ep = 4 * U * torch.where(p > 0, -x, torch.zeros_like(x))
    ep = ep + (p * ep).sum(1, keepdim=True) + U * (K / 16 + 32)
    f = counts.double() / (max(n, 1) * (labels.numel() // labels.shape[0]))
    t = (p * f).sum(1, keepdim=True)
    et = (p * f * (ep + 8 * U)).sum(1, keepdim=True) + 2.0 ** -125
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    c = abs(coef) * K / max(n, 1)
    loss, dS = ref.balance(S, labels, counts, n, scale, coef)
    e = c * scale * (p * ((ep + 8 * U) * (f + t) + et) + 2.0 ** -125 * (f + t))
    hs = half_step(dtype)
    return (loss, dS, c * et.sum() + 4 * U * loss.abs(),
            hs * dS.abs() + e * (1 + hs) + least / 2 + 2.0 ** -149)


def check_balance(fk, S, lab, scale=1.0, coef=1.0):
    N, K = S.shape
    counts, rows = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (K, 1))
    fk.fk_balance_counts(lab, counts, rows)
    loss, dS = torch.empty(1, device="cuda"), torch.full_like(S, 9.0)
    fk.fk_balance_loss(S, lab, counts, rows, loss, dS, fk.balance_workspace(N, K, S.dtype), scale,
                       coef)
    wl, wd, tl, td = balance_difference_tols(S, lab, counts, int(rows), scale, coef, S.dtype)
    within(loss, wl.reshape(1), tl, "loss")
    within(dS, wd, td, "dS")


BIG_K = [16, 64, 300, 1000, 4096, 4097, 8192, 9000]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", BIG_K)
def test_balance_rows_of_one_large_score(fk, K, dtype):
    """Rows of one value, whatever its size: p = 1 / K.  Also with one score far above."""
    values = [v for b in (1e3, 1e4, 1e5, 1e9, 1e10, 1e12, 1e20, 1e30, 3e38) for v in (b, -b)]
    S = torch.tensor(values, device="cuda").reshape(-1, 1).expand(-1, K)
    lab = make_labels(len(values), K, 2, 3, 0.0)
    check_balance(fk, S.to(TYPES[dtype]).contiguous(), lab)
    S = rnd((len(values), K), TYPES[dtype], 4, 2.0)
    S[:, K // 3] = torch.tensor(values, device="cuda").abs().to(TYPES[dtype])
    check_balance(fk, S, lab)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", BIG_K)
def test_balance_of_rows_masked_by_large_scores(fk, K, dtype):
    """All cells but one to sixteen are masked by a large negative score; the masked row that
    keeps none is even."""
    t = TYPES[dtype]
    for mask in (-1e3, -1e4, -1e9, -1e10, -1e12, -1e30, -3e38):
        S = torch.full((20, K), mask, device="cuda").to(t)
        real = rnd((20, K), t, 6, 2.0)
        for i in range(1, 20):
            at = torch.arange(min(i, 16), device="cuda") * (K // min(i, 16)) + i % 7 % (K // 16)
            S[i, at] = real[i, at]
        check_balance(fk, S, make_labels(20, K, 3, 5, 0.1))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", BIG_K)
def test_balance_of_shifted_scores(fk, K, dtype):
    """A common offset of a row's scores, as that of |c|^2 / 2: the bounds do not grow with it."""
    for shift in (0.0, -400.0, 1e3, -1e4, 1e5, -1e6):
        S = rnd((50, K), torch.float32, 7, 2.0)
        S = (S + shift * torch.linspace(0.5, 1, 50, device="cuda")[:, None]).to(TYPES[dtype])
        check_balance(fk, S, make_labels(50, K, 1, 8, 0.1), 0.7, -3.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", BIG_K)
def test_balance_with_a_large_or_small_scale(fk, K, dtype):
    lab = make_labels(50, K, 2, 9, 0.1)
    for scale, size in ((2.0 ** 30, 10.0), (2.0 ** 10, 1e6), (2.0 ** 100, 1e-25), (2.0 ** -40, 1e13),
                        (2.0 ** -100, 1e30)):
        check_balance(fk, rnd((50, K), TYPES[dtype], 10, size), lab, scale, 2.0 ** -20)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [5, 64, 4096, 9000])
def test_balance_at_the_largest_gradients(fk, K, dtype):
    """coef scale K just below its limit: padding rows and rows of -inf still get zeros."""
    t = TYPES[dtype]
    S = rnd((12, K), t, 11, 2.0)
    S[3] = float("-inf")
    lab = make_labels(12, K, 1, 12, 0.0)
    lab[5] = -1
    scale = 2.0 ** 100
    for coef in (9.9e37 / scale / K, -9.9e37 / scale / K):
        check_balance(fk, S, lab, scale, coef)
        counts, rows = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (K, 1))
        fk.fk_balance_counts(lab, counts, rows)
        loss, dS = torch.empty(1, device="cuda"), torch.full_like(S, 9.0)
        ws = fk.balance_workspace(12, K, t)
        fk.fk_balance_loss(S, lab, counts, rows, loss, dS, ws, scale, coef)
        assert torch.all(dS[3] == 0) and torch.all(dS[5] == 0) and bool(loss.isfinite())
    with pytest.raises(fk.FkError) as e:
        fk.fk_balance_loss(S, lab, counts, rows, loss, dS, ws, scale, 1.01e38 / scale / K)
    assert e.value.status == fk.FK_ERR_INVALID_ARG


# ------------------------------------------------------------- together, streams, graphs

def head_pass(fk, p, bufs, ws, stream=None):
    """The head as it is used: norm, expanding product, projection with residual, norm, then
    scores against centroids, their balance loss, and the gradients of all of it."""
    b = bufs
    s = dict(stream=stream)
    fk.fk_layer_norm(p["H"], p["g1"], p["b1"], b["A"], 1e-5, b["m1"], b["r1"], **s)
    fk.fk_linear(b["A"], p["W1"], b["B"], ws, bias=p["c1"], act="gelu", Z=b["Z1"], **s)
    fk.fk_linear(b["B"], p["W2"], b["D"], ws, bias=p["c2"], residual=p["H"], **s)
    fk.fk_layer_norm(b["D"], p["g2"], p["b2"], b["P"], 1e-5, b["m2"], b["r2"], **s)
    fk.fk_linear(b["P"], p["C"], b["S"], ws, bias=p["half"], **s)
    fk.fk_assign(b["P"], p["C"], b["lab"], b["aws"], **s)
    fk.fk_balance_counts(b["lab"], b["counts"], b["rows"], **s)
    fk.fk_balance_loss(b["S"], b["lab"], b["counts"], b["rows"], b["loss"], b["dS"], ws, 0.1,
                       **s)
    fk.fk_linear_backward(b["dS"], b["P"], p["C"], ws, dX=b["dP"], dW=b["dC"], dbias=b["dh"], **s)
    fk.fk_layer_norm_backward(b["dP"], b["D"], p["g2"], b["m2"], b["r2"], b["dD"], b["dg2"],
                              b["db2"], ws, **s)
    fk.fk_linear_backward(b["dD"], b["B"], p["W2"], ws, dX=b["dB"], dW=b["dW2"], dbias=b["dc2"],
                          **s)
    fk.fk_linear_backward(b["dB"], b["A"], p["W1"], ws, act="gelu", Z=b["Z1"], dX=b["dA"],
                          dW=b["dW1"], dbias=b["dc1"], **s)
    fk.fk_layer_norm_backward(b["dA"], p["H"], p["g1"], b["m1"], b["r1"], b["dH"], b["dg1"],
                              b["db1"], ws, **s)


def head_setup(fk, N=300, d=48, m=72, K=20, t=torch.float32, seed=0):
    f = torch.float32
    p = {"H": rnd((N, d), t, seed + 1), "g1": rnd((d,), f, 2, 0.1, 1.0), "b1": rnd((d,), f, 3, 0.1),
         "W1": rnd((m, d), t, 4, d ** -0.5), "c1": rnd((m,), f, 5, 0.1),
         "W2": rnd((d, m), t, 6, m ** -0.5), "c2": rnd((d,), f, 7, 0.1),
         "g2": rnd((d,), f, 8, 0.1, 1.0), "b2": rnd((d,), f, 9, 0.1), "C": rnd((K, d), t, 10)}
    cn = torch.empty(K, device="cuda")
    fk.fk_centroid_norms(p["C"].float(), cn)
    p["half"] = -cn / 2

    def e(*shape, dtype=t):
        return torch.empty(shape, dtype=dtype, device="cuda")

    b = {"A": e(N, d), "B": e(N, m), "Z1": e(N, m), "D": e(N, d), "P": e(N, d), "S": e(N, K),
         "lab": e(N, dtype=torch.int32), "counts": e(K, dtype=torch.int32),
         "rows": e(1, dtype=torch.int32), "loss": e(1, dtype=f), "dS": e(N, K), "dP": e(N, d),
         "dC": e(K, d), "dD": e(N, d), "dB": e(N, m), "dW2": e(d, m), "dA": e(N, d),
         "dW1": e(m, d), "dH": e(N, d)}
    for k, n in (("m1", N), ("r1", N), ("m2", N), ("r2", N), ("dh", K), ("dg2", d), ("db2", d),
                 ("dc2", d), ("dc1", m), ("dg1", d), ("db1", d)):
        b[k] = e(n, dtype=f)
    b["aws"] = fk.workspace(N, d, K, t, "l2")
    size = max(fk.linear_workspace(N, a, c, t, "meta").numel()
               for a, c in ((d, m), (m, d), (d, K)))
    size = max([size, fk.layer_norm_backward_workspace(N, d, t, "meta").numel(),
                fk.balance_workspace(N, K, t, "meta").numel()] +
               [fk.linear_backward_workspace(N, a, c, t, "meta").numel()
                for a, c in ((d, m), (m, d), (d, K))])
    return p, b, torch.zeros(size, dtype=torch.uint8, device="cuda")


def test_head_together_against_fp64_differentiation(fk):
    p, b, ws = head_setup(fk)
    head_pass(fk, p, b, ws)
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    a = ref.layer_norm(q["H"], q["g1"], q["b1"], 1e-5)[0]
    h = ref.linear(a, q["W1"], q["c1"], "gelu", None)[0]
    dd = ref.linear(h, q["W2"], q["c2"], "none", q["H"])[0]
    pts = ref.layer_norm(dd, q["g2"], q["b2"], 1e-5)[0]
    S = ref.linear(pts, q["C"], q["half"], "none", None)[0]
    # the labels are those of the largest score; take the GPU's for rows that nearly tie
    lab = b["lab"]
    top = S.max(1).values
    assert bool((top - S.gather(1, lab[:, None].long())[:, 0] <= 1e-3).all())
    counts, n = ref.balance_counts(lab, 20)
    assert torch.equal(counts, b["counts"].long()) and n == 300
    prob = torch.softmax(0.1 * S, 1)
    loss = 20 * ((counts.double() / n) * prob.mean(0)).sum()
    loss.backward()
    # every stage is off by about 2.2 n u of sums with n <= 72 terms, about 1e-5 of the largest
    # entry; seven such stages in a row
    assert abs(float(b["loss"]) - loss.item()) <= 1e-4 * loss.item()
    # the residual's gradient joins by hand: dH also gets dD
    dH = b["dH"].double() + b["dD"].double()
    for name, got, want in (("dH", dH, q["H"].grad), ("dW1", b["dW1"], q["W1"].grad),
                            ("dc1", b["dc1"], q["c1"].grad), ("dW2", b["dW2"], q["W2"].grad),
                            ("dc2", b["dc2"], q["c2"].grad), ("dg1", b["dg1"], q["g1"].grad),
                            ("db1", b["db1"], q["b1"].grad), ("dg2", b["dg2"], q["g2"].grad),
                            ("db2", b["db2"], q["b2"].grad), ("dC", b["dC"], q["C"].grad),
                            ("dh", b["dh"], q["half"].grad)):
        within(got, want, 2e-4 * want.abs().max() + 0 * want, name)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_repeats_streams_and_graphs_give_the_same_bits(fk, dtype):
    t = TYPES[dtype]
    p, b, ws = head_setup(fk, 700, 64, 128, 33, t)
    p["C"] = p["C"].float() if dtype == "f32" else p["C"]

    def run(stream=None):
        if dtype == "f32":
            head_pass(fk, p, b, ws, stream)
        else:  # fk_assign takes fp32 centroids
            q = dict(p)
            fk_assign = fk.fk_assign
            C32 = p["C"].float()
            torch.cuda.synchronize()

            class Shim:
                def __getattr__(self, name):
                    if name == "fk_assign":
                        return lambda X, C, lab, w, stream=None: fk_assign(X, C32, lab, w,
                                                                           stream=stream)
                    return getattr(fk, name)
            head_pass(Shim(), q, b, ws, stream)

    outs = [k for k in b if k != "aws"]
    run()
    torch.cuda.synchronize()
    first = {k: b[k].clone() for k in outs}

    def same():
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(b[k], first[k]), k
            b[k].fill_(3)

    same()
    run()
    same()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    run(side)
    same()
    if dtype == "f32":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        for _ in range(2):
            ws.fill_(0xA5)  # nothing of the workspace is kept from call to call
            ws[:256] = 0
            graph.replay()
            same()
        # other values through the same graph
        H0 = p["H"].clone()
        p["H"].mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: b[k].clone() for k in outs}
        run()
        torch.cuda.synchronize()
        for k in outs:
            assert torch.equal(b[k], got[k]), k
        p["H"].copy_(H0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,m", [(65, 33), (64, 40)])
def test_unaligned_views_give_the_aligned_bits(fk, d, m, dtype):
    """Rows behind an odd offset: the operators take any element-aligned pointer."""
    t = TYPES[dtype]
    N = 70

    def off(x):
        buf = torch.empty(x.numel() + 9, dtype=x.dtype, device="cuda")
        v = buf[1:1 + x.numel()].view(x.shape)
        v.copy_(x)
        return v

    X, W, dY, Z = rnd((N, d), t, 1), rnd((m, d), t, 2), rnd((N, m), t, 3), rnd((N, m), t, 4)
    bias, gamma = rnd((m,), seed=5), rnd((d,), seed=6)
    outs = []
    for f in (lambda x: x, off):
        x, w, dy, z, bi, ga = f(X), f(W), f(dY), f(Z), f(bias), f(gamma)
        y, zz, n = f(torch.empty_like(dY)), f(torch.empty_like(dY)), f(torch.empty_like(X))
        dx, dw = f(torch.empty_like(X)), f(torch.empty_like(W))
        db, dg, dbt = f(torch.empty_like(bias)), f(torch.empty_like(gamma)), f(
            torch.empty_like(gamma))
        mean, rstd = f(torch.empty(N, device="cuda")), f(torch.empty(N, device="cuda"))
        nx = f(torch.empty_like(X))
        fk.fk_linear(x, w, y, fk.linear_workspace(N, d, m, t), bias=bi, act="silu", residual=dy,
                     Z=zz)
        fk.fk_linear_backward(dy, x, w, fk.linear_backward_workspace(N, d, m, t), act="gelu",
                              Z=z, dX=dx, dW=dw, dbias=db)
        fk.fk_layer_norm(x, ga, None, n, 1e-5, mean, rstd)
        fk.fk_layer_norm_backward(x, n, ga, mean, rstd, nx, dg, dbt,
                                  fk.layer_norm_backward_workspace(N, d, t))
        lab = (torch.arange(N, dtype=torch.int32, device="cuda") * 7) % m
        c, r = torch.empty(m, dtype=torch.int32, device="cuda"), torch.empty(
            1, dtype=torch.int32, device="cuda")
        fk.fk_balance_counts(f(lab), c, r)
        loss, ds = f(torch.empty(1, device="cuda")), f(torch.empty_like(dY))
        fk.fk_balance_loss(z, f(lab), c, r, loss, ds, fk.balance_workspace(N, m, t))
        outs.append([v.clone() for v in (y, zz, dx, dw, db, n, mean, rstd, nx, dg, dbt, c, r,
                                         loss, ds)])
    y, z, ty, tz = linear_tols(X, W, bias, "silu", dY, t)
    within(outs[1][0], y, ty, "Y")
    within(outs[1][1], z, tz, "Z")
    want, tol = linear_backward_tols(dY, X, W, "gelu", Z, t)
    for i in range(3):
        within(outs[1][2 + i], want[i], tol[i], ("dX", "dW", "db")[i])
    within(outs[1][5], ref.layer_norm(X, gamma, None, 1e-5)[0],
           ln_tol(X, gamma, None, 1e-5, t)[0], "layer norm")
    assert torch.equal(outs[0][11], outs[1][11]) and torch.equal(outs[0][12], outs[1][12])
    for i in (8, 9, 10, 13, 14):
        a, c = outs[0][i].double(), outs[1][i].double()
        # two orders of the same fp32 sums (of at most 70 terms), then one rounding each
        assert bool(((a - c).abs() <= (2 * half_step(outs[0][i].dtype) + 512 * U)
                     * (c.abs() + c.abs().max())).all()), i


@pytest.mark.parametrize("N,d,m", [(300, 136, 200), (5000, 64, 72), (70, 65, 33)])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("which", ["X", "W", "dY", "Z", "X W"])
def test_linear_backward_with_some_operands_unaligned(fk, N, d, m, act, which):
    """A bf16 operand off 16 bytes changes only the products that read it; each output alone has
    the bits that it has with the others."""
    t = torch.bfloat16
    ts = {"X": rnd((N, d), t, 1), "W": rnd((m, d), t, 2, d ** -0.5), "dY": rnd((N, m), t, 5),
          "Z": rnd((N, m), t, 6)}
    if act == "none":
        ts["Z"] = None
    ws = fk.linear_backward_workspace(N, d, m, t)

    def grads(q, names):
        o = {"dX": torch.empty((N, d), dtype=t, device="cuda"),
             "dW": torch.empty((m, d), dtype=t, device="cuda"),
             "dbias": torch.empty(m, device="cuda")}
        o = {k: o[k].fill_(float("nan")) for k in names}
        fk.fk_linear_backward(q["dY"], q["X"], q["W"], ws, act=act, Z=q["Z"], **o)
        return o

    names = ("dX", "dW", "dbias")
    aligned = grads(ts, names)
    q = dict(ts)
    for k in which.split():
        if q[k] is not None:
            buf = torch.empty(q[k].numel() + 1, dtype=t, device="cuda")
            q[k] = buf[1:].view(q[k].shape).copy_(ts[k])
    got = grads(q, names)
    want, tol = linear_backward_tols(ts["dY"], ts["X"], ts["W"], act, ts["Z"], t)
    for name, a, b in zip(names, want, tol):
        within(got[name], a, b, name)
        assert torch.equal(grads(q, [name])[name], got[name]), name
    # what each product reads as it lies: dX dY and W, dW dY and X (dY not where it is staged)
    staged = act != "none" or m % 8 != 0
    for name, reads in (("dX", "W"), ("dW", "X"), ("dbias", "-")):
        if reads not in which.split() and (staged or which != "dY" or name == "dbias"):
            assert torch.equal(got[name], aligned[name]), name


def test_linear_backward_of_unaligned_operands_over_very_many_rows(fk):
    """Positive terms over 2^23 rows: fp32 sums round to bf16 once, whatever the route."""
    t, N = torch.bfloat16, 1 << 23
    buf = torch.empty(2, N * 8 + 1, dtype=t, device="cuda")
    X, dY = buf[0, 1:].view(N, 8), buf[1, :-1].view(N, 8)
    X.copy_(rnd((N, 8), seed=1).abs_())
    dY.copy_(rnd((N, 8), seed=2).abs_())
    dW = torch.empty((8, 8), dtype=t, device="cuda")
    fk.fk_linear_backward(dY, X, dW.clone(), fk.linear_backward_workspace(N, 8, 8, t), dW=dW)
    want = dY.double().t() @ X.double()
    # a run of 4096 and 2048 runs: (2^-24 / 3)(sqrt(4096) + sqrt(2048)) = 2.2e-6, next to 2^-8
    assert float(((dW.double() - want).abs() / want).max()) <= half_step(t) + 1e-5


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_few_rows_over_a_very_long_depth(fk, dtype):
    t = TYPES[dtype]
    for d in (1 << 20, (1 << 20) + 8, (1 << 20) + 9, (1 << 22) + 1032):
        X, W, b = rnd((2, d), t, 1), rnd((3, d), t, 2, d ** -0.5), rnd((3,), seed=3)
        Y = torch.empty((2, 3), dtype=t, device="cuda")
        fk.fk_linear(X, W, Y, fk.linear_workspace(2, d, 3, t), bias=b)
        want = X.double() @ W.double().t() + b.double()
        # sums of terms with signs: 2^-20 of their magnitudes, 0.64 sqrt(d)
        tol = half_step(t) * want.abs() + 2.0 ** -20 * (0.64 * d ** 0.5 + b.abs().double())
        within(Y, want, tol, d)


def test_calls_on_two_streams_at_once(fk):
    """Two chains of calls that overlap on the GPU, each with a workspace of its own."""
    chains = [head_setup(fk, 3000, 256, 512, 64, seed=s) for s in (0, 50)]
    for p, b, ws in chains:
        head_pass(fk, p, b, ws)
    torch.cuda.synchronize()
    first = [{k: v.clone() for k, v in b.items() if k != "aws"} for _, b, _ in chains]
    streams = [torch.cuda.Stream() for _ in chains]
    for _ in range(5):
        for (p, b, ws), s in zip(chains, streams):
            head_pass(fk, p, b, ws, s)
    torch.cuda.synchronize()
    for (_, b, _), want in zip(chains, first):
        for k, v in want.items():
            assert torch.equal(b[k], v), k


def test_the_first_call_of_a_process_can_be_captured(cuda_device):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = (
        "import sys, torch\n"
        f"sys.path[:0] = [{root!r}, {os.path.join(root, 'tests')!r}]\n"
        "from exact_lloyd_means_b200 import fk\n"
        "t = torch.float32\n"
        "X, W = torch.randn(300, 72, device='cuda'), torch.randn(40, 72, device='cuda')\n"
        "Y, Z = torch.empty(300, 40, device='cuda'), torch.empty(300, 40, device='cuda')\n"
        "n, m, r = torch.empty_like(X), torch.empty(300, device='cuda'), torch.empty(300, "
        "device='cuda')\n"
        "dX, dW = torch.empty_like(X), torch.empty_like(W)\n"
        "ws, wb = fk.linear_workspace(300, 72, 40), fk.linear_backward_workspace(300, 72, 40)\n"
        "lab = torch.arange(300, device='cuda', dtype=torch.int32) % 40\n"
        "c, q = (torch.empty(k, device='cuda', dtype=torch.int32) for k in (40, 1))\n"
        "L, bw = torch.empty(1, device='cuda'), fk.balance_workspace(300, 40)\n"
        "def run():\n"
        "    fk.fk_layer_norm(X, None, None, n, 1e-5, m, r)\n"
        "    fk.fk_linear(n, W, Y, ws, act='gelu', Z=Z)\n"
        "    fk.fk_balance_counts(lab, c, q)\n"
        "    fk.fk_balance_loss(Y, lab, c, q, L, Y, bw)\n"
        "    fk.fk_linear_backward(Y, n, W, wb, act='gelu', Z=Z, dX=dX, dW=dW)\n"
        "torch.cuda.synchronize()\n"
        "g = torch.cuda.CUDAGraph()\n"
        "with torch.cuda.graph(g):\n"
        "    run()\n"
        "g.replay(); torch.cuda.synchronize()\n"
        "a = [v.clone() for v in (Y, dX, dW, L)]\n"
        "run(); torch.cuda.synchronize()\n"
        "print(all(torch.equal(x, y) for x, y in zip(a, (Y, dX, dW, L))), "
        "bool(dW.isfinite().all()))\n")
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["True", "True"]


def test_binding_refuses_tensors_it_would_misread(fk):
    X, W, Y = rnd((12, 8)), rnd((4, 8)), torch.empty((12, 4), device="cuda")
    ws = fk.linear_workspace(12, 8, 4)
    for bad in (dict(X=rnd((8, 12)).t()), dict(W=rnd((8, 4)).t()), dict(Y=Y.t().contiguous().t()),
                dict(W=rnd((4, 9))), dict(bias=rnd((5,))), dict(Y=torch.empty(12, 4)),
                dict(residual=rnd((12, 5))), dict(X=rnd((12, 8, 1)))):
        a = dict(dict(X=X, W=W, Y=Y, ws=ws), **bad)
        with pytest.raises(ValueError):
            fk.fk_linear(**a)
    for bad in (dict(W=W.bfloat16()), dict(Y=Y.bfloat16()), dict(bias=rnd((4,)).double()),
                dict(X=X.half(), W=W.half(), Y=Y.half()), dict(ws=ws.int())):
        a = dict(dict(X=X, W=W, Y=Y, ws=ws), **bad)
        with pytest.raises(TypeError):
            fk.fk_linear(**a)
    with pytest.raises(ValueError):
        fk.fk_linear(X, W, Y, ws, act="tanh")
    with pytest.raises(fk.FkError) as e:
        fk.fk_linear(X, W, Y, ws[:64])
    assert e.value.status == fk.FK_ERR_WORKSPACE
    with pytest.raises(fk.FkError) as e:  # an output over an input
        fk.fk_layer_norm_backward(X, X, None, rnd((12,)), rnd((12,)), X, None, None,
                                  fk.layer_norm_backward_workspace(12, 8))
    assert e.value.status == fk.FK_ERR_INVALID_ARG


def test_no_rows(fk):
    X = torch.empty((0, 24), device="cuda")
    W, v = rnd((8, 24)), rnd((24,))
    Y = torch.empty((0, 8), device="cuda")
    e = torch.empty(0, device="cuda")
    fk.fk_layer_norm(X, v, v, torch.empty_like(X), 1e-5, e, e.clone())
    fk.fk_linear(X, W, Y, fk.linear_workspace(0, 24, 8))
    dW, db = torch.full_like(W, 5.0), torch.full((8,), 5.0, device="cuda")
    fk.fk_linear_backward(Y, X, W, fk.linear_backward_workspace(0, 24, 8),
                          dX=torch.empty_like(X), dW=dW, dbias=db)
    dg, dbt = torch.full((24,), 5.0, device="cuda"), torch.full((24,), 5.0, device="cuda")
    fk.fk_layer_norm_backward(X, X.clone(), v, e, e, torch.empty_like(X), dg, dbt,
                              fk.layer_norm_backward_workspace(0, 24))
    counts, rows = (torch.full((n,), 5, dtype=torch.int32, device="cuda") for n in (8, 1))
    lab = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    fk.fk_balance_counts(lab, counts, rows)
    loss = torch.full((1,), 5.0, device="cuda")
    fk.fk_balance_loss(Y, lab, counts, rows, loss, torch.empty_like(Y),
                       fk.balance_workspace(0, 8))
    for t in (dW, db, dg, dbt, counts, rows, loss):
        assert bool((t == 0).all())


def test_more_than_two_billion_elements(fk):
    """Offsets past 32 bits: the last rows of tensors of 2.1e9 and more elements."""
    t = torch.bfloat16
    N, m = (1 << 20) + 3, 2056
    tail = slice(N - 3, N)
    X, W = rnd((N, 16), t, 1), rnd((m, 16), t, 2, 0.25)
    Y = torch.empty((N, m), dtype=t, device="cuda")
    fk.fk_linear(X, W, Y, fk.linear_workspace(N, 16, m, t))
    y, _, ty, _ = linear_tols(X[tail], W, None, "none", None, t)
    within(Y[tail], y, ty, "linear")
    last = Y[tail].clone()
    mean, rstd = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    fk.fk_layer_norm(Y, None, None, Y, 1e-5, mean, rstd)
    within(Y[tail], ref.layer_norm(last, None, None, 1e-5)[0],
           ln_tol(last, None, None, 1e-5, t)[0], "layer norm")
    lab = torch.zeros(N, dtype=torch.int32, device="cuda")
    lab[tail] = 5
    counts = torch.empty(m, dtype=torch.int32, device="cuda")
    rows = torch.empty(1, dtype=torch.int32, device="cuda")
    fk.fk_balance_counts(lab, counts, rows)
    assert int(counts[0]) == N - 3 and int(counts[5]) == 3 and int(rows) == N
    S = Y[tail].clone()
    loss = torch.empty(1, device="cuda")
    ws = fk.balance_workspace(N, m, t)
    fk.fk_balance_loss(Y, lab, counts, rows, loss, Y, ws, coef=1e6)
    _, wd, _, td = balance_tols(S, lab[tail].reshape(3, 1), counts, N, 1.0, 1e6, t)
    within(Y[tail], wd, td, "balance")
    dX = torch.empty_like(X)
    last = Y[tail].clone()
    fk.fk_linear_backward(Y, X, W, fk.linear_backward_workspace(N, 16, m, t), dX=dX)
    want, tol = linear_backward_tols(last, X[tail], W, "none", None, t)
    within(dX[tail], want[0], tol[0], "linear backward")


def test_launch_fault_is_reported(cuda_device):
    """FK_FAULT=launch (read when the library is first used, so in a child process): every
    call reports a failed launch."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    code = (
        "import sys, torch\n"
        f"sys.path.insert(0, {root!r})\n"
        "from exact_lloyd_means_b200 import fk\n"
        "x = torch.zeros(4, 8, device='cuda'); v = torch.zeros(8, device='cuda')\n"
        "i = torch.zeros(4, dtype=torch.int32, device='cuda')\n"
        "c = torch.zeros(8, dtype=torch.int32, device='cuda')\n"
        "r = torch.zeros(1, dtype=torch.int32, device='cuda')\n"
        "ws = torch.zeros(1 << 20, dtype=torch.uint8, device='cuda')\n"
        "m = torch.zeros(4, device='cuda')\n"
        "w = torch.zeros(8, 8, device='cuda')\n"
        "y = torch.empty_like(x)\n"
        "calls = [lambda: fk.fk_layer_norm(x, v, v.clone(), y),\n"
        "  lambda: fk.fk_layer_norm_backward(x, x.clone(), v, m, m.clone(), y, None, None, ws),\n"
        "  lambda: fk.fk_linear(x, w, y, ws),\n"
        "  lambda: fk.fk_linear_backward(x, x.clone(), w, ws, dX=y),\n"
        "  lambda: fk.fk_balance_counts(i, c, r),\n"
        "  lambda: fk.fk_balance_loss(x, i, c, r, m[:1], y, ws)]\n"
        "for f in calls:\n"
        "    try:\n"
        "        f(); print(0)\n"
        "    except fk.FkError as e:\n"
        "        print(e.status)\n")
    out = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, FK_FAULT="launch"),
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr
    assert out.stdout.split() == ["4"] * 6


def test_loss_gradient_against_differences_through_the_head(fk):
    """The GPU's dH against central differences of the fp64 forward chain along random
    directions."""
    p, b, ws = head_setup(fk, 60, 24, 40, 12, seed=20)
    head_pass(fk, p, b, ws)
    counts, n = ref.balance_counts(b["lab"], 12)

    def loss(H):
        a = ref.layer_norm(H, p["g1"], p["b1"], 1e-5)[0]
        h = ref.linear(a, p["W1"], p["c1"], "gelu", None)[0]
        dd = ref.linear(h, p["W2"], p["c2"], "none", H)[0]
        pts = ref.layer_norm(dd, p["g2"], p["b2"], 1e-5)[0]
        S = ref.linear(pts, p["C"], p["half"], "none", None)[0]
        return ref.balance(S, b["lab"], counts, n, 0.1, 1.0)[0]

    H = p["H"].double()
    dH = b["dH"].double() + b["dD"].double()
    for seed in range(4):
        v = rnd((60, 24), torch.float32, 100 + seed).double()
        h = 1e-4
        num = float(loss(H + h * v) - loss(H - h * v)) / (2 * h)
        # the difference is off by h^2 of third derivatives (1e-8 of the scale), the gradient by
        # about 1e-5 of its norm a stage, seven stages
        assert math.isclose(num, float((dH * v).sum()), rel_tol=0,
                            abs_tol=2e-4 * float(dH.norm() * v.norm()) / 30 + 1e-9)
