"""The embedding-head operators (layer norm, linear, balance loss) refuse bad arguments on
the host before any device work (no GPU needed): C ABI and binding."""
import pytest
import torch

BIG = 1 << 30


@pytest.fixture(scope="module")
def fk():
    import __graft_entry__
    __graft_entry__.build()
    from exact_lloyd_means_b200 import fk as m
    return m


# Addresses a megabyte and more apart stand for buffers; nothing is launched on them.
def _at(i):
    return (i + 1) << 24


def _call(fn, order, defaults, **kw):
    a = dict(defaults, **kw)
    assert not set(kw) - set(defaults)
    return fn(*[a[k] for k in order])


def test_layer_norm_refusals(fk):
    order = "X dtype N d gamma beta eps Y mean rstd stream".split()
    ok = dict(X=_at(0), dtype=0, N=10, d=7, gamma=_at(1), beta=_at(2), eps=1e-5, Y=_at(3),
              mean=_at(4), rstd=_at(5), stream=None)

    def call(**kw):
        return _call(fk._lib.fk_layer_norm, order, ok, **kw)

    for bad in (dict(N=-1), dict(N=1 << 31), dict(d=0), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf")), dict(X=None), dict(Y=None), dict(Y=_at(0) + 4),
                dict(Y=_at(1)), dict(mean=_at(0)), dict(rstd=_at(4)), dict(mean=_at(3)),
                dict(N=(1 << 31) - 1, d=(1 << 31) - 1)):
        assert call(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(dtype=7), dict(X=_at(0) + 2), dict(Y=_at(3) + 1),
                dict(gamma=_at(1) + 2), dict(mean=_at(4) + 1), dict(dtype=1, X=_at(0) + 1)):
        assert call(**bad) == fk.FK_ERR_UNSUPPORTED, bad
    assert call(N=0, X=None, Y=None) == fk.FK_OK


def test_layer_norm_backward_refusals(fk):
    order = ("dY X dtype N d gamma mean rstd dX dgamma dbeta ws ws_bytes stream").split()
    ok = dict(dY=_at(0), X=_at(1), dtype=0, N=10, d=7, gamma=_at(2), mean=_at(3), rstd=_at(4),
              dX=_at(5), dgamma=_at(6), dbeta=_at(7), ws=_at(8), ws_bytes=BIG, stream=None)

    def call(**kw):
        return _call(fk._lib.fk_layer_norm_backward, order, ok, **kw)

    for bad in (dict(N=-1), dict(d=0), dict(dY=None), dict(X=None), dict(mean=None),
                dict(rstd=None), dict(dX=_at(1)), dict(dX=_at(0) + 4), dict(dgamma=_at(7)),
                dict(dbeta=_at(2)), dict(dgamma=_at(8) + 256), dict(ws=_at(0))):
        assert call(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(dX=_at(5) + 2), dict(dgamma=_at(6) + 1)):
        assert call(**bad) == fk.FK_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=_at(8) + 16), dict(ws_bytes=100)):
        assert call(**bad) == fk.FK_ERR_WORKSPACE, bad


def test_linear_refusals(fk):
    order = "X dtype N d W m bias act residual Y Z ws ws_bytes stream".split()
    ok = dict(X=_at(0), dtype=0, N=10, d=7, W=_at(1), m=5, bias=_at(2), act=0, residual=_at(3),
              Y=_at(4), Z=_at(5), ws=_at(6), ws_bytes=BIG, stream=None)

    def call(**kw):
        return _call(fk._lib.fk_linear, order, ok, **kw)

    for bad in (dict(N=-1), dict(N=1 << 31), dict(d=0), dict(m=0), dict(act=4), dict(act=-1),
                dict(X=None), dict(W=None), dict(Y=None), dict(Y=_at(0)), dict(Y=_at(1)),
                dict(Y=_at(3) + 4), dict(Z=_at(3)), dict(Z=_at(4)), dict(Y=_at(2)),
                dict(ws=_at(1)), dict(m=(1 << 31) - 1, d=(1 << 31) - 1)):
        assert call(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(X=_at(0) + 2), dict(bias=_at(2) + 2),
                dict(residual=_at(3) + 1), dict(Z=_at(5) + 1)):
        assert call(**bad) == fk.FK_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=_at(6) + 128), dict(ws_bytes=8)):
        assert call(**bad) == fk.FK_ERR_WORKSPACE, bad
    assert call(N=0, X=None, Y=None, residual=None) == fk.FK_OK


def test_linear_backward_refusals(fk):
    order = "dY X dtype N d W m act Z dX dW dbias ws ws_bytes stream".split()
    ok = dict(dY=_at(0), X=_at(1), dtype=0, N=10, d=7, W=_at(2), m=5, act=2, Z=_at(3),
              dX=_at(4), dW=_at(5), dbias=_at(6), ws=_at(7), ws_bytes=BIG, stream=None)

    def call(**kw):
        return _call(fk._lib.fk_linear_backward, order, ok, **kw)

    for bad in (dict(N=-1), dict(d=0), dict(m=0), dict(act=9), dict(dY=None), dict(X=None),
                dict(W=None), dict(Z=None), dict(dX=_at(0)), dict(dX=_at(1)), dict(dW=_at(2)),
                dict(dbias=_at(5)), dict(dX=_at(3)), dict(ws=_at(0))):
        assert call(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(dY=_at(0) + 2), dict(dbias=_at(6) + 2)):
        assert call(**bad) == fk.FK_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=_at(7) + 64), dict(ws_bytes=8)):
        assert call(**bad) == fk.FK_ERR_WORKSPACE, bad


def test_balance_refusals(fk):
    order = "labels N top K counts rows stream".split()
    ok = dict(labels=_at(0), N=10, top=2, K=5, counts=_at(1), rows=_at(2), stream=None)

    def counts(**kw):
        return _call(fk._lib.fk_balance_counts, order, ok, **kw)

    for bad in (dict(N=-1), dict(top=0), dict(K=0), dict(labels=None), dict(counts=None),
                dict(rows=None), dict(counts=_at(0)), dict(rows=_at(1) + 4),
                dict(N=1 << 30, top=2)):
        assert counts(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(labels=_at(0) + 2), dict(counts=_at(1) + 1), dict(rows=_at(2) + 2)):
        assert counts(**bad) == fk.FK_ERR_UNSUPPORTED, bad

    order2 = ("S dtype N K labels top counts rows scale coef loss dS ws ws_bytes stream").split()
    ok2 = dict(S=_at(0), dtype=0, N=10, K=5, labels=_at(1), top=2, counts=_at(2), rows=_at(3),
               scale=1.0, coef=1.0, loss=_at(4), dS=_at(5), ws=_at(6), ws_bytes=BIG,
               stream=None)

    def loss(**kw):
        return _call(fk._lib.fk_balance_loss, order2, ok2, **kw)

    nan, inf = float("nan"), float("inf")
    for bad in (dict(N=-1), dict(K=0), dict(top=0), dict(S=None), dict(labels=None),
                dict(counts=None), dict(rows=None), dict(loss=None), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=nan), dict(scale=inf), dict(scale=1e38),
                dict(coef=nan),
                dict(coef=inf), dict(dS=_at(0) + 4), dict(dS=_at(1)), dict(loss=_at(3)),
                dict(ws=_at(0)), dict(N=1 << 30, top=2)):
        assert loss(**bad) == fk.FK_ERR_INVALID_ARG, bad
    for bad in (dict(dtype=2), dict(S=_at(0) + 2), dict(dS=_at(5) + 1), dict(loss=_at(4) + 2)):
        assert loss(**bad) == fk.FK_ERR_UNSUPPORTED, bad
    for bad in (dict(ws=None), dict(ws=_at(6) + 8), dict(ws_bytes=8)):
        assert loss(**bad) == fk.FK_ERR_WORKSPACE, bad


def test_balance_refuses_gradients_past_fp32(fk):
    """coef scale K / n has to be a number, as padding rows multiply it by 0."""
    order = "S dtype N K labels top counts rows scale coef loss dS ws ws_bytes stream".split()
    ok = dict(S=_at(0), dtype=0, N=10, K=5, labels=_at(1), top=2, counts=_at(2), rows=_at(3),
              scale=1.0, coef=1.0, loss=_at(4), dS=_at(5), ws=_at(6), ws_bytes=BIG, stream=None)
    for bad in (dict(scale=1e37, coef=2.5), dict(scale=1e37, coef=-2.5), dict(coef=3e38),
                dict(scale=1e37, K=64), dict(scale=1e30, coef=1e30), dict(coef=-1e35, K=1 << 20)):
        assert _call(fk._lib.fk_balance_loss, order, ok, **bad) == fk.FK_ERR_INVALID_ARG, bad


def test_workspace_sizes(fk):
    for name, args in (("linear_workspace", (10, 7, 5)), ("linear_backward_workspace", (10, 7, 5)),
                       ("layer_norm_backward_workspace", (10, 7)),
                       ("balance_workspace", (10, 7))):
        fn = getattr(fk, name)
        for dtype in (torch.float32, torch.bfloat16):
            assert fn(*args, dtype, device="meta").numel() >= 256
            assert fn(0, *args[1:], dtype, device="meta").numel() >= 256
        with pytest.raises(TypeError):
            fn(*args, torch.float16, device="meta")
        with pytest.raises(fk.FkError) as e:
            fn(-1, *args[1:], torch.float32, device="meta")
        assert e.value.status == fk.FK_ERR_INVALID_ARG


def test_binding_rejects_wrong_tensors(fk):
    x, v, w = torch.zeros(4, 8), torch.zeros(8), torch.zeros(3, 8)
    ws = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError):
        fk.fk_layer_norm(x, v, v, x)  # CPU tensors
    with pytest.raises(ValueError):
        fk.fk_layer_norm(v, v, v, v)  # not a matrix
    with pytest.raises(TypeError):
        fk.fk_layer_norm(None, v, v, x)
    with pytest.raises(ValueError):
        fk.fk_linear(x, w, torch.zeros(4, 3), ws)
    with pytest.raises(ValueError):
        fk.fk_linear_backward(torch.zeros(4, 3), x, w, ws)
    with pytest.raises(ValueError):
        fk.fk_balance_counts(torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                             torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fk.fk_balance_loss(x, torch.zeros(4, dtype=torch.int32),
                           torch.zeros(8, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                           torch.zeros(1), None, ws)


def test_differences_agree_with_the_gradient_formulas():
    """The gradient formulas of the head, in fp64, against central differences of the forward
    formulas: what the GPU tests hold the kernels to."""
    import head_reference as ref
    g = torch.Generator().manual_seed(5)

    def rnd(*shape):
        return torch.randn(*shape, generator=g, dtype=torch.float64)

    def slope(f, x, i, h=1e-5):
        a, b = x.clone(), x.clone()
        a.view(-1)[i] += h
        b.view(-1)[i] -= h
        return float(f(a) - f(b)) / (2 * h)

    X, W, b, dY = rnd(5, 6), rnd(4, 6), rnd(4), rnd(5, 4)
    for act in ("none", "relu", "gelu", "silu"):
        dX, dW, db = ref.linear_backward(dY, X, W, act, ref.linear(X, W, b, act, None)[1])
        for grad, f, x in ((dX, lambda t: (ref.linear(t, W, b, act, None)[0] * dY).sum(), X),
                           (dW, lambda t: (ref.linear(X, t, b, act, None)[0] * dY).sum(), W),
                           (db, lambda t: (ref.linear(X, W, t, act, None)[0] * dY).sum(), b)):
            for i in range(x.numel()):
                assert abs(slope(f, x, i) - float(grad.view(-1)[i])) < 1e-7
    ga, be, dN = rnd(6), rnd(6), rnd(5, 6)
    y, mean, rstd = ref.layer_norm(X, ga, be, 1e-5)
    dX, dg, dbt = ref.layer_norm_backward(dN, X, ga, mean, rstd)
    for grad, f, x in ((dX, lambda t: (ref.layer_norm(t, ga, be, 1e-5)[0] * dN).sum(), X),
                       (dg, lambda t: (ref.layer_norm(X, t, be, 1e-5)[0] * dN).sum(), ga),
                       (dbt, lambda t: (ref.layer_norm(X, ga, t, 1e-5)[0] * dN).sum(), be)):
        for i in range(x.numel()):
            assert abs(slope(f, x, i) - float(grad.view(-1)[i])) < 1e-6
    S = rnd(5, 6)
    lab = torch.tensor([[0, 1], [-1, 3], [-1, -1], [2, 2], [5, 0]], dtype=torch.int32)
    counts, n = ref.balance_counts(lab, 6)
    assert counts.tolist() == [2, 1, 2, 1, 0, 1] and n == 4
    loss, dS = ref.balance(S, lab, counts, n, 0.7, 1.3)
    for i in range(S.numel()):
        assert abs(slope(lambda t: ref.balance(t, lab, counts, n, 0.7, 1.3)[0], S, i)
                   - float(dS.view(-1)[i])) < 1e-8
