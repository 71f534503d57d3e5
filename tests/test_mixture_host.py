"""What surrounds a mixture's products, on the CPU: pins of the plain implementation, and the
host-side refusals of the entry points (checked before anything touches a GPU)."""
import ctypes

import numpy as np
import pytest

import oracle.mixture as ox
import post_quantization_syrk_amd as kq

P = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host
ODD = ctypes.c_void_p(0x10001)
TWO = ctypes.c_void_p(0x10002)
INF = np.inf


def test_route_by_hand():
    """Two choices of four experts: ties to the lower index, closed experts, a padding row, a row with
    one open expert, a row without a softmax."""
    l = np.log([[1, 4, 2, 1], [3, 3, 3, 3], [1, 1, 1, 1], [1, 1, 1, 2], [1, 1, 1, 1]])
    l[2], l[3, :3], l[4, 1] = -INF, -INF, INF
    r = ox.route(l, 2, False)
    assert r["expert"].tolist() == [[1, 2], [0, 1], [-1, -1], [3, -1], [-1, -1]]
    assert np.allclose(r["weight"][:4], [[0.5, 0.25], [0.25, 0.25], [0, 0], [1, 0]]) and np.isnan(r["weight"][4]).all()
    assert r["counts"].tolist() == [1, 2, 1, 1, 5, 4] and r["offsets"].tolist() == [0, 1, 3, 4, 5]
    assert r["slot"].tolist() == [[1, 3], [0, 2], [-1, -1], [4, -1], [-1, -1]]
    assert r["index"].tolist() == [1, 0, 1, 0, 3, -1, -1, -1, -1, -1]
    assert np.isnan(r["loss"])
    r = ox.route(l[:4], 2, True)
    assert np.allclose(r["weight"], [[2 / 3, 1 / 3], [0.5, 0.5], [0, 0], [1, 0]])
    p = np.array([[1, 4, 2, 1], [2, 2, 2, 2], [0, 0, 0, 0], [0, 0, 0, 8]]) / 8
    assert r["loss"] == pytest.approx(4 * (np.array([1, 2, 1, 1]) / 5 * p.sum(0) / 3).sum())


def test_balance_loss_is_one_where_it_is_even():
    r = ox.route(np.zeros((8, 4)), 4, False)
    assert r["loss"] == pytest.approx(1.0)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_route_gradient_against_differences(normalize, masked):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((6, 9))
    if masked:
        l[1], l[2, :8], l[:, 4] = -INF, -INF, -INF
    r = ox.route(l, 3, normalize)
    dw, dloss = rng.standard_normal((6, 3)), 0.7
    g = ox.route_backward(r, dw, dloss, normalize)
    f = lambda x: ox.route_objective(x, r["expert"], r["counts"], dw, dloss, normalize)  # noqa: E731
    h = 1e-5
    for t, e in np.ndindex(*l.shape):
        if l[t, e] == -INF:
            assert g[t, e] == 0
            continue
        up, down = l.copy(), l.copy()
        up[t, e] += h
        down[t, e] -= h
        # a central difference is off by h^2 / 6 of a third derivative of order one, and by 2^-53 / h
        assert abs((f(up) - f(down)) / (2 * h) - g[t, e]) < 1e-9


def test_combine_gradients_against_differences():
    rng = np.random.default_rng(4)
    slot = np.array([[2, 0], [7, -1], [4, 1]])
    z, w, dy = rng.standard_normal((5, 3)), rng.standard_normal((3, 2)), rng.standard_normal((3, 3))
    dz, dw = ox.combine_backward(dy, z, slot, w)
    f = lambda z, w: float((ox.combine(z, slot, w) * dy).sum())  # noqa: E731
    assert np.isnan(dz[3]).all()
    for at in np.ndindex(3, 2):
        d = np.zeros((3, 2))
        d[at] = 1
        assert abs(f(z, w + d) - f(z, w) - dw[at]) < 1e-12      # linear in each
    for at in np.ndindex(5, 3):
        d = np.zeros((5, 3))
        d[at] = 1
        assert abs(f(z + d, w) - f(z, w) - np.nan_to_num(dz[at])) < 1e-12


def _route(**kw):
    a = dict(x=P, type=kq.KQ_F32, rows=8000, experts=4, ld=4, top=2, norm=0, w=P, e=P, s=P, i=P, o=P, c=P, loss=None,
             ws=P, bytes=1 << 20)
    a.update(kw)
    return kq.load_library().kq_route(*a.values(), None)


ROUTE = [(dict(x=None), kq.KQ_EINVAL), (dict(type=2), kq.KQ_EINVAL), (dict(x=TWO), kq.KQ_EINVAL), (dict(type=1, x=ODD), kq.KQ_EINVAL),
         (dict(norm=2), kq.KQ_EINVAL), (dict(experts=0, ld=0), kq.KQ_ESHAPE), (dict(experts=4097, ld=4097), kq.KQ_ESHAPE),
         (dict(top=0), kq.KQ_ESHAPE), (dict(top=5), kq.KQ_ESHAPE), (dict(top=17, experts=64, ld=64), kq.KQ_ESHAPE),
         (dict(rows=-1), kq.KQ_ESHAPE), (dict(rows=1 << 30), kq.KQ_ESHAPE), (dict(ld=3), kq.KQ_ESHAPE), (dict(w=None), kq.KQ_EINVAL),
         (dict(w=TWO), kq.KQ_EINVAL), (dict(e=None), kq.KQ_EINVAL), (dict(c=None), kq.KQ_EINVAL), (dict(c=TWO), kq.KQ_EINVAL)]


@pytest.mark.parametrize("kw,status", ROUTE + [
    (dict(s=None), kq.KQ_EINVAL), (dict(i=None), kq.KQ_EINVAL), (dict(o=None), kq.KQ_EINVAL), (dict(i=TWO), kq.KQ_EINVAL),
    (dict(loss=TWO), kq.KQ_EINVAL), (dict(ws=None), kq.KQ_EWORKSPACE), (dict(bytes=16), kq.KQ_EWORKSPACE),
    (dict(ws=ctypes.c_void_p(0x10008)), kq.KQ_EWORKSPACE)])
def test_route_refuses(kw, status):
    assert _route(**kw) == status
    assert kq.load_library().kq_last_error()


def _route_back(**kw):
    a = dict(x=P, type=kq.KQ_F32, rows=8, experts=4, ld=4, top=2, norm=0, w=P, e=P, c=P, dw=None, dl=None, g=P, ldd=4)
    a.update(kw)
    return kq.load_library().kq_route_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", ROUTE + [
    (dict(g=None), kq.KQ_EINVAL), (dict(g=TWO), kq.KQ_EINVAL), (dict(dw=TWO), kq.KQ_EINVAL),
    (dict(dl=TWO), kq.KQ_EINVAL), (dict(ldd=3), kq.KQ_ESHAPE), (dict(ldd=5), kq.KQ_EINVAL)])
def test_route_backward_refuses(kw, status):
    assert _route_back(**kw) == status


def test_route_workspace():
    assert kq.kq_route_workspace(0, 1, 1) == 0
    sizes = [kq.kq_route_workspace(r, 64, 2) for r in (1, 100, 10_000, 1 << 20, 1 << 29)]
    assert sizes == sorted(sizes) and 0 < sizes[2] and sizes[-1] < 1 << 25
    for experts in (1, 64, 256, 3000):      # what serves some rows serves fewer
        sizes = [kq.kq_route_workspace(r, experts, 1) for r in sorted({*range(1, 2000, 7), *range(2000, 300_000, 997), 131_072, 131_200})]
        assert sizes == sorted(sizes)
    for bad in ((-1, 4, 1), (4, 0, 1), (4, 4, 5), (1 << 30, 4, 2)):
        with pytest.raises(kq.KQError) as e:
            kq.kq_route_workspace(*bad)
        assert e.value.status == kq.KQ_ESHAPE
    assert kq.load_library().kq_route_workspace(1, 1, 1, None) == kq.KQ_EINVAL


def _combine(**kw):
    a = dict(z=P, zt=kq.KQ_BF16, slots=8, n=16, ldz=16, slot=P, w=None, rows=4, top=2, r=None, rt=0, ldr=0, y=P, yt=kq.KQ_F32, ldy=16)
    a.update(kw)
    return kq.load_library().kq_combine(*a.values(), None)


COMBINE = [(dict(z=None), kq.KQ_EINVAL), (dict(z=ODD), kq.KQ_EINVAL), (dict(zt=2), kq.KQ_EINVAL), (dict(slots=-1), kq.KQ_ESHAPE),
           (dict(slots=(1 << 30) + 1), kq.KQ_ESHAPE), (dict(n=0), kq.KQ_ESHAPE), (dict(n=(1 << 24) + 1), kq.KQ_ESHAPE),
           (dict(ldz=15), kq.KQ_ESHAPE), (dict(slot=None), kq.KQ_EINVAL), (dict(slot=TWO), kq.KQ_EINVAL), (dict(w=TWO), kq.KQ_EINVAL),
           (dict(rows=-1), kq.KQ_ESHAPE), (dict(top=0), kq.KQ_ESHAPE), (dict(top=65), kq.KQ_ESHAPE), (dict(rows=1 << 30, top=2), kq.KQ_ESHAPE)]


@pytest.mark.parametrize("kw,status", COMBINE + [
    (dict(y=None), kq.KQ_EINVAL), (dict(y=TWO), kq.KQ_EINVAL), (dict(yt=3), kq.KQ_EINVAL), (dict(ldy=15), kq.KQ_ESHAPE),
    (dict(r=P, rt=2, ldr=16), kq.KQ_EINVAL), (dict(r=P, ldr=15), kq.KQ_ESHAPE), (dict(r=TWO, ldr=16), kq.KQ_EINVAL),
    (dict(r=P, rt=1, ldr=16), kq.KQ_EINVAL), (dict(r=P, ldr=17), kq.KQ_EINVAL)])
def test_combine_refuses(kw, status):
    assert _combine(**kw) == status


def _combine_back(**kw):
    a = dict(dy=P, dyt=kq.KQ_F32, rows=4, n=16, lddy=16, z=P, zt=kq.KQ_BF16, slots=8, ldz=16, slot=P, w=None, top=2, dz=P, lddz=16, dw=P)
    a.update(kw)
    return kq.load_library().kq_combine_backward(*a.values(), None)


@pytest.mark.parametrize("kw,status", COMBINE + [
    (dict(dy=None), kq.KQ_EINVAL), (dict(dy=TWO), kq.KQ_EINVAL), (dict(dyt=2), kq.KQ_EINVAL), (dict(lddy=15), kq.KQ_ESHAPE),
    (dict(dz=ODD), kq.KQ_EINVAL), (dict(lddz=15), kq.KQ_ESHAPE), (dict(dw=TWO), kq.KQ_EINVAL), (dict(lddz=17), kq.KQ_EINVAL)])
def test_combine_backward_refuses(kw, status):
    assert _combine_back(**kw) == status


def test_nothing_to_do():
    assert _combine(rows=0, y=None, slot=None) == kq.KQ_OK
    assert _combine_back(rows=0, dy=None, slot=None) == kq.KQ_OK
    assert _combine_back(dz=None, dw=None, z=None) == kq.KQ_OK
    assert _route_back(rows=0, x=None, g=None) == kq.KQ_OK


def _product(experts=None, ep=None, **kw):
    a = dict(x=P, type=kq.KQ_BF16, rows=4, n=64, ldx=64, xs=None, d=None, sign=None, had=1, index=P, slots=4,
             offsets=P, wc=P, ws=P, out=16, y=P, ytype=kq.KQ_F32, ldy=16, work=P, bytes=4 * 68)
    a.update(kw)
    lib = kq.load_library()
    x = (a["x"], a["type"], a["rows"], a["n"], a["ldx"], a["xs"], a["d"], a["sign"], a["had"])
    e = dict(act=0, gated=0, bias=None, residual=None, residual_type=0, ldr=0)
    ep = None if ep is False else ctypes.byref(kq.Epilogue(*{**e, **(ep or {})}.values()))
    y = (a["wc"], a["ws"], a["out"], ep, a["y"], a["ytype"], a["ldy"], a["work"], a["bytes"], None)
    if experts is None:
        return lib.kq_mxfp4_linear_epilogue(*x, *y)
    return lib.kq_mxfp4_experts_epilogue(*x, a["index"], a["slots"], a["offsets"], experts, *y)


@pytest.mark.parametrize("experts", [None, 2])
@pytest.mark.parametrize("kw,status", [
    (dict(ep=False), kq.KQ_EINVAL), (dict(ep=dict(act=5)), kq.KQ_EINVAL), (dict(ep=dict(act=-1)), kq.KQ_EINVAL),
    (dict(ep=dict(gated=2)), kq.KQ_EINVAL), (dict(ep=dict(bias=TWO)), kq.KQ_EINVAL),
    (dict(ep=dict(residual=P, residual_type=2, ldr=16)), kq.KQ_EINVAL), (dict(ep=dict(residual=P, ldr=15)), kq.KQ_ESHAPE),
    (dict(ep=dict(residual=TWO, ldr=16)), kq.KQ_EINVAL), (dict(ep=dict(residual=ODD, residual_type=1, ldr=16)), kq.KQ_EINVAL),
    (dict(ep=dict(residual=P, residual_type=1, ldr=16)), kq.KQ_EINVAL), (dict(ep=dict(residual=P, ldr=17)), kq.KQ_EINVAL),
    (dict(ep=dict(gated=1), out=(1 << 23) + 1, ldy=1 << 24), kq.KQ_ESHAPE),
    (dict(ep=dict(gated=1), out=1 << 20, ldy=1 << 20, n=1 << 16, ldx=1 << 16, bytes=1 << 40), kq.KQ_ESHAPE),
    (dict(x=None), kq.KQ_EINVAL), (dict(wc=None), kq.KQ_EINVAL), (dict(y=None), kq.KQ_EINVAL), (dict(ldy=15), kq.KQ_ESHAPE),
    (dict(work=None), kq.KQ_EWORKSPACE), (dict(rows=-1), kq.KQ_ESHAPE),
])
def test_products_with_an_epilogue_refuse(kw, status, experts):
    assert _product(experts=experts, **kw) == status
    assert kq.load_library().kq_last_error()


def test_experts_epilogue_refuses():
    for kw, status in ((dict(experts=0), kq.KQ_ESHAPE), (dict(experts=4097), kq.KQ_ESHAPE), (dict(experts=2, slots=-1), kq.KQ_ESHAPE),
                       (dict(experts=2, offsets=None), kq.KQ_EINVAL), (dict(experts=2, index=None, slots=5), kq.KQ_ESHAPE)):
        assert _product(**kw) == status


def test_products_of_nothing():
    assert _product(rows=0, x=None, y=None, work=None, bytes=0) == kq.KQ_OK
    assert _product(experts=2, slots=0, y=None, ep=dict(gated=1, act=2)) == kq.KQ_OK


def test_the_binding_refuses_host_tensors():
    import torch
    f, i = torch.zeros(4, 4), torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: kq.kq_route(f, f, i, i, i, i, i), lambda: kq.kq_combine(f, i, f), lambda: kq.kq_combine_backward(f, f, i),
                 lambda: kq.kq_route_backward(f, f, f, i, i)):
        with pytest.raises((TypeError, RuntimeError)):
            call()
