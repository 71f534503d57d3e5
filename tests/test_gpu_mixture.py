"""GPU parity of what surrounds a mixture's products: routing with its balance loss and gradients,
products with an epilogue, the sum of the experts' rows and its gradients.

Choices, slots and counts are held to equality.  Bounds of the rest, with u = 2^-24 (half a step of
fp32) and half a step of bf16, 2^-8, where it is the type of the result:
  softmax       an exponent x - m rounds by u |x - m|, which is the relative error of the exponential;
                the exponential, the division and a sum of E terms add a few u and E u.  With D the
                largest |x - m| among logits above -inf: relative (2 D + E + 16) u
  loss          the softmax's, and a sum over a chunk's rows in fp32: (2 D + E + 16 + rows) u
  dlogits       terms p b, p sum p b, p w dw, w dw, each by the above, and sums of E or top terms
  products      (K + 2) u sum |x w| for the sum, then bias, activation (its slope is at most 1.13, its
                own error 10 u |v|), the gate's product and the residual, each rounded once
  combine       (top + 2) u (|r| + sum |w z|);  dweight (n + 2) u sum |dy z|;  dz one rounding
"""
import numpy as np
import pytest

import oracle.mixture as ox
import oracle.mxfp4 as om
from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_mxfp4 import (PATHS, _dev, _empty, _experts_ref, _forced, _layer, _processing, _random_codes, _rows, _sorted_slots,
                                  _values)

pytestmark = pytest.mark.gpu

U, INF = 2.0 ** -24, np.inf


def _kq():
    import post_quantization_syrk_amd as kq
    return kq


def _host(t):
    return t.double().cpu().numpy()


def _half(kind):
    return 2.0 ** -8 if kind == "bf16" else 2.0 ** -24


def _dtype(kind):
    torch = torch_cuda()
    return torch.bfloat16 if kind == "bf16" else torch.float32


def _within(got, want, bound, what=""):
    got, want = np.broadcast_arrays(np.asarray(got, np.float64), np.asarray(want, np.float64))
    fine = np.isfinite(want)
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    assert np.array_equal(got[~fine & ~np.isnan(want)], want[~fine & ~np.isnan(want)]), what
    over = np.abs(got - want)[fine] - np.broadcast_to(bound, want.shape)[fine]
    assert over.size == 0 or over.max() <= 0, (what, float(over.max()))


class Routes:
    """kq_route's outputs, filled with values that it must replace."""

    def __init__(self, rows, experts, top, train=True):
        torch = torch_cuda()
        full = lambda *s, v=77, k=torch.int32: torch.full(s, v, dtype=k, device="cuda")  # noqa: E731
        self.weight = full(rows, top, v=7.0, k=torch.float32)
        self.expert, self.slot, self.index = full(rows, top), full(rows, top), full(rows * top)
        self.offsets, self.counts = full(experts + 1), full(experts + 2)
        self.loss = full(1, v=7.0, k=torch.float32) if train else None

    def dict(self):
        return dict(self.__dict__)


def _logits(rng, rows, experts, kind, masked):
    x = 2 * rng.standard_normal((rows, experts)) + rng.standard_normal(experts)
    if masked:
        x[rng.random((rows, experts)) < 0.3] = -INF
        x[rng.random(rows) < 0.1] = -INF
        only = rng.random(rows) < 0.1
        x[only] = np.where(np.arange(experts) == rng.integers(experts), 0.5, -INF)
        x[rng.random(rows) < 0.1] = 1.25                      # all equal
        low = rng.random(rows) < 0.1
        x[low] = np.where(rng.random((int(low.sum()), experts)) < 0.5, -3.3e38, x[low])   # near the lowest value
    torch = torch_cuda()
    return torch.from_numpy(x).to(_dtype(kind))


def _route_check(r, x, top, normalize, want=None):
    """r's outputs against the oracle's for host logits x; returns the oracle's."""
    x = _host(x)
    rows, experts = x.shape
    want = want or ox.route(x, top, normalize)
    for k in ("expert", "slot", "index", "offsets", "counts"):
        assert np.array_equal(getattr(r, k).cpu().numpy(), want[k]), k
    with np.errstate(invalid="ignore"):
        d = np.where(x > -INF, np.max(x, 1, initial=-INF, keepdims=True) - x, 0)
    d = np.where(np.isfinite(d), np.minimum(d, 104.0), 0)    # (beyond it the exponential is zero in fp32)
    rel = (2 * d.max(initial=0) + experts + 16) * U
    _within(_host(r.weight), want["weight"], rel * np.abs(np.nan_to_num(want["weight"])) + 2.0 ** -126, "weight")
    if r.loss is not None:
        _within(_host(r.loss)[0], want["loss"], (rel + rows * U) * abs(want["loss"]), "loss")
    return want


ROUTES = [(1, 1, 1), (1, 8, 2), (2, 64, 6), (3, 5, 5), (5, 15, 2), (7, 16, 16), (33, 17, 4), (64, 32, 1), (65, 33, 3), (200, 60, 4),
          (130, 64, 8), (100, 100, 2), (77, 128, 8), (500, 256, 8), (37, 300, 6), (20, 512, 10), (9, 1000, 16), (6, 2048, 3), (5, 4096, 16),
          (5000, 8, 2), (2049, 64, 6), (4100, 3, 3), (150, 300, 6), (700, 256, 16), (1500, 250, 8),
          (300, 2000, 4), (129, 1, 1), (128, 64, 6), (1100, 1024, 9)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("rows,experts,top", ROUTES)
def test_route(rows, experts, top, masked, kind):
    announce(f"route {rows}x{experts} top {top} {kind} masked {masked}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows * 31 + experts)
    x = _logits(rng, rows, experts, kind, masked)
    normalize = bool((rows + top) % 2)
    r = Routes(rows, experts, top)
    kq.kq_route(x.cuda(), normalize=normalize, **r.dict())
    want = _route_check(r, x, top, normalize)
    again = Routes(rows, experts, top, train=False)
    kq.kq_route(x.cuda(), normalize=normalize, **again.dict())
    for k, v in again.dict().items():
        assert v is None or torch.equal(v, getattr(r, k)), k
    # the gradient
    dw, dloss = rng.standard_normal((rows, top)).astype(np.float32), np.float32(rows * 0.3)
    g = torch.full((rows, experts), 7.0, dtype=x.dtype, device="cuda")
    kq.kq_route_backward(x.cuda(), g, r.weight, r.expert, r.counts, dweight=_dev(dw), dloss=_dev(dloss.reshape(1)), normalize=normalize)
    _route_back_check(g, x, want, dw, dloss, normalize, kind)


def _route_back_check(g, x, want, dw, dloss, normalize, kind):
    x, p = _host(x), want["p"]
    rows, experts = x.shape
    top = dw.shape[1]
    ref = ox.route_backward(want, dw, dloss, normalize)
    made, used = max(want["counts"][experts], 1), max(want["counts"][experts + 1], 1)
    b = abs(float(dloss)) * experts * want["counts"][:experts] / (made * used)
    with np.errstate(invalid="ignore"):
        d = np.where(x > -INF, np.max(x, 1, initial=-INF, keepdims=True) - x, 0)
    d = np.where(np.isfinite(d), np.minimum(d, 104.0), 0).max(initial=0)
    c = (4 * d + 2 * experts + 2 * top + 64) * U
    chosen = want["expert"] >= 0
    wg = np.where(chosen, np.abs(np.nan_to_num(want["weight"]) * dw), 0)
    size = p * (b + (p * b).sum(1, keepdims=True) + wg.sum(1, keepdims=True))
    for j in range(top):
        t = np.nonzero(chosen[:, j])[0]
        size[t, want["expert"][t, j]] += wg[t, j] + np.abs(want["weight"][t, j]) * wg[t].sum(1)
    _within(_host(g), ref, c * size + _half(kind) * np.abs(ref) + 2.0 ** -126, "dlogits")


@pytest.mark.parametrize("top", [1, 4, 8, 9, 15, 16])
@pytest.mark.parametrize("experts", [16, 30, 64, 200, 256, 520, 1000])
def test_route_of_close_logits(experts, top):
    """Logits a few units in the last place apart, of either sign, zeros of both signs, numbers below the
    normal ones, the lowest number beside closed experts: the order is that of the whole values."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(experts + top)
    rows = 40
    bits = np.float32(1.75).view(np.int32) + rng.integers(0, 40, (rows, experts)).astype(np.int32)
    x = bits.view(np.float32).copy()
    x[1::2] *= -1
    x[4] = np.where(rng.random(experts) < 0.5, 0.0, -0.0)
    x[5] = rng.integers(-3, 4, experts) * np.float32(2.0 ** -149)
    x[6, ::2] = x[6, ::2] * 3
    x[7] = np.where(rng.random(experts) < 0.7, -INF, np.finfo(np.float32).min)
    x[8] = np.where(rng.random(experts) < 0.7, np.nextafter(np.finfo(np.float32).min, np.float32(0)), np.finfo(np.float32).min)
    x[9] = rng.standard_normal(experts)
    x[10, 1:] = -INF
    x[11] = np.where(rng.random(experts) < 0.5, 3e38, np.nextafter(np.float32(3e38), np.float32(INF)))
    x[12:20] = np.round(rng.standard_normal((8, experts)) * 2) / 2
    r = Routes(rows, experts, top)
    kq.kq_route(_dev(x), normalize=True, **r.dict())
    _route_check(r, torch.from_numpy(x), top, True)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [8, 60, 256, 700])
def test_route_of_rows_without_a_softmax(experts, kind):
    """NaN and +inf take their own row only; the loss is NaN."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(experts)
    x = _logits(rng, 40, experts, kind, False)
    x[3, 5], x[11, 0], x[12, 7], x[20], x[39, experts - 1] = np.nan, INF, -INF, np.nan, np.nan
    x[13] = -INF
    r = Routes(40, experts, 4)
    kq.kq_route(x.cuda(), **r.dict())
    want = _route_check(r, x, 4, False)
    assert np.isnan(want["loss"]) and (want["expert"][3] == -1).all()
    g = torch.full((40, experts), 7.0, dtype=x.dtype, device="cuda")
    kq.kq_route_backward(x.cuda(), g, r.weight, r.expert, r.counts, dweight=torch.ones(40, 4, device="cuda"))
    bad = torch.isnan(g).all(1).cpu()
    assert bad.nonzero()[:, 0].tolist() == [3, 11, 20, 39] and not torch.isnan(g[~bad.cuda()]).any()
    assert not g[13].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 2), (3, 4), (4, 4), (8, 8)])
@pytest.mark.parametrize("experts", [4, 30, 64, 250, 520])
def test_route_strided(experts, off, pad, kind):
    """Logits and their gradient inside wider buffers, at any element: nothing around them is written."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(off)
    x = _logits(rng, 50, experts, kind, True)
    wide = torch.full((52, off + experts + pad), 9.0, dtype=x.dtype, device="cuda")
    wide[1:-1, off:off + experts] = x.cuda()
    r, flat = Routes(50, experts, 3), Routes(50, experts, 3)
    kq.kq_route(wide[1:-1, off:off + experts], **r.dict())
    kq.kq_route(x.cuda(), **flat.dict())
    for k, v in r.dict().items():
        assert torch.equal(v, getattr(flat, k)), k
    dw, dl = _dev(rng.standard_normal((50, 3)).astype(np.float32)), torch.full((1,), 0.5, device="cuda")
    g = torch.empty_like(x, device="cuda")
    kq.kq_route_backward(x.cuda(), g, r.weight, r.expert, r.counts, dweight=dw, dloss=dl)
    to = torch.full_like(wide, 5.0)
    kq.kq_route_backward(wide[1:-1, off:off + experts], to[1:-1, off:off + experts], r.weight, r.expert, r.counts, dweight=dw, dloss=dl)
    assert torch.equal(to[1:-1, off:off + experts], g)
    to[1:-1, off:off + experts] = 5.0
    assert torch.equal(to, torch.full_like(wide, 5.0))
    # in place
    same = wide[1:-1, off:off + experts]
    kq.kq_route_backward(same, same, r.weight, r.expert, r.counts, dweight=dw, dloss=dl)
    assert torch.equal(same, g)


@pytest.mark.parametrize("normalize", [False, True])
def test_route_gradient_parts(normalize):
    """Without the weights' gradient, without the loss's, without either."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(8)
    x = _logits(rng, 300, 40, "f32", True)
    r = Routes(300, 40, 4)
    kq.kq_route(x.cuda(), normalize=normalize, **r.dict())
    want = _route_check(r, x, 4, normalize)
    dw, dl = rng.standard_normal((300, 4)).astype(np.float32), np.float32(11.0)
    for a, b in ((dw, None), (None, dl), (None, None)):
        g = torch.full((300, 40), 7.0, device="cuda")
        kq.kq_route_backward(x.cuda(), g, r.weight, r.expert, r.counts, dweight=_dev(a), normalize=normalize,
                             dloss=None if b is None else _dev(b.reshape(1)))
        _route_back_check(g, x, want, np.zeros_like(dw) if a is None else a, 0.0 if b is None else b, normalize, "f32")


def test_route_gradient_against_differences():
    """The library's gradient against differences of the objective in 64 bits."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(9)
    for normalize in (False, True):
        x = rng.standard_normal((5, 7)).astype(np.float32)
        r = Routes(5, 7, 3)
        kq.kq_route(_dev(x), normalize=normalize, **r.dict())
        dw, dl = rng.standard_normal((5, 3)).astype(np.float32), np.float32(3.0)
        g = torch.empty(5, 7, device="cuda")
        kq.kq_route_backward(_dev(x), g, r.weight, r.expert, r.counts, dweight=_dev(dw), dloss=_dev(dl.reshape(1)), normalize=normalize)
        f = lambda v: ox.route_objective(v, r.expert.cpu().numpy(), r.counts.cpu().numpy(), dw, dl, normalize)  # noqa: E731
        for at in np.ndindex(5, 7):
            h = np.zeros((5, 7))
            h[at] = 1e-5
            # the difference is off by 1e-9, the gradient by its fp32 roundings of terms of order ten
            assert abs((f(x + h) - f(x - h)) / 2e-5 - float(g[at])) < 1e-9 + 10 * 100 * U


def test_route_of_no_rows():
    torch = torch_cuda()
    kq = _kq()
    r = Routes(0, 6, 2)
    kq.kq_route(torch.empty(0, 6, device="cuda"), **r.dict())
    assert not r.offsets.any() and not r.counts.any() and float(r.loss) == 0
    r = Routes(3, 6, 2)
    kq.kq_route(torch.full((3, 6), -INF, device="cuda"), **r.dict())
    assert not r.offsets.any() and not r.counts.any() and float(r.loss) == 0 and (r.index == -1).all() and not r.weight.any()


@pytest.mark.parametrize("rows,experts,top", [(131072, 256, 8), (100_003, 60, 4), (300_000, 8, 2), (40_000, 4096, 2)])
def test_route_of_many_rows(rows, experts, top):
    """Against torch on the device: sorts and sums of integers are exact there."""
    announce(f"route {rows}x{experts}")
    torch = torch_cuda()
    kq = _kq()
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, experts, generator=gen, device="cuda").to(torch.bfloat16)      # many equal logits
    x[torch.rand(rows, generator=gen, device="cuda") < 0.05] = -INF
    r = Routes(rows, experts, top)
    kq.kq_route(x, normalize=True, **r.dict())
    value, expert = x.float().sort(dim=1, descending=True, stable=True)
    flat = torch.where(value > -INF, expert, -1)[:, :top].reshape(-1)
    assert torch.equal(r.expert.view(-1), flat.int())
    order = torch.argsort(torch.where(flat < 0, experts, flat), stable=True)
    made = int((flat >= 0).sum())
    assert int(r.counts[experts]) == made and torch.equal(r.index[:made], (order[:made] // top).int()) and (r.index[made:] == -1).all()
    assert torch.equal(r.slot.view(-1)[order[:made]], torch.arange(made, device="cuda", dtype=torch.int32))
    counts = torch.bincount(flat[flat >= 0], minlength=experts)
    assert torch.equal(r.counts[:experts], counts.int()) and torch.equal(r.offsets[1:].long(), counts.cumsum(0))
    p = torch.nan_to_num(torch.softmax(x.double(), 1))
    used = int((x[:, 0] > -INF).sum())
    loss = float(experts * (counts / made * p.sum(0) / used).sum())
    assert int(r.counts[experts + 1]) == used and abs(float(r.loss) - loss) <= (24 + experts + 16 + 1024) * U * loss


# ---- products with an epilogue ----

ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def _finish(s, err, bias, act, gated, residual, kind):
    """(values, bound) of the epilogue on sums s known to err."""
    out = s.shape[1] // 2 if gated else s.shape[1]
    if bias is not None:
        s = s + bias
        err = err + U * np.abs(s)
    half = ox.activation(s[:, :out], act)
    herr = err[:, :out] if act in ("none",) else 1.13 * err[:, :out] + 10 * U * np.abs(s[:, :out])
    if gated:
        other, oerr = s[:, out:], err[:, out:]
        v = half * other
        err = np.abs(half) * oerr + np.abs(other) * herr + herr * oerr + U * np.abs(v)
    else:
        v, err = half, herr
    if residual is not None:
        v = v + residual
        err = err + U * np.abs(v)
    return v, err * (1 + _half(kind)) + _half(kind) * np.abs(v)


def _residual(rng, rows, out, kind):
    torch = torch_cuda()
    return None if kind is None else torch.from_numpy(rng.standard_normal((rows, out))).to(_dtype(kind))


EPILOGUES = [("none", False, True, None), ("silu", True, False, None), ("gelu", False, True, "f32"), ("gelu_tanh", True, True, "bf16"),
             ("relu", True, False, "f32"), ("none", True, True, None), ("none", False, False, "bf16")]


@pytest.mark.parametrize("act,gated,biased,rk", EPILOGUES, ids=str)
@pytest.mark.parametrize("rows,n,out,had,xk,yk", [
    (1, 128, 1, 128, "bf16", "f32"), (1, 4096, 1030, 4096, "bf16", "bf16"), (2, 33, 17, 1, "f32", "f32"), (3, 1000, 515, 8, "bf16", "f32"),
    (16, 2048, 300, 2048, "bf16", "f32"), (33, 256, 31, 256, "f32", "bf16"), (64, 1024, 96, 1024, "bf16", "f32"), (70, 192, 1000, 64, "bf16", "bf16"),
    (150, 384, 515, 128, "bf16", "f32"), (257, 512, 700, 512, "f32", "bf16"), (513, 320, 1027, 64, "bf16", "bf16"), (900, 256, 1300, 256, "bf16", "f32"),
])
def test_linear_epilogue(rows, n, out, had, xk, yk, act, gated, biased, rk):
    announce(f"linear epilogue {rows}x{n} -> {out} {act} gated {gated} bias {biased} residual {rk}")
    _linear_case(rows, n, out, had, xk, yk, act, gated, biased, rk)


def _linear_case(rows, n, out, had, xk, yk, act, gated, biased, rk):
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows + 3 * n + 5 * out)
    x = _rows(rng, rows, n, xk)
    d, sg = _processing(rng, n, had > 1, had > 1)
    wide = out * (1 + gated)
    wc, ws, wv = _layer(rng, wide, n)
    bias = rng.standard_normal(wide).astype(np.float32) if biased else None
    res = _residual(rng, rows, out, rk)
    y = _empty((rows, out), yk)
    rest = dict(d=_dev(d), sign=_dev(sg), had=had, bias=_dev(bias), act=act, gated=gated)
    kq.kq_mxfp4_linear_epilogue(x.cuda(), wc, ws, y, residual=None if res is None else res.cuda(), **rest)
    xq = om.mx_round(om.mx_rotate_f32(x.float().numpy(), d, sg, had))
    want, bound = _finish(xq @ wv.T, (n + 2) * U * (np.abs(xq) @ np.abs(wv.T)), bias, act, gated, None if res is None else _host(res), yk)
    _within(_host(y), want, bound)
    # rows quantised beforehand give the same bits; so does a residual in y itself
    xc, xs = kq.kq_mxfp4_empty(rows, n)
    kq.kq_mxfp4_quantize(x.cuda(), xc, xs, d=rest.pop("d"), sign=rest.pop("sign"), had=rest.pop("had"))
    again = _empty((rows, out), yk)
    if rk == yk:
        again.copy_(res)
    kq.kq_mxfp4_linear_epilogue(xc, wc, ws, again, x_scales=xs, n=n, residual=again if rk == yk else None if res is None else res.cuda(), **rest)
    assert torch.equal(y, again)


@pytest.mark.parametrize("path", PATHS, ids=str)
@pytest.mark.parametrize("act,gated,biased,rk", EPILOGUES, ids=str)
def test_epilogue_on_every_path(act, gated, biased, rk, path):
    """Each implementation, for a layer and for experts with empty and ragged ones."""
    announce(f"epilogue {act} {gated} {biased} {rk} {path}")
    torch = torch_cuda()
    kq = _kq()
    with _forced(path):
        for rows, n, out, had in ((1, 1000, 130, 8), (13, 640, 65, 128), (150, 256, 300, 256), (520, 1152, 262, 128)):
            _linear_case(rows, n, out, had, "bf16", "f32" if out % 2 else "bf16", act, gated, biased, rk)
            rng = np.random.default_rng(rows)
            x = _rows(rng, rows, n, "f32")
            wide = 72 * (1 + gated)
            ec, es, ev = _layer(rng, wide, n, 5)
            bias = rng.standard_normal((5, wide)).astype(np.float32) if biased else None
            index, offsets = _sorted_slots(rng, rows, 2, 5, 1.0)
            offsets[3] = offsets[2]                                      # an expert's slots go to the next one
            res = _residual(rng, 2 * rows, 72, rk)
            for kind in ("f32", "bf16"):
                y = _empty((2 * rows, 72), kind)
                kq.kq_mxfp4_experts_epilogue(x.cuda(), _dev(index), _dev(offsets), ec, es, y, bias=_dev(bias), act=act, gated=gated,
                                             residual=None if res is None else res.cuda())
                xq = om.mx_round(x.double().numpy())
                s, mag = _experts_ref(xq, index, offsets, ev, 2 * rows, rows)
                per = None if bias is None else bias[np.searchsorted(offsets, np.arange(2 * rows), side="right") - 1]
                want, bound = _finish(s, (n + 2) * U * mag, per, act, gated, None if res is None else _host(res), kind)
                _within(_host(y), want, bound)


@pytest.mark.parametrize("rows", [1, 40, 150, 700])
@pytest.mark.parametrize("gated", [False, True])
def test_epilogue_strided(rows, gated):
    """Outputs and residuals inside wider buffers, at any element: nothing around them is written."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    x = _rows(rng, rows, 256, "bf16").cuda()
    wc, ws, _ = _layer(rng, 200 * (1 + gated), 256)
    for yk in ("bf16", "f32"):
        for rk in ("bf16", "f32"):
            res = _residual(rng, rows, 200, rk).cuda()
            want = _empty((rows, 200), yk)
            kq.kq_mxfp4_linear_epilogue(x, wc, ws, want, residual=res, gated=gated, act="silu")
            for off, pad in ((1, 2), (2, 0), (4, 4), (3, (1 << 20) if rows < 50 else 1)):      # (the last: rows far apart)
                wide, from_ = _empty((rows + 2, off + 200 + pad), yk), _empty((rows + 2, 200 + off), rk)
                from_[1:-1, off:] = res
                kq.kq_mxfp4_linear_epilogue(x, wc, ws, wide[1:-1, off:off + 200], residual=from_[1:-1, off:], gated=gated, act="silu")
                assert torch.equal(wide[1:-1, off:off + 200], want)
                wide[1:-1, off:off + 200] = 123.0
                assert bool((wide == 123.0).all())


def test_epilogue_without_anything_is_the_product():
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(2)
    for rows in (1, 30, 300):
        x = _rows(rng, rows, 512, "bf16").cuda()
        wc, ws, _ = _layer(rng, 130, 512)
        a, b, c = (_empty((rows, 130), "f32") for _ in range(3))
        kq.kq_mxfp4_linear(x, wc, ws, a)
        kq.kq_mxfp4_linear_epilogue(x, wc, ws, b)
        kq.kq_mxfp4_linear_epilogue(x, wc, ws, c, bias=torch.zeros(130, device="cuda"))
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("rows", [1, 20, 130, 600])
def test_epilogue_keeps_what_is_not_finite_in_its_place(rows):
    """NaN weights, an infinite bias and a NaN residual; saturated activations."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    x = _rows(rng, rows, 128, "bf16").cuda()
    wc, ws, _ = _layer(rng, 100, 128)
    ws[0, 60, 1] = 255                                   # column 10 of the other half
    bias, res = torch.zeros(100, device="cuda"), torch.zeros(rows, 50, device="cuda")
    bias[7], bias[8], bias[9], res[rows - 1, 3] = INF, -1e30, 1e30, np.nan
    y = _empty((rows, 50), "f32")
    kq.kq_mxfp4_linear_epilogue(x, wc, ws, y, bias=bias, act="silu", gated=True, residual=res)
    bad = torch.zeros(rows, 50, dtype=torch.bool, device="cuda")
    bad[:, 10] = True
    bad[rows - 1, 3] = True
    # the other half's sums, which may be zero: infinity times that is NaN
    both = _empty((rows, 100), "f32")
    kq.kq_mxfp4_linear(x, wc, ws, both)
    other = both[:, 50:]
    bad[:, 7] |= other[:, 7] == 0
    assert torch.equal(torch.isnan(y), bad)
    # the sums vanish beside 1e30, whose sigmoid is 1 and that of -1e30 0
    assert bool((y[:, 7].abs() == INF)[~bad[:, 7]].all()) and not y[:, 8].any()
    assert torch.equal(y[:, 9], torch.full_like(other[:, 9], 1e30) * other[:, 9])


def test_epilogue_of_rows_past_32_bits():
    """Quantised rows of more than 4 GiB, read through an index: the bits of the same rows side by side."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(11)
    rows, n, out, slots = 1_060_000, 8192, 70, 300
    codes, scales = _random_codes(rows, n)
    index = rng.integers(0, rows, slots).astype(np.int32)
    index[[0, 1, slots - 1]] = [rows - 1, 0, rows - 2]
    offsets = np.int32([0, 3, slots])
    picked = torch.from_numpy(index).long().cuda()
    xq = _values(codes, scales, index)
    for act, gated, biased, rk in (("silu", True, True, "f32"), ("gelu", False, True, "bf16")):
        wide = out * (1 + gated)
        wc, ws, wv = _layer(rng, wide, n, 2)
        bias, res = rng.standard_normal((2, wide)).astype(np.float32), _residual(rng, slots, out, rk)
        rest = dict(bias=_dev(bias), act=act, gated=gated, residual=res.cuda(), n=n)
        y, near = _empty((slots, out), "f32"), _empty((slots, out), "f32")
        kq.kq_mxfp4_experts_epilogue(codes, _dev(index), _dev(offsets), wc, ws, y, x_scales=scales, **rest)
        with _forced(dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=256)):
            kq.kq_mxfp4_experts_epilogue(codes[picked], None, _dev(offsets), wc, ws, near, x_scales=scales[:, picked].contiguous(), **rest)
        assert torch.equal(y, near)
        s, mag = _experts_ref(xq, None, offsets, wv, slots, slots)
        per = bias[np.searchsorted(offsets, np.arange(slots), side="right") - 1]
        want, bound = _finish(s, (n + 2) * U * mag, per, act, gated, _host(res), "f32")
        _within(_host(y), want, bound)


def test_epilogue_of_an_output_past_32_bits():
    """More than 4 GiB of output, which is its own residual."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(12)
    rows, n, out = 1_000_003, 128, 2200
    codes, scales = _random_codes(rows, n)
    wc, ws, wv = _layer(rng, out, n)
    bias = rng.standard_normal(out).astype(np.float32)
    y = torch.empty((rows, out), dtype=torch.bfloat16, device="cuda")
    y.copy_((torch.arange(rows, device="cuda") % 251)[:, None].expand(rows, out))
    kq.kq_mxfp4_linear_epilogue(codes, wc, ws, y, x_scales=scales, n=n, bias=_dev(bias), act="gelu_tanh", residual=y)
    some = np.concatenate([[0, 1, rows - 1, rows - 2, rows - 3], rng.integers(0, rows, 200)])
    xq = _values(codes, scales, some)
    want, bound = _finish(xq @ wv.T, (n + 2) * U * (np.abs(xq) @ np.abs(wv.T)), bias, "gelu_tanh", False, (some % 251)[:, None], "bf16")
    _within(_host(y[torch.from_numpy(some).cuda()]), want, bound)


@pytest.mark.parametrize("slots", [40, 600])
def test_epilogue_of_layers_past_32_bits(slots):
    """Gated layers that lie more than 4 GiB behind the first, from the sums of the call without an epilogue."""
    torch = torch_cuda()
    kq = _kq()
    n, out, experts = 8192, 2048, 260
    wc, ws = _random_codes(2 * out, n, experts)
    x, xs = _random_codes(slots, n)
    offsets = np.zeros(experts + 1, np.int32)
    offsets[2:] = slots // 2
    offsets[-1] = slots
    sums, y = _empty((slots, 2 * out), "f32"), _empty((slots, out), "f32")
    kq.kq_mxfp4_experts(x, None, _dev(offsets), wc, ws, sums, x_scales=xs, n=n)
    kq.kq_mxfp4_experts_epilogue(x, None, _dev(offsets), wc, ws, y, x_scales=xs, n=n, act="relu", gated=True)
    assert torch.equal(y, torch.relu(sums[:, :out]) * sums[:, out:])


# ---- the experts' rows together ----

def _choices(rng, rows, top, slots, dropped):
    """Distinct slots in any order, some choices without one, some far outside."""
    place = rng.permutation(max(slots, rows * top))[:rows * top].reshape(rows, top).astype(np.int32)
    if dropped:
        place[rng.random((rows, top)) < 0.2] = -1
        place[rng.random((rows, top)) < 0.05] = 2 ** 31 - 1
    return place                                         # (from `slots` on: outside)


COMBINES = [(1, 1, 1, 1), (1, 4096, 2, 2), (3, 7, 2, 5), (2, 16384, 3, 6), (50, 8, 4, 200), (33, 9, 1, 40), (17, 1000, 6, 102), (9, 2049, 8, 60),
            (64, 512, 2, 100), (5, 11008, 2, 10), (4, 100, 64, 256), (700, 130, 9, 7000), (300, 2048, 6, 1800), (1000, 64, 2, 2000)]


@pytest.mark.parametrize("zk,yk,rk", [("bf16", "bf16", "bf16"), ("f32", "f32", None), ("bf16", "f32", "f32"), ("f32", "bf16", "bf16"), ("bf16", "bf16", None)])
@pytest.mark.parametrize("rows,n,top,slots", COMBINES)
def test_combine(rows, n, top, slots, zk, yk, rk):
    announce(f"combine {rows}x{n} top {top} of {slots} {zk} {yk} {rk}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows + n + top)
    z = torch.from_numpy(rng.standard_normal((slots, n))).to(_dtype(zk))
    slot = _choices(rng, rows, top, slots, dropped=rows > 2)
    w = rng.standard_normal((rows, top)).astype(np.float32) if n % 3 else None
    res = _residual(rng, rows, n, rk)
    y = _empty((rows, n), yk)
    kq.kq_combine(z.cuda(), _dev(slot), y, weight=_dev(w), residual=None if res is None else res.cuda())
    zh, rh = _host(z), None if res is None else _host(res)
    want = ox.combine(zh, slot, w, rh)
    mag = ox.combine(np.abs(zh), slot, None if w is None else np.abs(w), None if rh is None else np.abs(rh))
    _within(_host(y), want, (top + 2) * U * mag * (1 + _half(yk)) + _half(yk) * np.abs(want), "y")
    if rk == yk:
        again = res.cuda()
        kq.kq_combine(z.cuda(), _dev(slot), again, weight=_dev(w), residual=again)
        assert torch.equal(again, y)
    # gradients
    dy = torch.from_numpy(rng.standard_normal((rows, n))).to(_dtype(yk))
    dz, dw = _empty((slots, n), zk), torch.full((rows, top), 123.0, device="cuda")
    kq.kq_combine_backward(dy.cuda(), z.cuda(), _dev(slot), dz, weight=_dev(w), dweight=dw)
    rz, rw = ox.combine_backward(_host(dy), zh, slot, w)
    _, mw = ox.combine_backward(np.abs(_host(dy)), np.abs(zh), slot)
    _within(_host(dw), rw, (n + 2) * U * mw, "dweight")
    named = ~np.isnan(rz)
    got = _host(dz)
    assert (got[~named] == 123.0).all()
    _within(got[named], rz[named], (U * (1 + _half(zk)) + _half(zk)) * np.abs(rz[named]), "dz")
    one, only = _empty((slots, n), zk), torch.full((rows, top), 123.0, device="cuda")
    kq.kq_combine_backward(dy.cuda(), z.cuda(), _dev(slot), one, weight=_dev(w))
    kq.kq_combine_backward(dy.cuda(), z.cuda(), _dev(slot), weight=_dev(w), dweight=only)
    assert torch.equal(one, dz) and torch.equal(only, dw)
    same = z.cuda()
    kq.kq_combine_backward(dy.cuda(), same, _dev(slot), same, weight=_dev(w), dweight=only)
    assert torch.equal(only, dw) and torch.equal(same.cpu()[torch.from_numpy(named)], dz.cpu()[torch.from_numpy(named)])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("off,pad", [(1, 2), (2, 1), (4, 4), (8, 8), (3, 0)])
@pytest.mark.parametrize("n", [1, 61, 512, 3001])
def test_combine_strided(n, off, pad, kind):
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(n + off)
    wide = lambda rows, v: torch.full((rows + 2, off + n + pad), v, dtype=_dtype(kind), device="cuda")  # noqa: E731
    inner = lambda t: t[1:-1, off:off + n]  # noqa: E731
    z, dy, res = (torch.from_numpy(rng.standard_normal((r, n))).to(_dtype(kind)).cuda() for r in (40, 15, 15))
    slot, w = _dev(_choices(rng, 15, 3, 40, True)), _dev(rng.standard_normal((15, 3)).astype(np.float32))
    y, dz, dw = _empty((15, n), kind), _empty((40, n), kind), torch.empty(15, 3, device="cuda")
    kq.kq_combine(z, slot, y, weight=w, residual=res)
    kq.kq_combine_backward(dy, z, slot, dz, weight=w, dweight=dw)
    zw, dyw, rw, yw, dzw = (wide(r, 123.0) for r in (40, 15, 15, 15, 40))
    for t, v in ((zw, z), (dyw, dy), (rw, res)):
        inner(t).copy_(v)
    kq.kq_combine(inner(zw), slot, inner(yw), weight=w, residual=inner(rw))
    assert torch.equal(inner(yw), y)
    d2 = torch.empty_like(dw)
    kq.kq_combine_backward(inner(dyw), inner(zw), slot, inner(dzw), weight=w, dweight=d2)
    assert torch.equal(inner(dzw), dz) and torch.equal(d2, dw)
    for t in (yw, dzw):
        inner(t).fill_(123.0)
        assert bool((t == 123.0).all())


def test_combine_of_what_is_not_finite():
    """A NaN weight without a slot shows; an infinite row reaches only the rows that choose it."""
    torch = torch_cuda()
    kq = _kq()
    z = torch.ones(4, 20, device="cuda")
    z[2] = INF
    slot = torch.tensor([[0, 1], [2, 3], [-1, 1], [-1, -1], [9, 0]], dtype=torch.int32, device="cuda")
    w = torch.full((5, 2), 0.5, device="cuda")
    w[2, 0] = np.nan
    y = torch.empty(5, 20, device="cuda")
    kq.kq_combine(z, slot, y, weight=w)
    assert torch.equal(y[0], torch.ones(20, device="cuda")) and torch.isinf(y[1]).all() and torch.isnan(y[2]).all()
    assert not y[3].any() and torch.equal(y[4], torch.full((20,), 0.5, device="cuda"))
    kq.kq_combine(z[:0], slot, y)
    assert not y.any()


def test_combine_past_32_bits():
    """More than 2^32 elements of z, named from both ends."""
    torch = torch_cuda()
    kq = _kq()
    slots, n = (1 << 20) + 5, 4100
    z = torch.zeros(slots, n, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    slot = torch.tensor([[0, slots - 1], [slots - 3, 7], [1 << 19, slots // 3]], dtype=torch.int32, device="cuda")
    z[slot.view(-1).long()] = torch.randn(6, n, generator=gen, device="cuda").to(torch.bfloat16)
    y = torch.empty(3, n, device="cuda")
    kq.kq_combine(z, slot, y)
    rows = z[slot.view(-1).long()].float().view(3, 2, n)
    assert torch.equal(y, rows[:, 0] + rows[:, 1])
    dw = torch.empty(3, 2, device="cuda")
    kq.kq_combine_backward(y, z, slot, z, dweight=dw)
    assert torch.equal(z[slot.view(-1).long()].view(3, 2, n), y.to(torch.bfloat16)[:, None].expand(3, 2, n))
    want = (rows.double() * y.double()[:, None]).sum(2)
    assert bool(((dw - want).abs() <= (n + 2) * U * (rows.double() * y.double()[:, None]).abs().sum(2)).all())


@pytest.mark.parametrize("zk,n,top", [("bf16", 4101, 4), ("f32", 2052, 4), ("bf16", 1500, 11)])
def test_combine_of_more_than_the_last_cache(zk, n, top):
    """Rows that go past the caches: the bits of the same rows in calls that do not."""
    announce(f"combine 8200 rows of {n} {zk} top {top}")
    torch = torch_cuda()
    kq = _kq()
    rows, size = 8200, 2 if zk == "bf16" else 4
    gen = torch.Generator(device="cuda").manual_seed(n)
    assert rows * top * n * size > 256 << 20
    z = torch.randn(rows * top, n + 3, generator=gen, device="cuda").to(_dtype(zk))[:, :n]
    slot = torch.randperm(rows * top, generator=gen, device="cuda").int().view(rows, top)
    slot[5, 1], slot[8199, 0] = -1, rows * top
    w = torch.randn(rows, top, generator=gen, device="cuda")
    res = torch.randn(rows, n, generator=gen, device="cuda").to(torch.bfloat16)

    def call(parts):
        y, dz, dw = _empty((rows, n), "bf16"), torch.full((rows * top, n), 5.0, dtype=z.dtype, device="cuda"), torch.empty(rows, top, device="cuda")
        for k in range(parts):
            a = slice(k * rows // parts, (k + 1) * rows // parts)
            kq.kq_combine(z, slot[a], y[a], weight=w[a], residual=res[a])
            kq.kq_combine_backward(res[a], z, slot[a], dz, weight=w[a], dweight=dw[a])
        return y, dz, dw

    for a, b in zip(call(1), call(4)):
        assert torch.equal(a, b)


# ---- a mixture, as it is used ----

def _mixture(rng, tokens, width, inner, experts):
    torch = torch_cuda()
    x = _rows(rng, tokens, width, "bf16").cuda()
    up, down = _layer(rng, 2 * inner, width, experts), _layer(rng, width, inner, experts)
    logits = _logits(rng, tokens, experts, "f32", True).cuda()
    return x, up, down, logits


@pytest.mark.parametrize("tokens", [1, 37, 400])
def test_a_mixture_and_its_routers_gradient(tokens):
    """Route, gated product, product, sum; then the gradients back to the router's logits."""
    announce(f"mixture of {tokens} tokens")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(tokens)
    width, inner, experts, top = 384, 160, 6, 2
    x, up, down, logits = _mixture(rng, tokens, width, inner, experts)
    r = Routes(tokens, experts, top)
    kq.kq_route(logits, normalize=True, **r.dict())
    h, z, y = _empty((tokens * top, inner), "bf16"), _empty((tokens * top, width), "bf16"), _empty((tokens, width), "f32")
    kq.kq_mxfp4_experts_epilogue(x, r.index, r.offsets, up[0], up[1], h, act="silu", gated=True)
    kq.kq_mxfp4_experts(h, None, r.offsets, down[0], down[1], z)
    kq.kq_combine(z, r.slot, y, weight=r.weight, residual=x)
    want = _route_check(r, logits, top, True)
    xq = om.mx_round(_host(x))
    s, mag = _experts_ref(xq, want["index"], want["offsets"], up[2], tokens * top, tokens)
    made = want["offsets"][experts]
    v, bound = _finish(s[:made], (width + 2) * U * mag[:made], None, "silu", True, None, "bf16")
    _within(_host(h)[:made], v, bound, "h")
    assert bool((h[made:] == 123.0).all()) and bool((z[made:] == 123.0).all())
    s, mag = _experts_ref(om.mx_round(_host(h)), None, want["offsets"], down[2], tokens * top, tokens * top)
    _within(_host(z)[:made], s[:made], (inner + 2) * U * mag[:made] * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(s[:made]), "z")
    w = _host(r.weight)
    _within(_host(y), ox.combine(_host(z), want["slot"], w, _host(x)),
            (top + 2) * U * ox.combine(np.abs(_host(z)), want["slot"], w, np.abs(_host(x))), "y")
    dy = torch.from_numpy(rng.standard_normal((tokens, width)).astype(np.float32)).cuda()
    dw, g, dloss = torch.empty(tokens, top, device="cuda"), torch.empty_like(logits), torch.full((1,), 0.01, device="cuda")
    kq.kq_combine_backward(dy, z, r.slot, weight=r.weight, dweight=dw)
    _, rw = ox.combine_backward(_host(dy), _host(z), want["slot"], w)
    _, mw = ox.combine_backward(np.abs(_host(dy)), np.abs(_host(z)), want["slot"], w)
    _within(_host(dw), rw, (width + 2) * U * mw, "dw")
    kq.kq_route_backward(logits, g, r.weight, r.expert, r.counts, dweight=dw, dloss=dloss, normalize=True)
    _route_back_check(g, logits, want, dw.cpu().numpy(), np.float32(0.01), True, "f32")


def test_a_captured_mixture():
    """The whole run replayed from a graph, with new tokens before each replay and eager work between."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(77)
    tokens, width, inner, experts, top = 90, 256, 128, 8, 2
    x, up, down, logits = _mixture(rng, tokens, width, inner, experts)
    ws = torch.empty(max(kq.kq_mxfp4_workspace(tokens, width), kq.kq_mxfp4_workspace(tokens * top, inner)), dtype=torch.uint8, device="cuda")
    wr = torch.empty(kq.kq_route_workspace(tokens, experts, top), dtype=torch.uint8, device="cuda")
    dy = torch.randn(tokens, width, device="cuda")

    def call(x, logits):
        r = Routes(tokens, experts, top)
        h, z, y = _empty((tokens * top, inner), "bf16"), _empty((tokens * top, width), "bf16"), _empty((tokens, width), "bf16")
        dz, dw, g = _empty((tokens * top, width), "bf16"), torch.empty(tokens, top, device="cuda"), torch.empty_like(logits)
        one = torch.ones(1, device="cuda")
        return (r, h, z, y, dz, dw, g, one), lambda: (
            kq.kq_route(logits, ws=wr, **r.dict()),
            kq.kq_mxfp4_experts_epilogue(x, r.index, r.offsets, up[0], up[1], h, ws, act="silu", gated=True),
            kq.kq_mxfp4_experts(h, None, r.offsets, down[0], down[1], z, ws),
            kq.kq_combine(z, r.slot, y, weight=r.weight, residual=x),
            kq.kq_combine_backward(y, z, r.slot, dz, weight=r.weight, dweight=dw),
            kq.kq_route_backward(logits, g, r.weight, r.expert, r.counts, dweight=dw, dloss=one))

    xs, ls = x.clone(), logits.clone()
    held, run = call(xs, ls)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        xs.copy_(_rows(rng, tokens, width, "bf16"))
        ls.copy_(_logits(rng, tokens, experts, "f32", k % 2 == 0))
        for t in held[1:5]:
            t.fill_(123.0)
        graph.replay()
        torch.cuda.synchronize()
        fresh, eager = call(xs, ls)
        eager()
        torch.cuda.synchronize()
        for a, b in zip(held[1:], fresh[1:]):
            assert torch.equal(a, b)
        for name, v in fresh[0].dict().items():
            assert torch.equal(v, getattr(held[0], name)), name


@pytest.mark.parametrize("tokens", [1, 33, 300])
def test_the_examples_router_gradient(tokens):
    """The example's gradient against autograd in 64 bits on the experts' rows that it computed."""
    torch = torch_cuda()
    import examples.mxfp4_mixture as ex
    torch.manual_seed(tokens)
    x, *weights = ex.make(128 + tokens, 256, 160, 6, seed=tokens)
    calibration, x = x[:128], x[128:]
    want = ex.plain(x, *weights, 2)          # (first: processing the weights is done in place)
    block = ex.Mixture(*weights, 2, calibration)
    out, kept = block.forward(x)
    dout = torch.randn_like(out)
    got = block.router_gradient(dout, kept, balance=0.5)
    _, logits, routes, z = kept
    l64 = logits.double().requires_grad_()
    p = torch.softmax(l64, 1)
    chosen = routes.expert.long()
    rows = z[routes.slot.long()].double()
    counts = routes.counts[:6].double()
    loss = 6 * (counts / counts.sum() * p.mean(0)).sum()
    w = p.gather(1, chosen)
    dl = torch.autograd.grad(((w[:, :, None] * rows).sum(1) * dout.double()).sum() + 0.5 * loss, l64)[0]
    assert abs(float(routes.loss) - float(loss.detach())) <= (100 + 6 + 16 + tokens) * U * float(loss.detach())
    # dweight is off by (n + 2) u sum |dy z|, the softmax by the module's bound, the product by (T + 2) u
    mag = (rows.abs() * dout.double().abs()[:, None]).sum(2)
    size = p.detach() * (w.detach() * mag).sum(1, keepdim=True) + 0.5 * p.detach()
    size = size.scatter_add(1, chosen, w.detach() * mag)
    xd = x.double()
    # (torch's fp32 product adds T terms in an order of its own)
    bound = xd.abs().T @ (size * (256 + 2 + 500) * U) + (tokens + 2) * U * (xd.abs().T @ dl.abs())
    assert bool(((got.double() - xd.T @ dl).abs() <= bound).all())
    assert float((out - want).norm() / want.norm()) < 0.25      # (as the block's own test has it)


def test_routing_on_two_streams_at_once():
    """Calls on two streams with the workspaces that the binding allocates: the bits of a call by itself."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(5)
    inputs = [_logits(rng, 3000, 64, "bf16", True).cuda() for _ in range(6)]
    want, got = [Routes(3000, 64, 6) for _ in inputs], [Routes(3000, 64, 6) for _ in inputs]
    for x, r in zip(inputs, want):
        kq.kq_route(x, **r.dict())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for k, x in enumerate(inputs):
        kq.kq_route(x, stream=streams[k % 2], **got[k].dict())
        torch.full((kq.kq_route_workspace(3000, 64, 6),), k, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for name, v in a.dict().items():
            assert torch.equal(v, getattr(b, name)), name


@pytest.mark.parametrize("rows", [1, 40, 500])
def test_epilogues_and_sums_on_given_streams(rows):
    """Calls on two streams with the workspaces that the binding allocates: the bits of a call by itself."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    n, out = 1024, 200
    wc, ws, _ = _layer(rng, 2 * out, n)
    slot = _dev(_choices(rng, rows, 3, 3 * rows, False))
    inputs = [_rows(rng, rows, n, "bf16").cuda() for _ in range(6)]
    z = [torch.randn(3 * rows, out, device="cuda") for _ in inputs]

    def call(x, z, stream=None):
        y, s = _empty((rows, out), "bf16"), _empty((rows, out), "f32")
        dz, dw = torch.empty_like(z), torch.empty(rows, 3, device="cuda")
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        kq.kq_mxfp4_linear_epilogue(x, wc, ws, y, act="gelu", gated=True, had=n, stream=stream)
        kq.kq_combine(z, slot, s, residual=y, stream=stream)
        kq.kq_combine_backward(s, z, slot, dz, dweight=dw, stream=stream)
        return y, s, dz, dw

    want = [call(x, v) for x, v in zip(inputs, z)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [call(x, v, streams[k % 2]) for k, (x, v) in enumerate(zip(inputs, z))]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_routing_with_a_larger_workspace():
    """One workspace for the largest batch serves all smaller ones."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(6)
    ws = torch.full((kq.kq_route_workspace(131_200, 16, 2),), 255, dtype=torch.uint8, device="cuda")
    for rows in (131_200, 131_072, 33_000, 4000, 70, 3):
        x = _logits(rng, rows, 16, "f32", False).cuda()
        r, own = Routes(rows, 16, 2), Routes(rows, 16, 2)
        kq.kq_route(x, ws=ws, **r.dict())
        kq.kq_route(x, **own.dict())
        for name, v in r.dict().items():
            assert torch.equal(v, getattr(own, name)), name


def test_the_binding_refuses():
    torch = torch_cuda()
    kq = _kq()
    x, r = torch.randn(8, 4, device="cuda"), Routes(8, 4, 2)
    kq.kq_route(x, **r.dict())
    for bad in (dict(weight=r.weight.double()), dict(expert=r.expert[:7]), dict(index=r.index[1:]), dict(offsets=r.offsets[:4]),
                dict(counts=r.counts[:5]), dict(loss=r.weight), dict(slot=r.slot.long()), dict(slot=r.slot.cpu())):
        with pytest.raises((TypeError, ValueError)):
            kq.kq_route(x, **{**r.dict(), **bad})
    with pytest.raises(kq.KQError):
        kq.kq_route(x[:1].expand(8, 4), **r.dict())                       # rows that overlap
    with pytest.raises(ValueError):
        kq.kq_route(x.t().contiguous().t(), **r.dict())
    many = Routes(5000, 4, 2)
    with pytest.raises(kq.KQError):
        kq.kq_route(torch.randn(5000, 4, device="cuda"), ws=torch.empty(16, dtype=torch.uint8, device="cuda"), **many.dict())
    with pytest.raises(ValueError):
        kq.kq_route_backward(x, x.bfloat16(), r.weight, r.expert, r.counts)
    z, y = torch.randn(16, 12, device="cuda"), torch.empty(8, 12, device="cuda")
    for bad in (dict(slot=r.slot[:7]), dict(y=y[:, :11]), dict(weight=r.weight[:, :1]), dict(residual=y[:7])):
        with pytest.raises((TypeError, ValueError)):
            kq.kq_combine(**{**dict(z=z, slot=r.slot, y=y), **bad})
    with pytest.raises(kq.KQError):
        kq.kq_combine(z[:1].expand(16, 12), r.slot, y)
    with pytest.raises(ValueError):
        kq.kq_combine_backward(y, z, r.slot, dz=z.bfloat16())
    codes, scales = kq.kq_mxfp4_empty(24, 128)
    xx = torch.randn(3, 128, device="cuda")
    out = torch.empty(3, 12, device="cuda")
    kq.kq_mxfp4_quantize(torch.randn(24, 128, device="cuda"), codes, scales)
    kq.kq_mxfp4_linear_epilogue(xx, codes, scales, out, gated=True, act="relu")
    for bad in (dict(gated=False), dict(act="swish"), dict(bias=torch.zeros(12, device="cuda")), dict(bias=torch.zeros(24, device="cuda").double()),
                dict(residual=out[:2]), dict(residual=out.half())):
        with pytest.raises((TypeError, ValueError)):
            kq.kq_mxfp4_linear_epilogue(xx, codes, scales, out, **{**dict(gated=True), **bad})
