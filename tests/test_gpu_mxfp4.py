"""GPU parity of the MXFP4 operators against plain 64-bit implementations.

Quantisation is held to equality: with no rotation the elements of a given fp32 or bf16 row
are determined, and with one the definition fixes every fp32 rounding (butterflies with
ascending strides), which numpy's fp32 repeats; against the 64-bit rotation they may differ
only next to a rounding boundary.  Products: a sum of K terms in fp32, in any order, is off by
at most (K + 2) 2^-24 sum |x w|, and by half an ulp more after the rounding to bf16.
"""
import numpy as np
import pytest

import oracle.mxfp4 as om
from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def _kq():
    import post_quantization_syrk_amd as kq
    return kq


def _rows(rng, rows, n, kind):
    torch = torch_cuda()
    x = rng.standard_normal((rows, n)) * np.exp(rng.standard_normal(n))
    x = torch.from_numpy(x.astype(np.float32))
    return x.to(torch.bfloat16) if kind == "bf16" else x


def _processing(rng, n, rescale, signed):
    d = np.exp(0.5 * rng.standard_normal(n)).astype(np.float32) if rescale else None
    s = rng.choice([-1, 1], n).astype(np.int8) if signed else None
    return d, s


def _dev(a):
    torch = torch_cuda()
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _quantize(x, d=None, sign=None, had=1, values=True, stream=None):
    """(codes, scale bytes, values) of device rows x, unpacked."""
    torch = torch_cuda()
    kq = _kq()
    rows, n = x.shape
    codes, scales = kq.kq_mxfp4_empty(rows, n)
    codes.fill_(0xAA)
    scales.fill_(0xAA)
    vals = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda") if values else None
    kq.kq_mxfp4_quantize(x, codes, scales, d=_dev(d), sign=_dev(sign), had=had, values=vals, stream=stream)
    torch.cuda.synchronize()
    return (*om.mx_unpack(codes.cpu().numpy(), scales.cpu().numpy()), vals.float().cpu().numpy() if values else None)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 31), (3, 32), (1, 33), (5, 100), (4, 128), (3, 129), (2, 1000),
                                    (1, 4096), (3, 4224), (2, 11008), (70, 515), (1, 8200), (300, 64)])
def test_quantize_without_rotation(rows, n, kind):
    announce(f"mxfp4 quantize {rows}x{n} {kind}")
    rng = np.random.default_rng(rows * 100003 + n)
    x = _rows(rng, rows, n, kind)
    code, scale, values = _quantize(x.cuda())
    ref = x.double().numpy()
    c, s = om.mx_encode(ref)
    assert np.array_equal(code & 7, c & 7) and np.array_equal(scale, s)
    assert np.array_equal(values, om.mx_values(c, s, n))
    d, sg = _processing(rng, n, True, True)
    code, scale, values = _quantize(x.cuda(), d, sg)
    c, s = om.mx_encode(om.mx_rotate_f32(x.float().numpy(), d, sg))
    assert np.array_equal(code, c) and np.array_equal(scale, s)
    assert np.array_equal(values, om.mx_values(c, s, n))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,had", [(2, 2, 2), (3, 36, 4), (5, 1000, 8), (2, 48, 16), (3, 96, 32), (2, 192, 64),
                                        (3, 384, 128), (9, 256, 256), (2, 11008, 256), (3, 1536, 512), (2, 1024, 1024),
                                        (2, 6144, 2048), (1, 4096, 4096), (33, 4096, 4096), (2, 12288, 4096),
                                        (1, 8192, 8192), (3, 24576, 8192), (17, 2048, 2048), (2, 8192, 16)])
def test_quantize_with_rotation(rows, n, had, kind):
    announce(f"mxfp4 quantize {rows}x{n} block {had} {kind}")
    rng = np.random.default_rng(rows + 7 * n + had)
    x = _rows(rng, rows, n, kind)
    d, sg = _processing(rng, n, True, True)
    code, scale, values = _quantize(x.cuda(), d, sg, had)
    xr = om.mx_rotate_f32(x.float().numpy(), d, sg, had)
    c, s = om.mx_encode(xr)
    assert np.array_equal(code & 7, c & 7) and np.array_equal(scale, s)
    assert np.array_equal(values, om.mx_values(c, s, n))
    # against the rotation in 64 bits: equal but next to a boundary.  Each of log2(had) + 2 stages
    # rounds by 2^-24 of a partial sum, so an entry is off by at most that times the block's norm
    exact = om.mx_rotate(x.double().numpy(), d, sg, had)
    norm = np.sqrt((exact.reshape(rows, -1, had) ** 2).sum(-1, keepdims=True))
    off = (np.log2(had) + 3) * 2.0 ** -24 * np.broadcast_to(norm, (rows, n // had, had)).reshape(rows, n)
    rel = np.minimum((off / np.maximum(np.abs(exact), 1e-30)), 0.5)
    differ = om.mx_round(exact) != values
    sure = (om.mx_round(exact - off) == om.mx_round(exact + off)) & ~om.mx_near_tie(exact, float(np.median(rel)) * 8)
    assert not (differ & sure).any()
    assert differ.mean() <= 1e-3


@pytest.mark.parametrize("signed,rescale,had", [(True, False, 1), (False, True, 1), (True, False, 64), (False, True, 64),
                                                (False, False, 64), (False, False, 0)])
def test_quantize_parts_of_the_processing(signed, rescale, had):
    rng = np.random.default_rng(3)
    x = _rows(rng, 7, 448, "f32")
    d, sg = _processing(rng, 448, rescale, signed)
    code, scale, values = _quantize(x.cuda(), d, sg, had)
    c, s = om.mx_encode(om.mx_rotate_f32(x.numpy(), d, sg, had or 64))
    assert np.array_equal(code & 7, c & 7) and np.array_equal(scale, s)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("had", [1, 4])
def test_quantize_edges(kind, had):
    """Zero blocks, the smallest and the largest numbers, ties, infinities and NaN."""
    announce(f"mxfp4 quantize edges {kind} block {had}")
    x = np.zeros((8, 128), np.float32)
    x[0, :8] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25]
    x[0, 32:40] = [-8, -7, -5, -3, -2.5, -1.5, -0.5, 7.96875]
    x[1, 5], x[1, 40], x[1, 70] = 2.0 ** -149 if kind == "f32" else 2.0 ** -133, 2.0 ** -126, 2.0 ** -127
    x[2, :4] = [3.3e38, -3.3e38, 1e30, 0] if had == 1 else [1e37, 1e30, 0, 0]
    x[3, 3], x[3, 64:66] = np.inf, [1, -2]
    x[4, 127], x[4, 0] = np.nan, 1
    x[5, 33] = -np.inf
    x[6] = -0.0
    x[7] = np.linspace(-7.9, 7.9, 128)
    torch = torch_cuda()
    xt = torch.from_numpy(x)
    xt = xt.to(torch.bfloat16) if kind == "bf16" else xt
    code, scale, values = _quantize(xt.cuda(), had=had)
    with np.errstate(invalid="ignore", over="ignore"):
        r = om.mx_rotate_f32(xt.float().numpy(), had=had)
    c, s = om.mx_encode(r)
    assert np.array_equal(scale, s)
    assert np.array_equal(code & 7, c & 7)
    assert np.array_equal(values, om.mx_values(c, s, 128), equal_nan=True)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad,had", [(1, 3, 1), (2, 6, 1), (0, 7, 1), (4, 4, 8), (1, 1, 8), (3, 0, 512), (8, 8, 512)])
def test_quantize_strides_and_alignment(kind, off, pad, had):
    """Rows inside a wider buffer, starting at any element; values into a wider buffer."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(off + pad)
    wide = _rows(rng, 6, off + 1024 + pad, kind).cuda()
    x = wide[:, off:off + 1024]
    values = torch.zeros((6, 1040), dtype=torch.bfloat16, device="cuda")
    codes, scales = kq.kq_mxfp4_empty(6, 1024)
    kq.kq_mxfp4_quantize(x, codes, scales, had=had, values=values[:, 5:1029])
    c, s = om.mx_encode(om.mx_rotate_f32(x.float().cpu().numpy(), had=had))
    v = values.float().cpu().numpy()
    assert np.array_equal(v[:, 5:1029], om.mx_values(c, s, 1024))
    assert not v[:, :5].any() and not v[:, 1029:].any()
    code, scale = om.mx_unpack(codes.cpu().numpy(), scales.cpu().numpy())
    assert np.array_equal(code & 7, c & 7) and np.array_equal(scale, s)


def _layer(rng, out, n, experts=None):
    """Codes and scales on the device of random weights, and their values [.., out, n]."""
    torch = torch_cuda()
    kq = _kq()
    lead = 1 if experts is None else experts
    codes, scales = kq.kq_mxfp4_empty(out, n, experts=lead)
    vals = []
    for e in range(lead):
        c, s = om.mx_encode(0.05 * rng.standard_normal((out, n)) * np.exp(0.5 * rng.standard_normal((out, 1))))
        vals.append(om.mx_values(c, s, n))
        pc, ps = om.mx_pack(c, s)
        codes[e].copy_(torch.from_numpy(pc))
        scales[e].copy_(torch.from_numpy(ps))
    return (codes[0], scales[0], vals[0]) if experts is None else (codes, scales, np.stack(vals))


def _close(y, xq, w, bf16):
    """y against xq w^T within the bound of an fp32 sum."""
    ref, mag = xq @ w.T, np.abs(xq) @ np.abs(w.T)
    bound = (xq.shape[1] + 2) * 2.0 ** -24 * mag
    if bf16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    y = y.double().cpu().numpy()
    assert np.all(np.abs(y - ref) <= bound), float((np.abs(y - ref) - bound).max())


def _empty(shape, kind):
    torch = torch_cuda()
    return torch.full(shape, 123.0, dtype=torch.bfloat16 if kind == "bf16" else torch.float32, device="cuda")


@pytest.mark.parametrize("rows,n,out,had,xk,yk", [
    (1, 128, 1, 128, "bf16", "f32"), (1, 4096, 4096, 4096, "bf16", "bf16"), (1, 33, 17, 1, "f32", "f32"),
    (2, 1, 3, 1, "f32", "bf16"), (3, 1000, 4099, 8, "bf16", "f32"), (1, 11008, 100, 256, "f32", "bf16"),
    (7, 512, 65, 512, "bf16", "bf16"), (16, 2048, 300, 2048, "bf16", "f32"), (17, 640, 128, 128, "f32", "f32"),
    (31, 192, 1000, 64, "bf16", "bf16"), (32, 256, 256, 256, "bf16", "f32"), (33, 256, 31, 256, "f32", "bf16"),
    (64, 4096, 96, 4096, "bf16", "f32"), (65, 1024, 130, 1024, "bf16", "bf16"), (100, 96, 1, 32, "f32", "f32"),
    (128, 384, 515, 128, "bf16", "bf16"), (200, 8192, 257, 8192, "bf16", "f32"), (256, 128, 256, 1, "bf16", "f32"),
    (257, 512, 700, 512, "f32", "bf16"), (300, 1000, 1001, 8, "bf16", "f32"), (513, 320, 2050, 64, "bf16", "bf16"),
    (1100, 2048, 600, 2048, "bf16", "f32"),
])
def test_linear(rows, n, out, had, xk, yk):
    announce(f"mxfp4 linear {rows}x{n} -> {out} block {had} {xk} {yk}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows + 3 * n + 5 * out)
    x = _rows(rng, rows, n, xk)
    if rows > 2:
        x[rows // 2] = 0
    d, sg = _processing(rng, n, had > 1, had > 1)
    wc, ws, wv = _layer(rng, out, n)
    y = _empty((rows, out), yk)
    kq.kq_mxfp4_linear(x.cuda(), wc, ws, y, d=_dev(d), sign=_dev(sg), had=had)
    xq = om.mx_round(om.mx_rotate_f32(x.float().numpy(), d, sg, had))
    _close(y, xq, wv, yk == "bf16")
    # activations quantised beforehand give the same bits; so does a second call
    xc, xs = kq.kq_mxfp4_empty(rows, n)
    kq.kq_mxfp4_quantize(x.cuda(), xc, xs, d=_dev(d), sign=_dev(sg), had=had)
    again = _empty((rows, out), yk)
    kq.kq_mxfp4_linear(xc, wc, ws, again, x_scales=xs, n=n)
    assert torch.equal(y, again)
    kq.kq_mxfp4_linear(x.cuda(), wc, ws, again, d=_dev(d), sign=_dev(sg), had=had)
    assert torch.equal(y, again)


@pytest.mark.parametrize("rows", [1, 5, 40, 150])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 2), (4, 4), (8, 8)])
def test_linear_strided_output(rows, off, pad):
    """An output inside a wider buffer, at any element: nothing around it is written."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    x = _rows(rng, rows, 256, "bf16").cuda()
    wc, ws, wv = _layer(rng, 200, 256)
    xq = om.mx_round(x.double().cpu().numpy())
    for kind in ("bf16", "f32"):
        wide = _empty((rows + 2, off + 200 + pad), kind)
        kq.kq_mxfp4_linear(x, wc, ws, wide[1:-1, off:off + 200])
        _close(wide[1:-1, off:off + 200], xq, wv, kind == "bf16")
        rest = wide.clone()
        rest[1:-1, off:off + 200] = 123.0
        assert torch.equal(rest, _empty(tuple(wide.shape), kind))


@pytest.mark.parametrize("rows", [1, 20, 130])
def test_not_finite_values_stay_in_their_rows(rows):
    """An infinity in an activation makes its own output row NaN; a NaN block in a weight row
    makes that output column NaN; everything else is untouched."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    x = _rows(rng, rows, 320, "f32")
    wc, ws, wv = _layer(rng, 150, 320)
    y0 = _empty((rows, 150), "f32")
    kq.kq_mxfp4_linear(x.cuda(), wc, ws, y0)
    x[rows - 1, 300] = np.inf
    ws2 = ws.clone()
    ws2[1, 77, 2] = 255
    y1 = _empty((rows, 150), "f32")
    kq.kq_mxfp4_linear(x.cuda(), wc, ws2, y1)
    bad = torch.zeros((rows, 150), dtype=torch.bool, device="cuda")
    bad[rows - 1] = True
    bad[:, 77] = True
    assert torch.equal(torch.isnan(y1), bad)
    assert torch.equal(y1[~bad], y0[~bad])


@pytest.mark.parametrize("rows", [1, 24, 140])
def test_linear_of_extreme_scales(rows):
    """Scale bytes from one end of their range to the other, with products inside fp32's."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(5)
    n, out = 256, 40
    code, scale = om.mx_encode(rng.standard_normal((rows, n)))
    wcode, wscale = om.mx_encode(rng.standard_normal((out, n)))
    for xb, wb in ((0, 127), (0, 240), (252, 10), (252, 100), (60, 80)):
        scale[:], wscale[:] = xb, wb
        xc, xs = (torch.from_numpy(a).cuda() for a in om.mx_pack(code, scale))
        wc, ws = (torch.from_numpy(a).cuda() for a in om.mx_pack(wcode, wscale))
        y = _empty((rows, out), "f32")
        kq.kq_mxfp4_linear(xc, wc, ws, y, x_scales=xs, n=n)
        ref = om.mx_values(code, scale, n) @ om.mx_values(wcode, wscale, n).T
        tiny = 2.0 ** -126 if xb + wb < 140 else 0.0   # results below fp32's normal range may be flushed
        assert np.all(np.abs(y.double().cpu().numpy() - ref) <= (n + 2) * 2.0 ** -24 * np.abs(ref).max() + tiny)


def _experts_ref(xq, index, offsets, w, slots, rows):
    want = np.full((slots, w.shape[1]), 123.0)
    mag = np.zeros_like(want)
    for e in range(w.shape[0]):
        lo = min(max(int(offsets[e]), 0), slots)
        hi = min(max(int(offsets[e + 1]), lo), slots)
        for s in range(lo, hi):
            r = s if index is None else int(index[s])
            x = xq[r] if 0 <= r < rows else np.zeros(xq.shape[1])
            want[s], mag[s] = w[e] @ x, np.abs(w[e]) @ np.abs(x)
    return want, mag


def _experts_check(y, want, mag, n, bf16):
    bound = (n + 2) * 2.0 ** -24 * mag
    if bf16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) * (mag > 0)
    got = y.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) - bound).max())


def _sorted_slots(rng, tokens, top, experts, skew):
    popular = skew * rng.standard_normal(experts)
    chosen = np.argsort(-(popular + rng.standard_normal((tokens, experts))), axis=1)[:, :top].reshape(-1)
    order = np.argsort(chosen, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(chosen, minlength=experts))])
    return (order // top).astype(np.int32), offsets.astype(np.int32)


@pytest.mark.parametrize("tokens,top,experts,n,out,had,xk,yk,skew", [
    (1, 1, 1, 128, 16, 128, "bf16", "f32", 0.0), (1, 2, 8, 512, 130, 512, "bf16", "bf16", 1.0),
    (5, 2, 4, 1000, 65, 8, "f32", "f32", 1.0), (33, 4, 16, 256, 200, 256, "bf16", "f32", 2.0),
    (96, 6, 64, 384, 100, 128, "bf16", "bf16", 1.0), (200, 1, 3, 640, 257, 128, "f32", "bf16", 2.0),
    (300, 2, 5, 256, 300, 256, "bf16", "f32", 1.0), (64, 8, 128, 128, 33, 128, "bf16", "f32", 0.5),
    (700, 2, 4, 512, 520, 512, "bf16", "bf16", 1.5), (3, 3, 300, 96, 20, 32, "f32", "f32", 0.0),
])
def test_experts(tokens, top, experts, n, out, had, xk, yk, skew):
    announce(f"mxfp4 experts {tokens}x{top} of {experts} {n} -> {out}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(tokens + experts + n)
    x = _rows(rng, tokens, n, xk)
    d, sg = _processing(rng, n, True, True)
    index, offsets = _sorted_slots(rng, tokens, top, experts, skew)
    wc, ws, wv = _layer(rng, out, n, experts)
    y = _empty((tokens * top, out), yk)
    kq.kq_mxfp4_experts(x.cuda(), _dev(index), _dev(offsets), wc, ws, y, d=_dev(d), sign=_dev(sg), had=had)
    xq = om.mx_round(om.mx_rotate_f32(x.float().numpy(), d, sg, had))
    want, mag = _experts_ref(xq, index, offsets, wv, tokens * top, tokens)
    _experts_check(y, want, mag, n, yk == "bf16")
    again = _empty((tokens * top, out), yk)
    xc, xs = kq.kq_mxfp4_empty(tokens, n)
    kq.kq_mxfp4_quantize(x.cuda(), xc, xs, d=_dev(d), sign=_dev(sg), had=had)
    kq.kq_mxfp4_experts(xc, _dev(index), _dev(offsets), wc, ws, again, x_scales=xs, n=n)
    assert torch.equal(y, again)


@pytest.mark.parametrize("slots,offsets", [
    (50, [0, 0, 0, 50, 50]),        # everything with one expert
    (50, [0, 0, 0, 0, 0]),          # nothing with any
    (50, [10, 20, 20, 30, 41]),     # slots before the first and after the last expert
    (50, [0, 1, 2, 3, 4]),          # one slot each
    (50, [-7, 20, 60, 70, 90]),     # offsets that leave the range are cut
    (50, [0, 30, 20, 25, 50]),      # decreasing: that expert has none
    (300, [0, 129, 129, 257, 300]),
])
@pytest.mark.parametrize("indexed", [True, False])
def test_experts_ranges(slots, offsets, indexed):
    """Slots outside every expert keep what y held; an index outside the rows reads zeros."""
    kq = _kq()
    rng = np.random.default_rng(slots + offsets[1])
    n, out = 160, 70
    rows = 20 if indexed else slots
    x = _rows(rng, rows, n, "bf16")
    index = rng.integers(0, rows, slots).astype(np.int32) if indexed else None
    if indexed:
        index[[0, 3, slots - 1]] = [-1, rows, 2 ** 31 - 1]
    wc, ws, wv = _layer(rng, out, n, 4)
    y = _empty((slots, out), "f32")
    kq.kq_mxfp4_experts(x.cuda(), _dev(index), _dev(np.int32(offsets)), wc, ws, y)
    # ranges may overlap where the offsets decrease: a later expert's rows are then any of the two
    want, mag = _experts_ref(om.mx_round(x.double().numpy()), index, offsets, wv, slots, rows)
    if offsets != sorted(offsets):
        want, mag, y = want[30:], mag[30:], y[30:]
    _experts_check(y, want, mag, n, False)


def test_experts_of_no_rows():
    """No rows of x at all: every index is outside, every reached slot is zero."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(0)
    wc, ws, _ = _layer(rng, 40, 128, 2)
    y = _empty((10, 40), "f32")
    x = torch.empty((0, 128), device="cuda")
    kq.kq_mxfp4_experts(x, torch.zeros(10, dtype=torch.int32, device="cuda"),
                        torch.tensor([0, 4, 9], dtype=torch.int32, device="cuda"), wc, ws, y)
    want = _empty((10, 40), "f32")
    want[:9] = 0
    assert torch.equal(y, want)


def test_another_stream_and_a_graph():
    """On a stream of its own, and captured: every replay gives the eager result of its inputs."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(9)
    d, sg = _processing(rng, 512, True, True)
    d, sg = _dev(d), _dev(sg)
    wc, ws, _ = _layer(rng, 200, 512)
    ec, es, _ = _layer(rng, 96, 512, 4)
    inputs = [_rows(rng, 40, 512, "bf16").cuda() for _ in range(4)]
    index, offsets = (_dev(v) for v in _sorted_slots(rng, 40, 2, 4, 1.0))
    x = inputs[0].clone()
    work = torch.empty(kq.kq_mxfp4_workspace(40, 512), dtype=torch.uint8, device="cuda")
    y, z = _empty((40, 200), "f32"), _empty((80, 96), "bf16")

    def both(x, y, z, work=work):
        kq.kq_mxfp4_linear(x, wc, ws, y, work, d=d, sign=sg, had=512)
        kq.kq_mxfp4_experts(x, index, offsets, ec, es, z, work, d=d, sign=sg, had=512)

    eager = []
    for v in inputs:
        a, b = _empty((40, 200), "f32"), _empty((80, 96), "bf16")
        both(v, a, b)
        eager.append((a, b))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        both(inputs[1], y, z)
    side.synchronize()
    assert torch.equal(y, eager[1][0]) and torch.equal(z, eager[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(x, y, z)
    for k in (1, 3, 2, 0, 3):
        x.copy_(inputs[k])
        y.fill_(5.0)
        graph.replay()
        a, b = _empty((40, 200), "f32"), _empty((80, 96), "bf16")
        torch.cuda.synchronize()
        both(inputs[k], a, b, torch.empty_like(work))
        assert torch.equal(y, eager[k][0]) and torch.equal(z, eager[k][1])
        assert torch.equal(a, y) and torch.equal(b, z)


def test_refusals_of_the_binding():
    torch = torch_cuda()
    kq = _kq()
    x = torch.zeros((4, 128), device="cuda")
    codes, scales = kq.kq_mxfp4_empty(4, 128)
    with pytest.raises(TypeError):
        kq.kq_mxfp4_quantize(x.half(), codes, scales)
    with pytest.raises(TypeError):
        kq.kq_mxfp4_quantize(x.cpu(), codes, scales)
    with pytest.raises(ValueError):
        kq.kq_mxfp4_quantize(x, codes[:3], scales)
    with pytest.raises(ValueError):
        kq.kq_mxfp4_quantize(x, codes, scales, d=torch.ones(127, device="cuda"))
    with pytest.raises(ValueError):
        kq.kq_mxfp4_quantize(x.T.contiguous().T, codes, scales)
    with pytest.raises(kq.KQError) as e:
        kq.kq_mxfp4_quantize(x, codes, scales, had=256)
    assert e.value.status == kq.KQ_ESHAPE
    wc, ws = kq.kq_mxfp4_empty(8, 128)
    y = torch.zeros((4, 8), device="cuda")
    with pytest.raises(ValueError):
        kq.kq_mxfp4_linear(x, wc, ws, y[:, :7])
    with pytest.raises(ValueError):
        kq.kq_mxfp4_linear(codes, wc, ws, y, x_scales=scales)
    with pytest.raises(kq.KQError) as e:
        kq.kq_mxfp4_linear(x, wc, ws, y, torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == kq.KQ_EWORKSPACE
    ec, es = kq.kq_mxfp4_empty(8, 128, experts=2)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        kq.kq_mxfp4_experts(x, None, off.long(), ec, es, y)
    with pytest.raises(ValueError):
        kq.kq_mxfp4_experts(x, None, off[:2], ec, es, y)


def _forced(knobs):
    """A context in which the implementation paths are chosen by `knobs` (name -> value)."""
    from contextlib import ExitStack
    kq = _kq()
    stack = ExitStack()
    for name, value in knobs.items():
        stack.enter_context(kq.testing_select(getattr(kq, name), value))
    return stack


PATHS = [dict(KQ_TESTING_MX_FUSED=0), dict(KQ_TESTING_MX_FUSED=1 << 20),
         *(dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=t) for t in (256, 128, 64)),
         dict(KQ_TESTING_MX_FEW=1 << 20)]


@pytest.mark.parametrize("path", PATHS, ids=str)
@pytest.mark.parametrize("rows,n,out,had", [(1, 4096, 300, 4096), (3, 1000, 515, 8), (13, 640, 64, 128), (16, 2048, 96, 2048),
                                            (2, 8192, 130, 8192), (40, 384, 257, 128), (64, 1536, 300, 512),
                                            (150, 256, 1000, 256), (700, 1152, 520, 128), (1300, 128, 1100, 128)])
def test_every_path(rows, n, out, had, path):
    """Each implementation gives the product within the bound, for a layer and for experts."""
    announce(f"mxfp4 {rows}x{n} -> {out} {path}")
    kq = _kq()
    rng = np.random.default_rng(rows + n)
    x = _rows(rng, rows, n, "bf16")
    d, sg = _processing(rng, n, True, True)
    wc, ws, wv = _layer(rng, out, n)
    ec, es, ev = _layer(rng, 72, n, 5)
    index, offsets = _sorted_slots(rng, rows, 2, 5, 1.0)
    xq = om.mx_round(om.mx_rotate_f32(x.float().numpy(), d, sg, had))
    want, mag = _experts_ref(xq, index, offsets, ev, 2 * rows, rows)
    with _forced(path):
        for kind in ("f32", "bf16"):
            y, z = _empty((rows, out), kind), _empty((2 * rows, 72), kind)
            kq.kq_mxfp4_linear(x.cuda(), wc, ws, y, d=_dev(d), sign=_dev(sg), had=had)
            _close(y, xq, wv, kind == "bf16")
            kq.kq_mxfp4_experts(x.cuda(), _dev(index), _dev(offsets), ec, es, z, d=_dev(d), sign=_dev(sg), had=had)
            _experts_check(z, want, mag, n, kind == "bf16")


def _random_codes(rows, n, experts=None):
    """Device codes of any elements with scales 2^-3 .. 2^3 (NaN blocks would spread)."""
    torch = torch_cuda()
    kq = _kq()
    gen = torch.Generator(device="cuda").manual_seed(rows + n)
    codes, scales = kq.kq_mxfp4_empty(rows, n, experts)
    codes.random_(0, 256, generator=gen)
    scales.random_(124, 131, generator=gen)
    return codes, scales


def _values(codes, scales, rows):
    """64-bit values of the given rows of device codes."""
    torch = torch_cuda()
    rows = torch.as_tensor(rows, device="cuda")
    return om.mx_values(*om.mx_unpack(codes[rows].cpu().numpy(), scales[:, rows].contiguous().cpu().numpy()), 2 * codes.shape[1])


@pytest.mark.parametrize("rows", [700_000, 1_060_000])
def test_experts_of_rows_past_32_bits(rows):
    """Quantised rows of more than 2 GiB and of more than 4 GiB, read through an index."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    n, out, slots = 8192, 70, 150
    codes, scales = _random_codes(rows, n)
    index = rng.integers(0, rows, slots).astype(np.int32)
    index[[0, 1, 149]] = [rows - 1, 0, rows - 2]
    wc, ws, wv = _layer(rng, out, n, 2)
    y = _empty((slots, out), "f32")
    offsets = np.int32([0, 3, slots])
    kq.kq_mxfp4_experts(codes, _dev(index), _dev(offsets), wc, ws, y, x_scales=scales, n=n)
    xq = _values(codes, scales, index)
    want, mag = _experts_ref(xq, None, offsets, wv, slots, slots)
    _experts_check(y, want, mag, n, False)
    near = _empty((slots, out), "f32")   # the same rows side by side: the same sums
    picked = torch.from_numpy(index).long().cuda()
    with _forced(dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=256)):
        kq.kq_mxfp4_experts(codes[picked], None, _dev(offsets), wc, ws, near,
                            x_scales=scales[:, picked].contiguous(), n=n)
    assert rows < 1_000_000 or torch.equal(y, near)


def test_linear_of_an_output_past_32_bits():
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(3)
    rows, n, out = 1_000_003, 128, 2200
    codes, scales = _random_codes(rows, n)
    wc, ws, wv = _layer(rng, out, n)
    y = _empty((rows, out), "bf16")
    kq.kq_mxfp4_linear(codes, wc, ws, y, x_scales=scales, n=n)
    some = np.concatenate([[0, 1, rows - 1, rows - 2, rows - 3], rng.integers(0, rows, 200)])
    _close(y[torch.from_numpy(some).cuda()], _values(codes, scales, some), wv, True)


@pytest.mark.parametrize("slots", [40, 600])
def test_experts_of_layers_past_32_bits(slots):
    kq = _kq()
    rng = np.random.default_rng(slots)
    n, out, experts = 8192, 4096, 260
    wc, ws = _random_codes(out, n, experts)
    x, xs = _random_codes(slots, n)
    offsets = np.zeros(experts + 1, np.int32)
    offsets[2:] = slots // 2          # the first half to expert 1, the rest to the last
    offsets[-1] = slots
    y = _empty((slots, out), "f32")
    kq.kq_mxfp4_experts(x, None, _dev(offsets), wc, ws, y, x_scales=xs, n=n)
    xq = _values(x, xs, np.arange(slots))
    for lo, hi, e in ((0, slots // 2, 1), (slots // 2, slots, experts - 1)):
        _close(y[lo:hi], xq[lo:hi], _values(wc[e], ws[e], np.arange(out)), False)


def test_quantize_past_32_bits():
    """The last rows of more than 4 GiB of input, and of more than 2^31 values, as a small call has them."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(4)
    rows, n, had = 140_000, 16384, 4096
    d, sg = (_dev(v) for v in _processing(rng, n, True, True))
    x = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = kq.kq_mxfp4_empty(rows, n)
    values = torch.empty_like(x)
    kq.kq_mxfp4_quantize(x, codes, scales, d=d, sign=sg, had=had, values=values)
    for lo in (0, 65_536, rows - 9):
        c, s = kq.kq_mxfp4_empty(9, n)
        v = torch.empty((9, n), dtype=torch.bfloat16, device="cuda")
        kq.kq_mxfp4_quantize(x[lo:lo + 9], c, s, d=d, sign=sg, had=had, values=v)
        assert torch.equal(codes[lo:lo + 9], c) and torch.equal(scales[:, lo:lo + 9], s)
        assert torch.equal(values[lo:lo + 9], v)


@pytest.mark.parametrize("rows", [1, 20, 70, 300])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_output_rows_far_apart(rows, kind):
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    x = _rows(rng, rows, 384, "bf16")
    wc, ws, wv = _layer(rng, 150, 384)
    wide = _empty((rows, (1 << 20) + 8), kind)
    xq = om.mx_round(x.double().numpy())
    for path in ({}, dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=256), dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=64)):
        wide.fill_(123.0)
        with _forced(path):
            kq.kq_mxfp4_linear(x.cuda(), wc, ws, wide[:, 3:153])
        _close(wide[:, 3:153], xq, wv, kind == "bf16")
        assert bool((wide[:, :3] == 123.0).all()) and bool((wide[:, 153:] == 123.0).all())


@pytest.mark.parametrize("path", [{}, dict(KQ_TESTING_MX_FEW=0), *PATHS[2:5]], ids=str)
@pytest.mark.parametrize("tokens,top,experts,n,out", [(300, 4, 2000, 128, 70), (40, 2, 1025, 384, 40),
                                                     (4000, 2, 5, 128, 2500), (3000, 1, 1, 640, 1900)])
def test_many_experts_and_tiles(tokens, top, experts, n, out, path):
    """More experts than a table in shared memory holds; more tiles than workgroups, behind an index."""
    announce(f"mxfp4 experts {tokens}x{top} of {experts} {n} -> {out} {path}")
    kq = _kq()
    rng = np.random.default_rng(tokens)
    index, offsets = _sorted_slots(rng, tokens, top, experts, 1.0)
    index = rng.permutation(tokens).astype(np.int32) if top == 1 else index
    x, xs = _random_codes(tokens, n)
    w, ws = _random_codes(out, n, experts)
    y = _empty((tokens * top, out), "f32")
    with _forced(path):
        kq.kq_mxfp4_experts(x, _dev(index), _dev(offsets), w, ws, y, x_scales=xs, n=n)
    xq = _values(x, xs, np.arange(tokens))
    for e in np.flatnonzero(np.diff(offsets)):
        lo, hi = offsets[e], offsets[e + 1]
        _close(y[lo:hi], xq[index[lo:hi]], _values(w[e], ws[e], np.arange(out)), False)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("rows,n,had", [(1, 4096, 4096), (1, 640, 128), (3, 8192, 8192), (40, 1536, 512), (1, 100, 4),
                                        (2, 7, 1)])
def test_operands_at_any_element(rows, n, had, kind):
    """Rows, factors and signs that begin anywhere, rows any distance apart: the same bits."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(n)
    x = _rows(rng, rows, n, kind).cuda()
    d, sg = _processing(rng, n, True, True)
    wc, ws, _ = _layer(rng, 50, n)
    want = (*_quantize(x, d, sg, had), _empty((rows, 50), "f32"))
    kq.kq_mxfp4_linear(x, wc, ws, want[3], d=_dev(d), sign=_dev(sg), had=had)
    for off, pad in ((1, 1), (2, 0), (3, 4), (8, 3)):
        wide = torch.full((rows, off + n + pad), float("nan"), dtype=x.dtype, device="cuda")
        wide[:, off:off + n] = x
        moved_d = torch.cat([torch.full((off,), float("nan")), torch.from_numpy(d)]).cuda()[off:]
        moved_s = torch.cat([torch.zeros(off, dtype=torch.int8), torch.from_numpy(sg)]).cuda()[off:]
        codes, scales = kq.kq_mxfp4_empty(rows, n)
        values = torch.full((rows, off + n + pad), 7.0, dtype=torch.bfloat16, device="cuda")
        kq.kq_mxfp4_quantize(wide[:, off:off + n], codes, scales, d=moved_d, sign=moved_s, had=had,
                             values=values[:, off:off + n])
        code, scale = om.mx_unpack(codes.cpu().numpy(), scales.cpu().numpy())
        assert np.array_equal(code, want[0]) and np.array_equal(scale, want[1])
        assert np.array_equal(values[:, off:off + n].float().cpu().numpy(), want[2])
        assert bool((values[:, :off] == 7).all()) and bool((values[:, off + n:] == 7).all())
        y = _empty((rows, 50), "f32")
        kq.kq_mxfp4_linear(wide[:, off:off + n], wc, ws, y, d=moved_d, sign=moved_s, had=had)
        assert torch.equal(y, want[3])


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,had", [(1024, 4), (512, 8), (512, 16), (512, 64), (768, 256), (1024, 1024), (2048, 2048),
                                   (4096, 4096)])
def test_quantize_near_the_smallest_numbers(n, had, kind):
    """Rows of every magnitude from the smallest subnormal on, and rows with blocks of all of them:
    the products with 1 / sqrt(had) are rounded where they are subnormal, as defined."""
    announce(f"mxfp4 quantize tiny {n} block {had} {kind}")
    torch = torch_cuda()
    rng = np.random.default_rng(had)
    power = np.arange(-149, -100)
    x = np.ldexp(rng.standard_normal((len(power) + 6, n)), np.concatenate([power, [0] * 6])[:, None])
    x[-6:] = np.ldexp(x[-6:], np.repeat(rng.integers(-150, -60, (6, n // 32)), 32, axis=1))
    x = torch.from_numpy(x.astype(np.float32))
    x = x.to(torch.bfloat16) if kind == "bf16" else x
    for d, sg in ((None, None), _processing(rng, n, True, True)):
        code, scale, values = _quantize(x.cuda(), d, sg, had)
        c, s = om.mx_encode(om.mx_rotate_f32(x.float().numpy(), d, sg, had))
        assert np.array_equal(scale, s) and np.array_equal(code, c)
        assert np.array_equal(values, om.mx_values(c, s, n).astype(np.float32))


@pytest.mark.parametrize("tokens", [1, 150])
def test_mixture_example(tokens):
    """The example's block against its products done one by one in 64 bits on the values that the
    codes stand for, and against fp32: the processing has to help where channels are large."""
    torch = torch_cuda()
    import examples.mxfp4_mixture as ex
    torch.manual_seed(tokens)
    x, *weights = ex.make(256 + tokens, 512, 320, 6, seed=tokens)
    calibration, x = x[:256], x[256:]
    want = ex.plain(x, *weights, 2)
    error = {}
    for processed in (False, True):
        block = ex.Mixture(*weights, 2, calibration, processed)
        index, offsets, weight = ex.route(x, weights[3], 2)
        got = block.up.experts(x, index, offsets)
        layers = block.up
        host = lambda v: None if v is None else v.cpu().numpy()  # noqa: E731
        xq = om.mx_round(om.mx_rotate_f32(x.float().cpu().numpy(), host(layers.d), host(layers.sign), layers.had))
        w = np.stack([_values(layers.codes[e], layers.scales[e], np.arange(layers.out)) for e in range(6)])
        ref, mag = _experts_ref(xq, host(index), host(offsets), w, 2 * tokens, tokens)
        _experts_check(got, ref, mag, 512, True)
        error[processed] = float((block(x) - want).norm() / want.norm())
    # four-bit elements are off by up to 1/4 of themselves: 0.1 or so of a product of two of them
    assert error[True] < 0.25 and error[True] < 0.75 * error[False], error


@pytest.mark.parametrize("rows", [64, 500])
def test_default_workspaces_on_given_streams(rows):
    """Calls on two streams of their own, with the workspaces that the binding allocates, while the
    current stream allocates and fills blocks of the same size: the bits of a call by itself."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(rows)
    n, out, experts = 2048, 300, 3
    d, sg = (_dev(v) for v in _processing(rng, n, True, True))
    wc, ws, _ = _layer(rng, out, n)
    ec, es = _random_codes(96, n, experts)
    index, offsets = (_dev(v) for v in _sorted_slots(rng, rows, 2, experts, 1.0))
    inputs = [_rows(rng, rows, n, "bf16").cuda() for _ in range(8)]
    size = kq.kq_mxfp4_workspace(rows, n)
    want = []
    for x in inputs:
        work = torch.empty(size, dtype=torch.uint8, device="cuda")
        y, z = _empty((rows, out), "f32"), _empty((2 * rows, 96), "bf16")
        kq.kq_mxfp4_linear(x, wc, ws, y, work, d=d, sign=sg, had=n)
        kq.kq_mxfp4_experts(x, index, offsets, ec, es, z, work, d=d, sign=sg, had=n)
        want.append((y, z))
    got = [(_empty((rows, out), "f32"), _empty((2 * rows, 96), "bf16")) for _ in inputs]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    filled = []
    for k, x in enumerate(inputs):
        y, z = got[k]
        kq.kq_mxfp4_linear(x, wc, ws, y, d=d, sign=sg, had=n, stream=streams[k % 2])
        filled.append(torch.full((size,), k, dtype=torch.uint8, device="cuda"))
        kq.kq_mxfp4_experts(x, index, offsets, ec, es, z, d=d, sign=sg, had=n, stream=streams[k % 2])
        torch.full((size,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for (y, z), (a, b) in zip(got, want):
        assert torch.equal(y, a) and torch.equal(z, b)
    assert all(bool((f == k).all()) for k, f in enumerate(filled))


def test_experts_of_the_most_rows():
    """2^30 quantised rows, the most there may be, read through an index up to the last one."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(30)
    rows, n, out, slots = 1 << 30, 128, 70, 300
    codes, scales = kq.kq_mxfp4_empty(rows, n)       # 68 GiB, of which the rows below are filled
    index = rng.integers(0, rows, slots).astype(np.int32)
    index[:12] = rows - 1 - np.arange(12)
    index[[20, 250]] = [-1, rows]
    index[200:208] = rows - 1 - np.arange(8)
    inside = (index >= 0) & (index < rows)
    picked = torch.from_numpy(np.unique(index[inside])).long().cuda()
    some, some_scales = _random_codes(len(picked), n)
    codes[picked] = some
    scales[:, picked] = some_scales
    wc, ws, wv = _layer(rng, out, n, 2)
    offsets = np.int32([0, 130, slots])
    xq = np.zeros((slots, n))
    xq[inside] = _values(codes, scales, index[inside])
    want, mag = _experts_ref(xq, None, offsets, wv, slots, slots)
    y = _empty((slots, out), "f32")
    kq.kq_mxfp4_experts(codes, _dev(index), _dev(offsets), wc, ws, y, x_scales=scales, n=n)
    _experts_check(y, want, mag, n, False)
    del codes, scales
    torch.cuda.empty_cache()


@pytest.mark.parametrize("path", [{}, *PATHS[2:]], ids=str)
@pytest.mark.parametrize("kind", ["three times over", "down at the end of 64", "any", "many"])
def test_experts_of_decreasing_offsets(kind, path):
    """An offset below an earlier one counts as that one: every later expert keeps its slots."""
    announce(f"mxfp4 experts, offsets {kind} {path}")
    kq = _kq()
    rng = np.random.default_rng(len(kind))
    slots, n, out = 2000, 128, 20
    if kind == "three times over":
        offsets = np.array([0, 1000, 0, 1000, 0, 1000, 2000])
    elif kind == "down at the end of 64":
        offsets = np.concatenate([np.linspace(0, 1500, 65), np.linspace(900, 2000, 40)]).astype(int)
    else:
        offsets = rng.integers(-500, 2500, 9 if kind == "any" else 1300)
        offsets[-400:] = np.sort(offsets[-400:])
    cut = np.maximum.accumulate(np.clip(offsets, 0, slots))
    experts = len(offsets) - 1
    x, xs = _random_codes(slots, n)
    w, ws = _random_codes(out, n, experts)
    y = _empty((slots, out), "f32")
    with _forced(path):
        kq.kq_mxfp4_experts(x, None, _dev(offsets.astype(np.int32)), w, ws, y, x_scales=xs, n=n)
    xq = _values(x, xs, np.arange(slots))
    for e in np.flatnonzero(np.diff(cut))[::-1]:
        lo, hi = cut[e], cut[e + 1]
        _close(y[lo:hi], xq[lo:hi], _values(w[e], ws[e], np.arange(out)), False)
    outside = np.r_[0:cut[0], cut[-1]:slots]
    assert bool((y[outside] == 123.0).all())


def test_experts_of_offsets_that_swing():
    """2^30 slots, offsets that go up to all of them and down to none 2048 times: the first expert's."""
    torch = torch_cuda()
    kq = _kq()
    slots, rows, n, experts = 1 << 30, 4, 100, 4096
    x, xs = _random_codes(rows, n)
    w, ws = _random_codes(1, n, experts)
    few = _empty((rows, 1), "bf16")
    kq.kq_mxfp4_linear(x, w[0], ws[0], few, x_scales=xs, n=n)
    index = torch.arange(rows, dtype=torch.int32, device="cuda").repeat(slots // rows)
    offsets = torch.tensor([0, slots], dtype=torch.int32, device="cuda").repeat(experts // 2 + 1)[:experts + 1]
    y = _empty((slots, 1), "bf16")
    kq.kq_mxfp4_experts(x, index, offsets.contiguous(), w, ws, y, x_scales=xs, n=n)
    assert bool((y.view(-1, rows) == few.view(1, rows)).all())
    del index, y
    torch.cuda.empty_cache()


def _device_values(codes, scales, rows):
    torch = torch_cuda()
    return torch.from_numpy(_values(codes, scales, rows)).cuda()


def _close_everywhere(y, xq, w, bf16):
    """_close for device operands in 64 bits, every entry."""
    ref, mag = xq @ w.T, xq.abs() @ w.abs().T
    bound = (xq.shape[1] + 2) * 2.0 ** -24 * mag
    if bf16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * ref.abs()
    off = (y.double() - ref).abs() - bound
    assert bool((off <= 0).all()), float(off.max())


TILES = [dict(KQ_TESTING_MX_FEW=0, KQ_TESTING_MX_TILE=t) for t in (256, 128, 64)]


@pytest.mark.parametrize("path", TILES, ids=str)
@pytest.mark.parametrize("n", [1152, 2304])
@pytest.mark.parametrize("yk,indexed", [("bf16", True), ("f32", True), ("bf16", False)])
def test_experts_of_many_tiles_and_rounds(n, yk, indexed, path):
    """Several tiles for every workgroup, each of several rounds of the ring (odd and even numbers of
    128 columns, last rounds with and without stages past the end), behind a shuffled index that
    leaves the rows in places: what runs while one tile follows another."""
    announce(f"mxfp4 experts, many tiles, {n} {yk} {indexed} {path}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(n)
    slots, rows, out, experts = 8000, 4000 if indexed else 8000, 2500, 5
    offsets = np.int32([3, 1900, 1900, 4333, 7990, 7997])
    x, xs = _random_codes(rows, n)
    w, ws = _random_codes(out, n, experts)
    index = rng.integers(0, rows, slots).astype(np.int32)
    index[rng.integers(0, slots, 200)] = rng.choice([-1, rows, -2 ** 31, 2 ** 31 - 1], 200)
    index = index if indexed else None
    y = _empty((slots, out), yk)
    with _forced(path):
        kq.kq_mxfp4_experts(x, _dev(index), _dev(offsets), w, ws, y, x_scales=xs, n=n)
    xq = _device_values(x, xs, np.arange(rows))
    if indexed:
        inside = torch.from_numpy((index >= 0) & (index < rows)).cuda()
        at = torch.from_numpy(np.clip(index, 0, rows - 1)).long().cuda()
        xq = xq[at] * inside[:, None]
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            _close_everywhere(y[lo:hi], xq[lo:hi], _device_values(w[e], ws[e], np.arange(out)), yk == "bf16")
    assert bool((y[:3] == 123.0).all()) and bool((y[7997:] == 123.0).all())


@pytest.mark.parametrize("path", TILES, ids=str)
@pytest.mark.parametrize("rows,n,out,yk", [(5000, 1408, 4200, "bf16"), (5001, 1280, 4199, "f32")])
def test_linear_of_many_tiles_and_rounds(rows, n, out, yk, path):
    announce(f"mxfp4 linear, many tiles, {rows}x{n} -> {out} {yk} {path}")
    kq = _kq()
    x, xs = _random_codes(rows, n)
    w, ws = _random_codes(out, n)
    y = _empty((rows, out), yk)
    with _forced(path):
        kq.kq_mxfp4_linear(x, w, ws, y, x_scales=xs, n=n)
    _close_everywhere(y, _device_values(x, xs, np.arange(rows)), _device_values(w, ws, np.arange(out)), yk == "bf16")


def test_experts_of_rows_past_32_bits_over_many_tiles():
    """Rows of more than 4 GiB behind an index, several tiles for every workgroup."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(12)
    rows, n, slots, out, experts = 1_060_000, 8192, 8000, 2500, 5
    offsets = np.int32([0, 1900, 1900, 4333, 7990, 8000])
    x, xs = _random_codes(rows, n)
    w, ws = _random_codes(out, n, experts)
    index = rng.integers(0, rows, slots).astype(np.int32)
    index[[0, 1, 4332, 4333, 7999]] = [rows - 1, -1, rows - 2, rows, 0]
    y = _empty((slots, out), "bf16")
    kq.kq_mxfp4_experts(x, _dev(index), _dev(offsets), w, ws, y, x_scales=xs, n=n)
    inside = (index >= 0) & (index < rows)
    xq = _device_values(x, xs, np.clip(index, 0, rows - 1)) * torch.from_numpy(inside).cuda()[:, None]
    for e in range(experts):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo < hi:
            _close_everywhere(y[lo:hi], xq[lo:hi], _device_values(w[e], ws[e], np.arange(out)), True)
