"""MXFP4 on the CPU: pins of the plain implementation, the held layout, and the host-side
refusals of the MXFP4 entry points (checked before anything touches a GPU)."""
import ctypes

import numpy as np
import pytest

import oracle.mxfp4 as om
import post_quantization_syrk_amd as kq

P = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host
ODD = ctypes.c_void_p(0x10001)


def test_elements_by_hand():
    """One block whose largest magnitude is 6: scale 2^0; every tie goes to the even code."""
    x = np.zeros((1, 32))
    x[0, :16] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -0.75, -5.01, 4.99, 0.26, 0.24, -2.49, 3]
    code, scale = om.mx_encode(x)
    assert scale[0, 0] == 127
    want = [6, 4, 4, 2, 2, 1, 1, 0, 0, -1, -6, 4, 0.5, 0, -2, 3]
    assert np.array_equal(om.mx_values(code, scale, 32)[0, :16], want)


@pytest.mark.parametrize("top,byte", [(8.0, 128), (7.999, 127), (4.0, 127), (3.999, 126), (1.0, 125),
                                      (2.0 ** -125, 0), (2.0 ** -126, 0), (2.0 ** -149, 0), (0.0, 0),
                                      (2.0 ** 127, 252)])
def test_scale_exponents(top, byte):
    x = np.zeros((1, 40))
    x[0, 33] = -top
    code, scale = om.mx_encode(x)
    assert scale[0, 1] == byte and scale[0, 0] == 0
    v = om.mx_values(code, scale, 40)
    assert v[0, 33] == -min(om.MAGNITUDES[-1] * 2.0 ** (byte - 127), top) or abs(v[0, 33] + top) <= 0.125 * top \
        or top < 2.0 ** -127


def test_rounding_against_brute_force():
    """Every fp32 number near the boundaries, and random ones: the chosen element is the nearest."""
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-6, 6, 3200), np.nextafter(np.float32([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5] * 32), 9)])
    x = x[: x.size // 31 * 31].reshape(-1, 31)
    x = np.concatenate([np.full((x.shape[0], 1), 6.0), x], axis=1)
    v = om.mx_round(x)
    best = np.abs(np.abs(x)[..., None] - om.MAGNITUDES).min(-1)
    assert np.array_equal(np.abs(np.abs(x) - np.abs(v)), best)
    assert np.all((v == 0) | (np.sign(v) == np.sign(x)))


def test_not_finite_blocks():
    x = np.ones((2, 96))
    x[0, 40], x[1, 95] = np.inf, np.nan
    code, scale = om.mx_encode(x)
    v = om.mx_values(code, scale, 96)
    assert np.isnan(v[0, 32:64]).all() and np.isfinite(v[0, :32]).all() and np.isfinite(v[0, 64:]).all()
    assert np.isnan(v[1, 64:]).all() and scale[1, 2] == 255 and not code[1, 64:96].any()


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 33), (2, 128), (5, 1000)])
def test_layout_round_trip(rows, n):
    rng = np.random.default_rng(n)
    code, scale = om.mx_encode(rng.standard_normal((rows, n)))
    codes, scales = om.mx_pack(code, scale)
    assert codes.shape == (rows, kq.kq_mxfp4_padded(n) // 2) and scales.shape == (kq.kq_mxfp4_padded(n) // 128, rows, 4)
    c2, s2 = om.mx_unpack(codes, scales)
    assert np.array_equal(code, c2) and np.array_equal(scale, s2)
    r, b = rows - 1, (n - 1) // 32
    assert scales.reshape(-1)[((b // 4) * rows + r) * 4 + b % 4] == scale[r, b]


def test_rotation_in_fp32_is_the_rotation():
    rng = np.random.default_rng(1)
    x, d = rng.standard_normal((3, 768)), np.exp(rng.standard_normal(768)).astype(np.float32)
    s = rng.choice([-1, 1], 768).astype(np.int8)
    a, b = om.mx_rotate(x, d, s, 256), om.mx_rotate_f32(x, d, s, 256)
    # ten roundings of relative 2^-24, in the norm (each stage is orthogonal up to its scale)
    assert np.linalg.norm(a - b) <= 12 * 2.0 ** -24 * np.linalg.norm(a)


def _quantize(**kw):
    a = dict(src=P, type=kq.KQ_F32, rows=4, n=64, ld=64, d=None, sign=None, had=1, codes=P, scales=P, values=None,
             ldv=0)
    a.update(kw)
    return kq.load_library().kq_mxfp4_quantize(a["src"], a["type"], a["rows"], a["n"], a["ld"], a["d"], a["sign"],
                                               a["had"], a["codes"], a["scales"], a["values"], a["ldv"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(src=None), kq.KQ_EINVAL), (dict(codes=None), kq.KQ_EINVAL), (dict(scales=None), kq.KQ_EINVAL),
    (dict(type=2), kq.KQ_EINVAL), (dict(type=-1), kq.KQ_EINVAL), (dict(src=ODD), kq.KQ_EINVAL),
    (dict(src=ODD, type=kq.KQ_BF16), kq.KQ_EINVAL), (dict(codes=ctypes.c_void_p(0x10008)), kq.KQ_EINVAL),
    (dict(scales=ctypes.c_void_p(0x10004)), kq.KQ_EINVAL), (dict(values=ODD, ldv=64), kq.KQ_EINVAL),
    (dict(rows=-1), kq.KQ_ESHAPE), (dict(rows=(1 << 30) + 1), kq.KQ_ESHAPE), (dict(n=0), kq.KQ_ESHAPE),
    (dict(n=(1 << 24) + 1, ld=1 << 25), kq.KQ_ESHAPE), (dict(ld=63), kq.KQ_ESHAPE),
    (dict(values=P, ldv=63), kq.KQ_ESHAPE), (dict(had=-1), kq.KQ_ESHAPE), (dict(had=3), kq.KQ_ESHAPE),
    (dict(had=128), kq.KQ_ESHAPE), (dict(had=16384, n=16384, ld=16384), kq.KQ_ESHAPE),
    (dict(had=0, n=16384, ld=16384), kq.KQ_ENOTIMPL),
])
def test_quantize_refuses(kw, status):
    assert _quantize(**kw) == status
    assert kq.load_library().kq_last_error()


def test_quantize_of_no_rows_is_nothing():
    assert _quantize(rows=0, src=None, codes=None, scales=None) == kq.KQ_OK


def _product(experts=None, **kw):
    a = dict(x=P, type=kq.KQ_BF16, rows=4, n=64, ldx=64, xs=None, d=None, sign=None, had=1, index=P, slots=4,
             offsets=P, wc=P, ws=P, out=16, y=P, ytype=kq.KQ_F32, ldy=16, work=P, bytes=4 * 68)
    a.update(kw)
    lib = kq.load_library()
    x = (a["x"], a["type"], a["rows"], a["n"], a["ldx"], a["xs"], a["d"], a["sign"], a["had"])
    y = (a["wc"], a["ws"], a["out"], a["y"], a["ytype"], a["ldy"], a["work"], a["bytes"], None)
    if experts is None:
        return lib.kq_mxfp4_linear(*x, *y)
    return lib.kq_mxfp4_experts(*x, a["index"], a["slots"], a["offsets"], experts, *y)


REFUSED = [
    (dict(x=None), kq.KQ_EINVAL), (dict(wc=None), kq.KQ_EINVAL), (dict(ws=None), kq.KQ_EINVAL),
    (dict(y=None), kq.KQ_EINVAL), (dict(type=3), kq.KQ_EINVAL), (dict(ytype=2), kq.KQ_EINVAL),
    (dict(xs=P), kq.KQ_EINVAL), (dict(type=kq.KQ_MXFP4, ldx=128), kq.KQ_EINVAL),
    (dict(type=kq.KQ_MXFP4, ldx=64, xs=P), kq.KQ_ESHAPE), (dict(type=kq.KQ_MXFP4, ldx=128, xs=P, d=P), kq.KQ_EINVAL),
    (dict(type=kq.KQ_MXFP4, ldx=128, xs=P, sign=P), kq.KQ_EINVAL),
    (dict(type=kq.KQ_MXFP4, ldx=128, xs=P, had=64), kq.KQ_EINVAL),
    (dict(type=kq.KQ_MXFP4, ldx=128, xs=P, x=ctypes.c_void_p(0x10008)), kq.KQ_EINVAL),
    (dict(wc=ctypes.c_void_p(0x10008)), kq.KQ_EINVAL), (dict(ws=ctypes.c_void_p(0x10004)), kq.KQ_EINVAL),
    (dict(y=ctypes.c_void_p(0x10002)), kq.KQ_EINVAL), (dict(rows=-1), kq.KQ_ESHAPE), (dict(n=0), kq.KQ_ESHAPE),
    (dict(out=0, ldy=0), kq.KQ_ESHAPE), (dict(out=(1 << 24) + 1, ldy=1 << 25), kq.KQ_ESHAPE),
    (dict(ldx=63), kq.KQ_ESHAPE), (dict(ldy=15), kq.KQ_ESHAPE), (dict(had=48), kq.KQ_ESHAPE),
    (dict(work=None), kq.KQ_EWORKSPACE), (dict(bytes=4 * 68 - 1), kq.KQ_EWORKSPACE),
    (dict(work=ctypes.c_void_p(0x10008)), kq.KQ_EWORKSPACE),
]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_linear_refuses(kw, status):
    assert _product(**kw) == status


@pytest.mark.parametrize("kw,status", REFUSED + [
    (dict(experts=0), kq.KQ_ESHAPE), (dict(experts=4097), kq.KQ_ESHAPE), (dict(slots=-1), kq.KQ_ESHAPE),
    (dict(offsets=None), kq.KQ_EINVAL), (dict(offsets=ctypes.c_void_p(0x10002)), kq.KQ_EINVAL),
    (dict(index=ctypes.c_void_p(0x10002)), kq.KQ_EINVAL), (dict(index=None, slots=5), kq.KQ_ESHAPE),
])
def test_experts_refuses(kw, status):
    assert _product(**{"experts": 2, **kw}) == status


def test_products_of_nothing():
    assert _product(rows=0, x=None, y=None, work=None, bytes=0) == kq.KQ_OK
    assert _product(experts=2, slots=0, y=None) == kq.KQ_OK


def test_workspace():
    assert kq.kq_mxfp4_workspace(3, 129) == 3 * 2 * 68
    assert kq.kq_mxfp4_workspace(0, 5) == 0
    for rows, n in ((-1, 4), (1, 0)):
        with pytest.raises(kq.KQError) as e:
            kq.kq_mxfp4_workspace(rows, n)
        assert e.value.status == kq.KQ_ESHAPE
    assert kq.load_library().kq_mxfp4_workspace(1, 1, None) == kq.KQ_EINVAL
