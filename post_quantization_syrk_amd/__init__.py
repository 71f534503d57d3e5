"""Python binding of libkq, the KronQ per-layer quantization engine for MI355X.

Thin ctypes marshalling over the C ABI declared in include/kq.h: each
function takes PyTorch tensors (device memory) or numpy arrays (host memory),
checks dtypes, devices and sizes, and passes raw pointers and the current HIP
stream.  Every step of the computation runs in the library's HIP kernels; this
module computes nothing itself and has no fallback: if libkq.so is missing or
fails to load, importing the engine raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkq.so")

KQ_OK, KQ_EINVAL, KQ_ESHAPE, KQ_ENOTSPD, KQ_EWORKSPACE, KQ_ENOTIMPL, KQ_EHIP = range(7)
KQ_BIIP_FULL, KQ_BIIP_NO_RESCALE, KQ_BIIP_IN_ONLY, KQ_BIIP_OUT_ONLY = range(4)
KQ_F32, KQ_BF16, KQ_MXFP4 = range(3)
STATUS_NAMES = {0: "KQ_OK", 1: "KQ_EINVAL", 2: "KQ_ESHAPE", 3: "KQ_ENOTSPD", 4: "KQ_EWORKSPACE",
                5: "KQ_ENOTIMPL", 6: "KQ_EHIP"}

EXPORTED = ("kq_version", "kq_last_error", "kq_accumulate_hessian", "kq_sensitivity",
            "kq_sensitivity_async",
            "kq_biip_rotate", "kq_quantize_layer_workspace", "kq_quantize_layer",
            "kq_quantize_layer_noalloc", "kq_quantize_layer_async",
            "kq_allocate_bits", "kq_deploy_linear", "kq_deploy_linear_group",
            "kq_flipflop_workspace", "kq_flipflop", "kq_quantize_two_sided_workspace",
            "kq_quantize_two_sided", "kq_mxfp4_quantize", "kq_mxfp4_workspace", "kq_mxfp4_linear",
            "kq_mxfp4_experts", "kq_testing_select")


class KQError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn} -> {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class NotSPDError(KQError):
    pass


class DeployLayer(ctypes.Structure):
    """kq_deploy_layer (include/kq.h)."""
    _fields_ = [("packed", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("zeros", ctypes.c_void_p),
                ("bits", ctypes.c_int), ("group", ctypes.c_int), ("out", ctypes.c_int64),
                ("d_in", ctypes.c_void_p), ("d_out", ctypes.c_void_p), ("sign_in", ctypes.c_void_p),
                ("sign_out", ctypes.c_void_p), ("had_in", ctypes.c_int64), ("had_out", ctypes.c_int64),
                ("y", ctypes.c_void_p)]


class QuantParams(ctypes.Structure):
    _fields_ = [("bits", ctypes.c_int), ("group", ctypes.c_int), ("block", ctypes.c_int),
                ("damp", ctypes.c_float), ("asym", ctypes.c_int), ("act_order", ctypes.c_int),
                ("w_clip", ctypes.c_int)]


_vp, _i64, _int, _f32, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "kq_version": ([], ctypes.c_int),
    "kq_last_error": ([], ctypes.c_char_p),
    "kq_accumulate_hessian": ([_vp, _i64, _i64, _i64, _vp, _i64, _int, _vp], _int),
    "kq_sensitivity": ([_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp], _int),
    "kq_sensitivity_async": ([_vp, _i64, _i64, _vp, _i64, _i64, _vp, _vp], _int),
    "kq_biip_rotate": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _f32, _int,
                        _vp, _vp, _vp], _int),
    "kq_quantize_layer_workspace": ([ctypes.POINTER(QuantParams), _i64, _i64, _int,
                                     ctypes.POINTER(_sz)], _int),
    "kq_quantize_layer": ([ctypes.POINTER(QuantParams), _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                           _vp, _vp, _sz, _vp], _int),
    "kq_quantize_layer_async": ([ctypes.POINTER(QuantParams), _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                 _vp, _vp, _vp, _vp, _vp, _sz, _vp], _int),
    "kq_quantize_layer_noalloc": ([ctypes.POINTER(QuantParams), _vp, _vp, _vp, _i64, _i64, _vp, _vp,
                                   _vp, _vp, _vp, _vp], _int),
    "kq_allocate_bits": ([_vp, _vp, _i64, _vp, _int, _i64, _i64, _vp], _int),
    "kq_deploy_linear": ([_vp, _vp, _vp, _int, _int, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64,
                          _vp, _vp, _vp], _int),
    "kq_deploy_linear_group": ([ctypes.POINTER(DeployLayer), _int, _i64, _vp, _vp], _int),
    "kq_flipflop_workspace": ([_i64, _i64, _i64, ctypes.POINTER(_sz)], _int),
    "kq_quantize_two_sided_workspace": ([ctypes.POINTER(QuantParams), _i64, _i64, ctypes.POINTER(_sz)], _int),
    "kq_quantize_two_sided": ([ctypes.POINTER(QuantParams), _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp,
                               _sz, _vp, _vp], _int),
    "kq_flipflop": ([_vp, _i64, _vp, _i64, _i64, _i64, _i64, _int, _vp, _vp, _vp, _sz,
                     ctypes.POINTER(ctypes.c_double), _vp], _int),
    "kq_mxfp4_quantize": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _i64, _vp], _int),
    "kq_mxfp4_workspace": ([_i64, _i64, ctypes.POINTER(_sz)], _int),
    "kq_mxfp4_linear": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _vp, _i64, _vp, _int, _i64,
                         _vp, _sz, _vp], _int),
    "kq_mxfp4_experts": ([_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _i64, _vp, _i64, _vp, _int, _vp, _vp,
                          _i64, _vp, _int, _i64, _vp, _sz, _vp], _int),
    "kq_testing_select": ([_int, _i64], _int),
}

# include/kq_testing.h: implementation selection for tests
(KQ_TESTING_SYRK_KERNEL, KQ_TESTING_FACTOR_SUPERBLOCK, KQ_TESTING_ROW_LDS_BYTES,
 KQ_TESTING_MX_TILE, KQ_TESTING_MX_FEW, KQ_TESTING_MX_FUSED) = range(6)

_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libkq.so (raises OSError/ImportError if it is missing)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(p)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    if path is None:
        _lib = lib
    return lib


class testing_select:
    """Context manager over kq_testing_select: forces one implementation path for the calls
    made inside the block, then restores the default."""

    def __init__(self, knob: int, value: int):
        self.knob, self.value = knob, value

    def __enter__(self):
        _check(load_library().kq_testing_select(self.knob, self.value), "kq_testing_select")
        return self

    def __exit__(self, *exc):
        _check(load_library().kq_testing_select(self.knob, -1), "kq_testing_select")
        return False


def _check(status: int, fn: str) -> None:
    if status != KQ_OK:
        msg = _lib.kq_last_error().decode(errors="replace")
        if status == KQ_ENOTSPD:
            raise NotSPDError(status, fn, msg)
        raise KQError(status, fn, msg)


def _torch():
    import torch
    return torch


def _dev_ptr(t, name: str, dtypes=None, allow_none: bool = False):
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a device (cuda/hip) tensor")
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _workspace(nbytes: int, device, stream):
    """Uninitialised device bytes for work on `stream` (None: the current one), from that stream's
    own pool: whoever had them before, and whoever gets them next, is ordered on the same stream.
    The caller holds them until the work has been enqueued."""
    torch = _torch()
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _ld(t, name: str) -> int:
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return t.stride(0)


def version() -> int:
    return load_library().kq_version()


def kq_accumulate_hessian(A, H, accumulate: bool = False, stream=None) -> None:
    """H = A^T A (or H += A^T A): A bf16 [T x n] (token-major), H fp32 [n x n]."""
    torch = _torch()
    lib = load_library()
    T, n = A.shape
    if H.shape != (n, n):
        raise ValueError("H must be n x n")
    st = lib.kq_accumulate_hessian(_dev_ptr(A, "A", (torch.bfloat16, torch.int16, torch.uint16)),
                                   T, n, _ld(A, "A"), _dev_ptr(H, "H", (torch.float32,)), _ld(H, "H"),
                                   1 if accumulate else 0, _stream(stream))
    _check(st, "kq_accumulate_hessian")


def kq_sensitivity(HX, HG, stream=None) -> tuple[float, float, float]:
    """(tr H_X, tr H_G, tr H_G * tr H_X); synchronizes the stream."""
    torch = _torch()
    lib = load_library()
    out = (ctypes.c_double * 3)()
    st = lib.kq_sensitivity(_dev_ptr(HX, "HX", (torch.float32,)), HX.shape[0], _ld(HX, "HX"),
                            _dev_ptr(HG, "HG", (torch.float32,)), HG.shape[0], _ld(HG, "HG"),
                            ctypes.cast(out, ctypes.c_void_p), _stream(stream))
    _check(st, "kq_sensitivity")
    return out[0], out[1], out[2]


def kq_sensitivity_async(HX, HG, out, stream=None) -> None:
    """Traces and sensitivity into `out` (device float64, 3 entries); does not synchronize."""
    torch = _torch()
    lib = load_library()
    if out.numel() < 3:
        raise ValueError("kq_sensitivity_async: out needs 3 entries")
    st = lib.kq_sensitivity_async(_dev_ptr(HX, "HX", (torch.float32,)), HX.shape[0], _ld(HX, "HX"),
                                  _dev_ptr(HG, "HG", (torch.float32,)), HG.shape[0], _ld(HG, "HG"),
                                  _dev_ptr(out, "out", (torch.float64,)), _stream(stream))
    _check(st, "kq_sensitivity_async")


def kq_biip_rotate(W_src, W_dst, HX_src, HX_dst, HG_src, HG_dst, sign_in, sign_out, d_in, d_out,
                   alpha: float = 0.25, mode: int = KQ_BIIP_FULL, had_block_in: int = 0,
                   had_block_out: int = 0, stream=None) -> None:
    """Bidirectional incoherence processing (rescale + randomized Hadamard, both sides)."""
    torch = _torch()
    lib = load_library()
    out_n, in_n = W_src.shape
    f32 = (torch.float32,)
    i8 = (torch.int8,)
    st = lib.kq_biip_rotate(
        _dev_ptr(W_src, "W_src", f32), _dev_ptr(W_dst, "W_dst", f32), out_n, in_n,
        _dev_ptr(HX_src, "HX_src", f32), _dev_ptr(HX_dst, "HX_dst", f32),
        _dev_ptr(HG_src, "HG_src", f32, True), _dev_ptr(HG_dst, "HG_dst", f32, True),
        _dev_ptr(sign_in, "sign_in", i8, True), _dev_ptr(sign_out, "sign_out", i8, True),
        had_block_in, had_block_out, alpha, mode, _dev_ptr(d_in, "d_in", f32),
        _dev_ptr(d_out, "d_out", f32), _stream(stream))
    _check(st, "kq_biip_rotate")


def make_params(bits: int = 2, group: int = 128, block: int = 128, damp: float = 0.01,
                asym: int = 1, act_order: int = 0, w_clip: int = 0) -> QuantParams:
    return QuantParams(bits, group, block, damp, asym, act_order, w_clip)


def kq_quantize_layer_workspace(p: QuantParams, out_n: int, in_n: int, with_loss: bool) -> int:
    lib = load_library()
    sz = ctypes.c_size_t(0)
    st = lib.kq_quantize_layer_workspace(ctypes.byref(p), out_n, in_n, 1 if with_loss else 0,
                                         ctypes.byref(sz))
    _check(st, "kq_quantize_layer_workspace")
    return sz.value


def kq_quantize_layer(p: QuantParams, W_rot, HX_rot, HG_rot, packed, scales, zeros, ws,
                      codes=None, want_loss: bool = False, stream=None):
    """GPTQ to packed codes; returns (loss_direct, loss_pred) if want_loss else None."""
    torch = _torch()
    lib = load_library()
    out_n, in_n = W_rot.shape
    loss = (ctypes.c_double * 2)() if want_loss else None
    st = lib.kq_quantize_layer(
        ctypes.byref(p), _dev_ptr(W_rot, "W_rot", (torch.float32,)),
        _dev_ptr(HX_rot, "HX_rot", (torch.float32,)),
        _dev_ptr(HG_rot, "HG_rot", (torch.float32,), True), out_n, in_n,
        _dev_ptr(packed, "packed", (torch.int32, torch.uint32)),
        _dev_ptr(scales, "scales", (torch.float32,)), _dev_ptr(zeros, "zeros", (torch.uint8,)),
        _dev_ptr(codes, "codes", (torch.uint8,), True),
        ctypes.cast(loss, ctypes.c_void_p) if loss is not None else None,
        _dev_ptr(ws, "ws", (torch.uint8,)), ws.numel(), _stream(stream))
    _check(st, "kq_quantize_layer")
    return (loss[0], loss[1]) if want_loss else None


def kq_quantize_layer_async(p: QuantParams, W_rot, HX_rot, HG_rot, packed, scales, zeros, ws,
                            status, codes=None, loss=None, stream=None) -> None:
    """kq_quantize_layer without waiting: `status` (device int32, 1 entry) receives KQ_OK or
    KQ_ENOTSPD and `loss` (device float64, 2 entries, optional) the two losses, when the work
    has run."""
    torch = _torch()
    lib = load_library()
    out_n, in_n = W_rot.shape
    st = lib.kq_quantize_layer_async(
        ctypes.byref(p), _dev_ptr(W_rot, "W_rot", (torch.float32,)),
        _dev_ptr(HX_rot, "HX_rot", (torch.float32,)),
        _dev_ptr(HG_rot, "HG_rot", (torch.float32,), True), out_n, in_n,
        _dev_ptr(packed, "packed", (torch.int32, torch.uint32)),
        _dev_ptr(scales, "scales", (torch.float32,)), _dev_ptr(zeros, "zeros", (torch.uint8,)),
        _dev_ptr(codes, "codes", (torch.uint8,), True), _dev_ptr(loss, "loss", (torch.float64,), True),
        _dev_ptr(status, "status", (torch.int32,)), _dev_ptr(ws, "ws", (torch.uint8,)), ws.numel(),
        _stream(stream))
    _check(st, "kq_quantize_layer_async")


KQ_NOALLOC_WORKSPACE_BYTES = 64 << 20


def kq_quantize_layer_noalloc(p: QuantParams, W_rot, HX_rot, HG_rot, packed, scales, zeros,
                              codes=None, want_loss: bool = False, stream=None):
    """kq_quantize_layer on the library's fixed per-GPU workspace (no allocation); returns
    (loss_direct, loss_pred) if want_loss else None."""
    torch = _torch()
    lib = load_library()
    out_n, in_n = W_rot.shape
    loss = (ctypes.c_double * 2)() if want_loss else None
    st = lib.kq_quantize_layer_noalloc(
        ctypes.byref(p), _dev_ptr(W_rot, "W_rot", (torch.float32,)),
        _dev_ptr(HX_rot, "HX_rot", (torch.float32,)),
        _dev_ptr(HG_rot, "HG_rot", (torch.float32,), True), out_n, in_n,
        _dev_ptr(packed, "packed", (torch.int32, torch.uint32)),
        _dev_ptr(scales, "scales", (torch.float32,)), _dev_ptr(zeros, "zeros", (torch.uint8,)),
        _dev_ptr(codes, "codes", (torch.uint8,), True),
        ctypes.cast(loss, ctypes.c_void_p) if loss is not None else None, _stream(stream))
    _check(st, "kq_quantize_layer_noalloc")
    return (loss[0], loss[1]) if want_loss else None


def kq_allocate_bits(sens, numel, allowed=(2, 3, 4), target_num: int = 5, target_den: int = 2):
    """Per-sublayer bit widths (host computation inside the library)."""
    lib = load_library()
    s = np.ascontiguousarray(sens, dtype=np.float64)
    n = np.ascontiguousarray(numel, dtype=np.int64)
    a = np.ascontiguousarray(allowed, dtype=np.int32)
    if s.shape != n.shape or s.ndim != 1:
        raise ValueError("sens and numel must be 1-D of equal length")
    out = np.zeros(s.shape[0], dtype=np.int32)
    st = lib.kq_allocate_bits(s.ctypes.data_as(ctypes.c_void_p), n.ctypes.data_as(ctypes.c_void_p),
                              s.shape[0], a.ctypes.data_as(ctypes.c_void_p), a.shape[0], target_num,
                              target_den, out.ctypes.data_as(ctypes.c_void_p))
    _check(st, "kq_allocate_bits")
    return out.tolist()


def kq_deploy_linear(packed, scales, zeros, bits: int, group: int, d_in, d_out, sign_in, sign_out,
                     had_in: int, had_out: int, x, y, stream=None) -> None:
    """y = D_out^-1 P_out^T Qhat P_in D_in^-1 x for one quantized layer (batch 1)."""
    torch = _torch()
    lib = load_library()
    out_n = packed.shape[0]
    in_n = x.shape[-1]
    st = lib.kq_deploy_linear(
        _dev_ptr(packed, "packed", (torch.int32, torch.uint32)),
        _dev_ptr(scales, "scales", (torch.float32,)), _dev_ptr(zeros, "zeros", (torch.uint8,)),
        bits, group, out_n, in_n,
        _dev_ptr(d_in, "d_in", (torch.float32,), True), _dev_ptr(d_out, "d_out", (torch.float32,), True),
        _dev_ptr(sign_in, "sign_in", (torch.int8,), True),
        _dev_ptr(sign_out, "sign_out", (torch.int8,), True), had_in, had_out,
        _dev_ptr(x, "x", (torch.float32,)), _dev_ptr(y, "y", (torch.float32,)), _stream(stream))
    _check(st, "kq_deploy_linear")


def kq_deploy_linear_group(layers, x, stream=None) -> None:
    """kq_deploy_linear for several layers reading the same x, in one launch.

    layers: sequence of dicts with the keyword arguments of kq_deploy_linear other than x
    (packed, scales, zeros, bits, group, d_in, d_out, sign_in, sign_out, had_in, had_out, y)."""
    torch = _torch()
    lib = load_library()
    arr = (DeployLayer * max(1, len(layers)))()
    for i, L in enumerate(layers):
        arr[i] = DeployLayer(
            _dev_ptr(L["packed"], "packed", (torch.int32, torch.uint32)),
            _dev_ptr(L["scales"], "scales", (torch.float32,)),
            _dev_ptr(L["zeros"], "zeros", (torch.uint8,)), L["bits"], L["group"], L["packed"].shape[0],
            _dev_ptr(L.get("d_in"), "d_in", (torch.float32,), True),
            _dev_ptr(L.get("d_out"), "d_out", (torch.float32,), True),
            _dev_ptr(L.get("sign_in"), "sign_in", (torch.int8,), True),
            _dev_ptr(L.get("sign_out"), "sign_out", (torch.int8,), True),
            L.get("had_in", 0), L.get("had_out", 0), _dev_ptr(L["y"], "y", (torch.float32,)))
    st = lib.kq_deploy_linear_group(arr, len(layers), x.shape[-1], _dev_ptr(x, "x", (torch.float32,)),
                                    _stream(stream))
    _check(st, "kq_deploy_linear_group")


def kq_flipflop_workspace(T: int, n: int, m: int) -> int:
    lib = load_library()
    b = ctypes.c_size_t(0)
    _check(lib.kq_flipflop_workspace(T, n, m, ctypes.byref(b)), "kq_flipflop_workspace")
    return b.value


def kq_flipflop(X, G, iters: int, A, B, ws=None, stream=None, phases: bool = False):
    """FlipFlop factors A (n x n) and B (m x m) from bf16 streams X (T x n) and G (T x m),
    given as int16/uint16/bfloat16 tensors of bit patterns, after `iters` iterations.
    With phases=True, returns the summed HIP-event milliseconds of {factor, quadratic
    forms, scaling, syrk}."""
    torch = _torch()
    lib = load_library()
    T, n = X.shape
    m = G.shape[1]
    if G.shape[0] != T:
        raise ValueError("X and G need the same token count")
    if ws is None:
        ws = _workspace(kq_flipflop_workspace(T, n, m), X.device, stream)
    bf = (torch.int16, torch.uint16, torch.bfloat16)
    ph = (ctypes.c_double * 4)() if phases else None
    st = lib.kq_flipflop(_dev_ptr(X, "X", bf), _ld(X, "X"), _dev_ptr(G, "G", bf), _ld(G, "G"), T, n, m,
                         iters, _dev_ptr(A, "A", (torch.float32,)), _dev_ptr(B, "B", (torch.float32,)),
                         _dev_ptr(ws, "ws", (torch.uint8,)), ws.numel(), ph, _stream(stream))
    _check(st, "kq_flipflop")
    if phases:
        return dict(zip(("factor", "quadratic_forms", "scale", "syrk"), list(ph)))
    return None


def kq_quantize_two_sided_workspace(p: QuantParams, out_n: int, in_n: int) -> int:
    lib = load_library()
    b = ctypes.c_size_t(0)
    _check(lib.kq_quantize_two_sided_workspace(ctypes.byref(p), out_n, in_n, ctypes.byref(b)),
           "kq_quantize_two_sided_workspace")
    return b.value


def kq_quantize_two_sided(p: QuantParams, W, HX, HG, packed, scales, zeros, ws=None, codes=None,
                          stream=None) -> None:
    """Two-sided rounding of W (out x in) under H_X (x) H_G into packed codes, scales and
    zero points (the layout of kq_quantize_layer)."""
    torch = _torch()
    lib = load_library()
    out_n, in_n = W.shape
    if ws is None:
        ws = _workspace(kq_quantize_two_sided_workspace(p, out_n, in_n), W.device, stream)
    f32 = (torch.float32,)
    st = lib.kq_quantize_two_sided(
        ctypes.byref(p), _dev_ptr(W, "W", f32), _dev_ptr(HX, "HX", f32), _dev_ptr(HG, "HG", f32),
        out_n, in_n, _dev_ptr(packed, "packed", (torch.int32, torch.uint32)),
        _dev_ptr(scales, "scales", f32), _dev_ptr(zeros, "zeros", (torch.uint8,)),
        _dev_ptr(ws, "ws", (torch.uint8,)), ws.numel(), _dev_ptr(codes, "codes", (torch.uint8,), True),
        _stream(stream))
    _check(st, "kq_quantize_two_sided")


def kq_mxfp4_padded(n: int) -> int:
    """Columns of a quantised row of n values: n rounded up to a multiple of 128."""
    return -(-n // 128) * 128


def kq_mxfp4_empty(rows: int, n: int, experts: int | None = None, device="cuda"):
    """Uninitialised (codes, scales) for `rows` quantised rows of n values: codes uint8
    [rows, np / 2], scales uint8 [np / 128, rows, 4], np = kq_mxfp4_padded(n); with `experts`,
    that many of each, one after another."""
    torch = _torch()
    lead = () if experts is None else (experts,)
    np_ = kq_mxfp4_padded(n)
    return (torch.empty((*lead, rows, np_ // 2), dtype=torch.uint8, device=device),
            torch.empty((*lead, np_ // 128, rows, 4), dtype=torch.uint8, device=device))


# One token's call takes no longer on the GPU than these checks take here, so they read each tensor's
# properties once and pass plain integers.
_mx_types = None   # tensor type -> KQ_*, and the types below, once torch is imported
_mx_f32 = _mx_bf16 = _mx_u8 = _mx_i8 = _mx_i32 = None
_mx_stream_of = _mx_device = None


def _mx_setup() -> None:
    global _mx_types, _mx_f32, _mx_bf16, _mx_u8, _mx_i8, _mx_i32, _mx_stream_of, _mx_device
    torch = _torch()
    _mx_f32, _mx_bf16, _mx_u8, _mx_i8, _mx_i32 = (torch.float32, torch.bfloat16, torch.uint8, torch.int8, torch.int32)
    _mx_stream_of, _mx_device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
    _mx_types = {_mx_f32: KQ_F32, _mx_bf16: KQ_BF16}
    load_library()


def _mx_ptr(t, name: str, dtype) -> int:
    try:
        if t.dtype is dtype and t.is_cuda:
            return t.data_ptr()
        kind = f"{t.dtype} on {t.device}"
    except AttributeError:
        kind = type(t).__name__
    raise TypeError(f"{name} must be a device (cuda/hip) tensor of {dtype}, not {kind}")


def _mx_matrix(t, name: str):
    """(pointer, KQ_* type, rows, columns, leading dimension) of an fp32 or bf16 matrix."""
    try:
        kind = _mx_types.get(t.dtype)
        if kind is None or not t.is_cuda:
            raise TypeError(f"{name} must be a device (cuda/hip) tensor of float32 or bfloat16, not {t.dtype} on {t.device}")
        rows, cols = t.shape
        ld, step = t.stride()
    except AttributeError:
        raise TypeError(f"{name} must be a device (cuda/hip) tensor, not {type(t).__name__}") from None
    except ValueError:
        raise ValueError(f"{name} must be a matrix, not {tuple(t.shape)}") from None
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have unit column stride")
    return t.data_ptr(), kind, rows, cols, ld if rows > 1 else cols


def _mx_vector(v, name: str, n: int, dtype):
    if v is None:
        return None
    p = _mx_ptr(v, name, dtype)
    if v.numel() != n or not v.is_contiguous():
        raise ValueError(f"{name} must hold {n} contiguous entries")
    return p


def _mx_check(codes, scales, shape: tuple, n: int, name: str):
    cp, sp, groups = _mx_ptr(codes, f"{name} codes", _mx_u8), _mx_ptr(scales, f"{name} scales", _mx_u8), -(-n // 128)
    if codes.shape != (*shape, 64 * groups) or not codes.is_contiguous():
        raise ValueError(f"{name} codes must be contiguous {(*shape, 64 * groups)}")
    if scales.shape != (*shape[:-1], groups, shape[-1], 4) or not scales.is_contiguous():
        raise ValueError(f"{name} scales must be contiguous {(*shape[:-1], groups, shape[-1], 4)}")
    return cp, sp


def kq_mxfp4_quantize(src, codes, scales, d=None, sign=None, had: int = 1, values=None, stream=None) -> None:
    """Rows of src (fp32 or bf16, rows x n) to MXFP4 codes and scales (kq_mxfp4_empty) of
    P D^-1 src; `values` (bf16, rows x n, optional) receives what they stand for."""
    if _mx_types is None:
        _mx_setup()
    xp, xt, rows, n, ld = _mx_matrix(src, "src")
    cp, sp = _mx_check(codes, scales, (rows,), n, "output")
    vp, ldv = None, 0
    if values is not None:
        vp, vt, vrows, vcols, ldv = _mx_matrix(values, "values")
        if vt != KQ_BF16:
            raise TypeError("values must be bfloat16")
        if vrows != rows or vcols != n:
            raise ValueError("values must have src's shape")
    st = _lib.kq_mxfp4_quantize(xp, xt, rows, n, ld, _mx_vector(d, "d", n, _mx_f32),
                                _mx_vector(sign, "sign", n, _mx_i8), had, cp, sp, vp, ldv,
                                _mx_stream_of(_mx_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "kq_mxfp4_quantize")


def kq_mxfp4_workspace(rows: int, n: int) -> int:
    """Workspace bytes of kq_mxfp4_linear and kq_mxfp4_experts for `rows` rows of n activations."""
    lib = load_library()
    b = ctypes.c_size_t(0)
    _check(lib.kq_mxfp4_workspace(rows, n, ctypes.byref(b)), "kq_mxfp4_workspace")
    return b.value


def _mx_rows(x, x_scales, d, sign, n, ws, stream):
    """(pointer, type, rows, n, ld, scales, d, sign, ws, ws bytes) of the activations, and the workspace
    itself, which the caller holds until the call has returned."""
    if _mx_types is None:
        _mx_setup()
    if x_scales is not None:
        if n is None:
            raise ValueError("quantised rows need n, their number of values")
        if d is not None or sign is not None:
            raise ValueError("quantised rows take no rescale and no signs")
        xp, sp = _mx_check(x, x_scales, (x.shape[0],), n, "x")
        return xp, KQ_MXFP4, x.shape[0], n, kq_mxfp4_padded(n), sp, None, None, None, 0, None
    xp, xt, rows, cols, ld = _mx_matrix(x, "x")
    if n is not None and n != cols:
        raise ValueError(f"x has {cols} columns, not {n}")
    if ws is None:
        ws = _workspace(kq_mxfp4_workspace(rows, cols), x.device, stream)
    return (xp, xt, rows, cols, ld, None, _mx_vector(d, "d", cols, _mx_f32), _mx_vector(sign, "sign", cols, _mx_i8),
            _mx_ptr(ws, "ws", _mx_u8), ws.numel(), ws)


def kq_mxfp4_linear(x, w_codes, w_scales, y, ws=None, d=None, sign=None, had: int = 1, x_scales=None,
                    n=None, stream=None) -> None:
    """y = Q(P D^-1 x) W^T for a layer held in MXFP4: x fp32 or bf16 [rows, n] (or codes, with
    x_scales and n), y fp32 or bf16 [rows, out]."""
    xp, xt, rows, n, ldx, xsp, dp, gp, wp, wb, ws = _mx_rows(x, x_scales, d, sign, n, ws, stream)
    out = w_codes.shape[0]
    cp, sp = _mx_check(w_codes, w_scales, (out,), n, "weight")
    yp, yt, yrows, ycols, ldy = _mx_matrix(y, "y")
    if yrows != rows or ycols != out:
        raise ValueError(f"y must be {(rows, out)}")
    st = _lib.kq_mxfp4_linear(xp, xt, rows, n, ldx, xsp, dp, gp, had, cp, sp, out, yp, yt, ldy, wp, wb,
                              _mx_stream_of(_mx_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "kq_mxfp4_linear")


def kq_mxfp4_experts(x, index, offsets, w_codes, w_scales, y, ws=None, d=None, sign=None, had: int = 1,
                     x_scales=None, n=None, stream=None) -> None:
    """y[s] = Q(P D^-1 x[index[s]]) W_e^T for the slots s of expert e, [offsets[e], offsets[e + 1]):
    index int32 [slots] or None, offsets int32 [experts + 1], weights of kq_mxfp4_empty(out, n,
    experts), y fp32 or bf16 [slots, out].  Offsets and index stay on the device."""
    xp, xt, rows, n, ldx, xsp, dp, gp, wp, wb, ws = _mx_rows(x, x_scales, d, sign, n, ws, stream)
    experts, out = w_codes.shape[0], w_codes.shape[1]
    cp, sp = _mx_check(w_codes, w_scales, (experts, out), n, "weight")
    yp, yt, slots, ycols, ldy = _mx_matrix(y, "y")
    if ycols != out:
        raise ValueError(f"y must have {out} columns")
    st = _lib.kq_mxfp4_experts(xp, xt, rows, n, ldx, xsp, dp, gp, had, _mx_vector(index, "index", slots, _mx_i32), slots,
                               _mx_vector(offsets, "offsets", experts + 1, _mx_i32), experts, cp, sp, out, yp, yt, ldy,
                               wp, wb, _mx_stream_of(_mx_device()) if stream is None else stream.cuda_stream)
    if st:
        _check(st, "kq_mxfp4_experts")
