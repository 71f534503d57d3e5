"""Workspaces that the binding allocates itself, on the CPU: tensors that claim to be on the
device, a library whose launches only look, and a torch whose allocations note the stream that
was current."""
import contextlib
import gc
import types
import weakref

import pytest
import torch

import post_quantization_syrk_amd as kq

STREAM = types.SimpleNamespace(cuda_stream=0x70)


class OnDevice(torch.Tensor):
    """A host tensor that the binding's checks take for a device tensor."""

    @property
    def is_cuda(self):
        return True


def on_device(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Watched:
    """Stands in for torch and for the library: what was allocated, on which stream, and whether
    it was still held when the library was called."""

    def __init__(self, launch):
        self.allocated = []   # (weak reference, bytes, address, current stream)
        self.current = None
        self.calls = 0
        self.launch = launch
        self.real = kq.load_library()

    # torch
    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *shape, **kw):
        t = torch.empty(*shape, **kw).as_subclass(OnDevice)
        self.allocated.append((weakref.ref(t), t.numel(), t.data_ptr(), self.current))
        return t

    @property
    def cuda(self):
        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before
        return types.SimpleNamespace(stream=stream, current_stream=lambda: types.SimpleNamespace(cuda_stream=0))

    # the library
    def library(self):
        watched = self

        class Library:
            def __getattr__(self, name):
                if name != watched.launch:
                    return getattr(watched.real, name)

                def called(*args):
                    gc.collect()
                    watched.calls += 1
                    values = [getattr(a, "value", a) for a in args]
                    for held, size, address, _ in watched.allocated:
                        assert held() is not None, f"{name}: its workspace was given up before the call"
                        assert address in values and size in values
                    return kq.KQ_OK
                return called
        return Library()


@pytest.fixture
def watch(monkeypatch):
    def start(launch):
        w = Watched(launch)
        if kq._mx_types is None:
            kq._mx_setup()
        monkeypatch.setattr(kq, "_lib", w.library())
        monkeypatch.setattr(kq, "_torch", lambda: w)
        monkeypatch.setattr(kq, "_mx_device", lambda: 0)
        monkeypatch.setattr(kq, "_mx_stream_of", lambda device: 0)
        return w
    return start


def _check(w, calls, stream):
    assert w.calls == calls and len(w.allocated) == calls
    assert all(on is stream for *_, on in w.allocated)   # the pool of the stream that uses it


@pytest.mark.parametrize("stream", [None, STREAM], ids=["current", "given"])
@pytest.mark.parametrize("experts", [False, True])
def test_mxfp4_products_hold_their_workspace(watch, experts, stream):
    w = watch("kq_mxfp4_experts" if experts else "kq_mxfp4_linear")
    x, y = on_device(40, 256), on_device(40, 24)
    lead = (3,) if experts else ()
    codes, scales = on_device(*lead, 24, 128, dtype=torch.uint8), on_device(*lead, 2, 24, 4, dtype=torch.uint8)
    if experts:
        kq.kq_mxfp4_experts(x, None, on_device(4, dtype=torch.int32), codes, scales, y, stream=stream)
    else:
        kq.kq_mxfp4_linear(x, codes, scales, y, stream=stream)
    _check(w, 1, stream)


@pytest.mark.parametrize("stream", [None, STREAM], ids=["current", "given"])
def test_flipflop_takes_its_workspace_from_its_stream(watch, stream):
    w = watch("kq_flipflop")
    x, g = on_device(256, 256, dtype=torch.bfloat16), on_device(256, 128, dtype=torch.bfloat16)
    kq.kq_flipflop(x, g, 1, on_device(256, 256), on_device(128, 128), stream=stream)
    _check(w, 1, stream)


@pytest.mark.parametrize("stream", [None, STREAM], ids=["current", "given"])
def test_two_sided_takes_its_workspace_from_its_stream(watch, stream):
    w = watch("kq_quantize_two_sided")
    params = kq.make_params(bits=4, group=128)
    packed, scales, zeros = on_device(128, 16, dtype=torch.int32), on_device(128, 1), on_device(128, 1, dtype=torch.uint8)
    kq.kq_quantize_two_sided(params, on_device(128, 128), on_device(128, 128), on_device(128, 128), packed, scales,
                             zeros, stream=stream)
    _check(w, 1, stream)
