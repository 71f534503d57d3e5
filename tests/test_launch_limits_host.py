"""Refusals of sizes with more threads than a launch has (checked before anything touches a GPU)."""
import ctypes

import pytest

import post_quantization_syrk_amd as kq

P = ctypes.c_void_p(0x10000)          # aligned, never dereferenced on the host


@pytest.mark.parametrize("mode,out,n,had_in,had_out", [
    (kq.KQ_BIIP_IN_ONLY, (1 << 22) + 4, 4096, 4, 1), (kq.KQ_BIIP_IN_ONLY, 1 << 23, 4096, 8, 1), (kq.KQ_BIIP_IN_ONLY, 1 << 24, 4096, 1024, 1),
    (kq.KQ_BIIP_IN_ONLY, 1 << 23, 4096, 2048, 1), (kq.KQ_BIIP_IN_ONLY, 4, 1 << 17, 4, 1), (kq.KQ_BIIP_OUT_ONLY, 1 << 17, 4, 1, 4)])
def test_transforms_of_more_blocks_than_threads(mode, out, n, had_in, had_out):
    lib = kq.load_library()
    hg = P if mode != kq.KQ_BIIP_IN_ONLY else None
    st = lib.kq_biip_rotate(P, P, out, n, P, P, hg, hg, P, P, had_in, had_out, 0.25, mode, P, P, None)
    assert st == 2 and b"in blocks of" in lib.kq_last_error()      # KQ_ESHAPE
