"""Sizes of the per-layer steps that have more elements or tokens than one launch has threads (2^32)."""
import numpy as np
import pytest

from tests.gpu_util import announce, torch_cuda

pytestmark = pytest.mark.gpu


def _kq():
    import post_quantization_syrk_amd as kq
    return kq


def test_flipflop_of_more_tokens_than_threads_of_256():
    """2^24 tokens and a few, of which the first 512 and the last 512 are not zero: the factors of those, but
    for the mean over all.  Tolerance: the factors' 1e-3 (test_gpu_flipflop.py)."""
    announce("flipflop T = 2^24 + 100")
    torch = torch_cuda()
    kq = _kq()
    T, k = (1 << 24) + 100, 128
    gen = torch.Generator(device="cuda").manual_seed(4)
    X, G = (torch.zeros((T, k), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    some = torch.cat((torch.arange(512), torch.arange(T - 512, T))).cuda()
    for s in (X, G):
        s[some] = torch.randn(1024, k, generator=gen, device="cuda").to(torch.bfloat16)
    A, B = torch.empty((k, k), device="cuda"), torch.empty((k, k), device="cuda")
    kq.kq_flipflop(X, G, 1, A, B)
    x, g = X[some].double().cpu().numpy(), G[some].double().cpu().numpy()
    want = (x * (g * g).sum(1, keepdims=True)).T @ x / (T * k)
    assert np.linalg.norm(A.double().cpu().numpy() - want) <= 1e-3 * np.linalg.norm(want)
    want = (g * (x * np.linalg.solve(want, x.T).T).sum(1, keepdims=True)).T @ g / (T * k)
    assert np.linalg.norm(B.double().cpu().numpy() - want) <= 1e-3 * np.linalg.norm(want)


def test_flipflop_from_an_identity_of_many_workgroups():
    """16512 gradient channels: the first factor is that of the identity, all of which has to be there."""
    announce("flipflop m = 16512")
    torch = torch_cuda()
    kq = _kq()
    T, n, m = 300, 128, 16512
    gen = torch.Generator(device="cuda").manual_seed(5)
    X = torch.randn(T, n, generator=gen, device="cuda").to(torch.bfloat16)
    G = torch.randn(T, m, generator=gen, device="cuda").to(torch.bfloat16)
    A, B = torch.empty((n, n), device="cuda"), torch.empty((m, m), device="cuda")
    kq.kq_flipflop(X, G, 1, A, B)
    x, g = X.double().cpu().numpy(), G.double().cpu().numpy()
    want = (x * (g * g).sum(1, keepdims=True)).T @ x / (T * m)
    assert np.linalg.norm(A.double().cpu().numpy() - want) <= 1e-3 * np.linalg.norm(want)


def test_scaling_of_more_weights_than_threads():
    """2^34 weights and a few rows, signs only (alpha = 0 leaves the rescale at 1): every weight times its sign."""
    announce("biip 2^22 + 4 x 4096 without a transform")
    torch = torch_cuda()
    kq = _kq()
    out, n = (1 << 22) + 4, 4096
    gen = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(4, n, generator=gen, device="cuda")
    W = base.repeat(out // 4, 1)
    H = torch.eye(n, device="cuda")
    sign = (2 * torch.randint(0, 2, (n,), generator=gen, device="cuda") - 1).to(torch.int8)
    d_in, d_out = torch.empty(n, device="cuda"), torch.empty(out, device="cuda")
    kq.kq_biip_rotate(W, W, H, H, None, None, sign, None, d_in, d_out, alpha=0.0, mode=kq.KQ_BIIP_IN_ONLY, had_block_in=1)
    assert bool((d_in == 1).all())
    want = base * sign.float()
    for at in range(0, out, 1 << 18):
        assert bool((W[at:at + (1 << 18)].view(-1, 4, n) == want).all()), at


def test_reordered_columns_of_more_than_65535_rows():
    """act_order with 70000 output channels through the path of rows too long for LDS, where rows lie along
    the grid's second dimension: the bits of the path through LDS."""
    announce("gptq act_order 70000 x 256")
    torch = torch_cuda()
    kq = _kq()
    out, n = 70_000, 256
    gen = torch.Generator(device="cuda").manual_seed(7)
    W0 = torch.randn(out, n, generator=gen, device="cuda")
    X = torch.randn(2000, n, generator=gen, device="cuda") * torch.rand(n, generator=gen, device="cuda")
    H = X.T @ X + torch.eye(n, device="cuda")
    p = kq.make_params(4, n, 128, 0.01, act_order=1)
    ws = torch.empty(kq.kq_quantize_layer_workspace(p, out, n, False), dtype=torch.uint8, device="cuda")

    def run():
        W, codes = W0.clone(), torch.empty((out, n), dtype=torch.uint8, device="cuda")
        packed = torch.empty((out, n * 4 // 32), dtype=torch.int32, device="cuda")
        scales, zeros = torch.empty((out, 1), device="cuda"), torch.empty((out, 1), dtype=torch.uint8, device="cuda")
        kq.kq_quantize_layer(p, W, H.clone(), None, packed, scales, zeros, ws, codes=codes)
        return W, codes, packed, scales, zeros

    want = run()
    with kq.testing_select(kq.KQ_TESTING_ROW_LDS_BYTES, 0):
        got = run()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
