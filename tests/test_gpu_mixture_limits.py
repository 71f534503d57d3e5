"""GPU parity at the far ends of what the mixture operators accept: more rows than one launch has threads,
sizes next to a limit of the launch, gradients over many rows of each lane layout.

Results are exact where nothing is rounded (one choice, no weights: a row of z or dy itself, and products of
two bf16 values, which fp32 holds); the other bounds are those of test_gpu_mixture.py.
"""
import numpy as np
import pytest

from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_mixture import Routes, _dev, _logits, _route_back_check, _route_check

pytestmark = pytest.mark.gpu


def _kq():
    import post_quantization_syrk_amd as kq
    return kq


def test_combine_backward_of_more_rows_than_threads_of_64():
    """2^26 rows and a few: a wave for each would be 2^32 threads."""
    announce("combine_backward (2^26 + 5) x 1")
    torch = torch_cuda()
    kq = _kq()
    rows = (1 << 26) + 5
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy = torch.randint(-200, 200, (rows, 1), generator=gen, device="cuda").to(torch.bfloat16)
    z = torch.randint(-200, 200, (rows, 1), generator=gen, device="cuda").to(torch.bfloat16)
    slot = torch.arange(rows - 1, -1, -1, dtype=torch.int32, device="cuda").view(rows, 1)
    dz, dweight = torch.full_like(z, 7.0), torch.full((rows, 1), 7.0, device="cuda")
    kq.kq_combine_backward(dy, z, slot, dz=dz, dweight=dweight)
    assert torch.equal(dz, dy.flip(0))
    assert torch.equal(dweight, dy.float() * z.flip(0).float())


def test_combine_backward_of_more_rows_than_threads_of_256():
    """2^24 rows and a few of more than 2048 columns: four waves for each would be 2^32 threads."""
    announce("combine_backward (2^24 + 3) x 2049")
    torch = torch_cuda()
    kq = _kq()
    rows, n = (1 << 24) + 3, 2049
    named = [0, 1, (1 << 20) - 1, 1 << 20, (1 << 24) - 1, 1 << 24, rows - 1]     # the rows with a slot
    gen = torch.Generator(device="cuda").manual_seed(2)
    dy = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")               # (the others' are not used)
    z = torch.randint(-3, 4, (len(named) + 1, n), generator=gen, device="cuda").to(torch.bfloat16)
    slot = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    for s, t in enumerate(named):
        dy[t] = torch.randint(-3, 4, (n,), generator=gen, device="cuda").to(torch.bfloat16)
        slot[t] = s
    dz, dweight = torch.full_like(z, 7.0), torch.full((rows, 1), 7.0, device="cuda")
    kq.kq_combine_backward(dy, z, slot, dz=dz, dweight=dweight)
    assert torch.equal(dz[:-1], dy[named]) and bool((dz[-1] == 7.0).all())
    # (whole numbers up to 9 * 2049: exact in any order)
    assert torch.equal(dweight[named, 0], (dy[named].float() * z[:-1].float()).sum(1))
    dweight[named] = 0
    assert not dweight.any()


def test_combine_of_more_columns_than_threads():
    """2^30 rows of 25 columns, eight a lane: 2^32 lanes."""
    announce("combine 2^30 x 25")
    torch = torch_cuda()
    kq = _kq()
    rows, n = 1 << 30, 25
    gen = torch.Generator(device="cuda").manual_seed(3)
    table = torch.randn(4, n, generator=gen, device="cuda").to(torch.bfloat16)
    table[3] = 0                                                                    # (slot 3 is none of z's)
    pattern = torch.randint(0, 4, (1 << 16,), generator=gen, dtype=torch.int32, device="cuda")
    slot = pattern.repeat(rows >> 16).view(rows, 1)
    y = torch.empty((rows, n), dtype=torch.bfloat16, device="cuda")
    y[-1], y[0] = 7.0, 7.0
    kq.kq_combine(table[:3], slot, y)
    want = table[pattern.long()]
    for at in range(0, rows, 1 << 24):
        assert bool((y[at:at + (1 << 24)].view(-1, 1 << 16, n) == want).all()), at


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("experts", [1635, 1636, 1637, 1638, 1639])
def test_route_next_to_64_kb_of_counts(experts, kind):
    """Experts whose counts take about 64 KB of LDS, with what the kernel holds beside them or without."""
    announce(f"route 70 x {experts} {kind}")
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(experts)
    for rows in (70, 6):
        x = _logits(rng, rows, experts, kind, True)
        r = Routes(rows, experts, 5)
        kq.kq_route(x.cuda(), normalize=True, **r.dict())
        want = _route_check(r, x, 5, True)
        dw, dloss = rng.standard_normal((rows, 5)).astype(np.float32), np.float32(2.0)
        g = torch.full((rows, experts), 7.0, dtype=x.dtype, device="cuda")
        kq.kq_route_backward(x.cuda(), g, r.weight, r.expert, r.counts, dweight=_dev(dw), dloss=_dev(dloss.reshape(1)), normalize=True)
        _route_back_check(g, x, want, dw, dloss, True, kind)
