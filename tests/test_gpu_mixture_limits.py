"""GPU parity at the far ends of what the mixture operators accept: more rows than one launch has threads,
sizes next to a limit of the launch, gradients over many rows of each lane layout.

Results are exact where nothing is rounded (one choice, no weights: a row of z or dy itself, and products of
two bf16 values, which fp32 holds); the other bounds are those of test_gpu_mixture.py.
"""
import numpy as np
import pytest

from tests.gpu_util import announce, torch_cuda
from tests.test_gpu_mixture import INF, U, Routes, _dev, _half, _logits, _route_back_check, _route_check

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


# (rows so many that every wave of the gradient's kernel has several groups of them, and no whole number; a
# case for each number of lanes a row and of values a lane)
MANY = [(70_001, 8, 2), (50_003, 30, 9), (99_998, 60, 4), (40_007, 100, 16), (131_075, 256, 8), (20_005, 300, 6), (17_001, 1000, 9),
        (9_001, 2000, 3), (12_291, 4000, 16)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("rows,experts,top", MANY)
def test_route_gradient_of_many_rows(rows, experts, top, normalize, kind):
    """Against the formula in 64 bits on the device, with the choices that kq_route made."""
    announce(f"route gradient {rows}x{experts} top {top} {kind} normalize {normalize}")
    torch = torch_cuda()
    kq = _kq()
    gen = torch.Generator(device="cuda").manual_seed(rows + normalize)
    x = 2 * torch.randn(rows, experts, generator=gen, device="cuda") + torch.randn(experts, generator=gen, device="cuda")
    x[torch.rand(rows, experts, generator=gen, device="cuda") < 0.2] = -INF
    x[torch.rand(rows, generator=gen, device="cuda") < 0.05] = -INF
    x = x.to(torch.bfloat16 if kind == "bf16" else torch.float32)
    dw, dloss = torch.randn(rows, top, generator=gen, device="cuda"), torch.full((1,), 0.3 * rows, device="cuda")
    r = Routes(rows, experts, top)
    kq.kq_route(x, normalize=normalize, **r.dict())
    g = torch.full_like(x, 7.0)
    kq.kq_route_backward(x, g, r.weight, r.expert, r.counts, dweight=dw, dloss=dloss, normalize=normalize)

    v = x.double()
    most = v.amax(1, keepdim=True)
    there = v > -INF
    far = torch.where(there, most - v, 0.0).max()
    e = torch.where(there, torch.exp(v - torch.where(most > -INF, most, 0.0)), 0.0)
    total = e.sum(1, keepdim=True)
    p = e / torch.where(total > 0, total, 1.0)
    chosen = r.expert >= 0
    at = r.expert.clamp(min=0).long()
    w = torch.where(chosen, e.gather(1, at), 0.0)
    under = w.sum(1, keepdim=True) if normalize else total
    w = w / torch.where(under > 0, under, 1.0)
    dw64 = torch.where(chosen, dw.double(), 0.0)
    made, used = max(int(r.counts[experts]), 1), max(int(r.counts[experts + 1]), 1)
    b = float(dloss) * experts * r.counts[:experts].double() / (float(made) * used)
    wg = (w * dw64).sum(1, keepdim=True)
    want = p * (b - (p * b).sum(1, keepdim=True) - (0.0 if normalize else wg))
    want.scatter_add_(1, at, w * (dw64 - wg) if normalize else w * dw64)      # (missing choices add zero)
    size_of = (w * dw64).abs()
    size = p * (b + (p * b).sum(1, keepdim=True) + size_of.sum(1, keepdim=True))
    size.scatter_add_(1, at, size_of + w * size_of.sum(1, keepdim=True))
    bound = (4 * far + 2 * experts + 2 * top + 64) * U * size + _half(kind) * want.abs() + 2.0 ** -126
    over = (g.double() - want).abs() - bound
    assert bool((over <= 0).all()), float(over.max())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("dloss", [INF, -INF, np.nan])
@pytest.mark.parametrize("experts", [7, 64, 256, 900])
def test_route_gradient_of_padding_beside_a_loss_that_is_not_finite(experts, dloss, kind):
    """Rows without a logit above -inf get zeros whatever comes back from the loss; choices that are missing
    take nothing from their weights' gradients."""
    torch = torch_cuda()
    kq = _kq()
    rng = np.random.default_rng(experts)
    x = _logits(rng, 60, experts, kind, False).cuda()
    padding = [0, 5, 17, 58, 59]
    x[padding] = -INF
    x[30, 1:] = -INF                       # (one choice of its three)
    dw = torch.ones(60, 3, device="cuda")
    dw[padding], dw[30, 1:] = np.nan, np.nan
    for normalize in (False, True):
        r = Routes(60, experts, 3)
        kq.kq_route(x, normalize=normalize, **r.dict())
        g = torch.full_like(x, 7.0)
        kq.kq_route_backward(x, g, r.weight, r.expert, r.counts, dweight=dw, normalize=normalize,
                             dloss=torch.full((1,), dloss, device="cuda"))
        assert not g[padding].any()
        rest = [t for t in range(60) if t not in padding]
        assert not torch.isfinite(g[rest]).all(1).any()
        kq.kq_route_backward(x, g, r.weight, r.expert, r.counts, dweight=dw, normalize=normalize)
        assert torch.isfinite(g).all() and not g[padding].any()


@pytest.mark.parametrize("zk,yk,rows,n,top,slots", [("bf16", "bf16", 16384, 2048, 6, 300), ("f32", "bf16", 9000, 4099, 8, 1), ("bf16", "f32", 70_000, 1025, 2, 140_001)])
def test_combine_of_slots_that_many_rows_name(zk, yk, rows, n, top, slots):
    """Few rows of z behind many choices, and more slots than choices: the sums in the order of the choices."""
    announce(f"combine {rows}x{n} top {top} of {slots} slots {zk} {yk}")
    torch = torch_cuda()
    kq = _kq()
    gen = torch.Generator(device="cuda").manual_seed(n)
    kind = {"bf16": torch.bfloat16, "f32": torch.float32}
    z = torch.randn(slots, n, generator=gen, device="cuda").to(kind[zk])
    slot = torch.randint(-1, slots + 1, (rows, top), generator=gen, device="cuda", dtype=torch.int32)    # (either end: none)
    weight = torch.randn(rows, top, generator=gen, device="cuda")
    y = torch.full((rows, n), 7.0, dtype=kind[yk], device="cuda")
    kq.kq_combine(z, slot, y, weight=weight)
    want, size = torch.zeros(rows, n, dtype=torch.float64, device="cuda"), torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    for j in range(top):
        there = (slot[:, j] >= 0) & (slot[:, j] < slots)
        term = z[slot[:, j].clamp(0, slots - 1).long()].double() * torch.where(there, weight[:, j].double(), 0.0)[:, None]
        want += term
        size += term.abs()
    bound = (top + 2) * U * size
    assert bool(((y.double() - want).abs() <= bound * (1 + _half(yk)) + _half(yk) * want.abs() + 2.0 ** -126).all())
