"""A mixture of experts served in MXFP4: rotated on the input side, quantised, applied.

    python examples/mxfp4_mixture.py --tokens 512 --width 2048 --inner 1408 --experts 16 --top 2

The block: every token goes through a shared layer and through `top` of the experts
(h = silu(gate) * up, then down), weighted by the router.  Weights are random; activations have a
few large channels, as those of language models do.  Preparation, once: the Hessian factor of the
activations (kq_accumulate_hessian), the input side of the incoherence processing
(kq_biip_rotate, KQ_BIIP_IN_ONLY; the experts of one product share its rescale and signs, so their
weights go through it as one matrix) and kq_mxfp4_quantize.  Serving, per call: one
kq_mxfp4_linear and two kq_mxfp4_experts.  Prints each product's error against fp32 with and
without the processing, and the time of a call.
"""
import argparse
import os
import sys

import torch

if __name__ == "__main__":
    sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import post_quantization_syrk_amd as kq


class Layers:
    """Layers W [experts, out, n] that read the same kind of rows, held in MXFP4."""

    def __init__(self, w, rows, processed=True):
        experts, out, n = w.shape
        self.d = self.sign = None
        self.had = 1
        flat = w.reshape(experts * out, n).float().contiguous()
        if processed:
            self.had = min(n & -n, 8192)
            h = torch.empty((n, n), device="cuda")
            kq.kq_accumulate_hessian(rows.to(torch.bfloat16).contiguous(), h)
            self.sign = (2 * torch.randint(0, 2, (n,), device="cuda") - 1).to(torch.int8)
            self.d, d_out = torch.empty(n, device="cuda"), torch.empty(experts * out, device="cuda")
            kq.kq_biip_rotate(flat, flat, h, h, None, None, self.sign, None, self.d, d_out,
                              mode=kq.KQ_BIIP_IN_ONLY, had_block_in=self.had)
        self.codes, self.scales = kq.kq_mxfp4_empty(out, n, experts)
        for e in range(experts):
            kq.kq_mxfp4_quantize(flat[e * out:(e + 1) * out], self.codes[e], self.scales[e])
        self.out, self.n = out, n

    def linear(self, x):
        y = torch.empty((x.shape[0], self.out), dtype=torch.bfloat16, device="cuda")
        kq.kq_mxfp4_linear(x, self.codes[0], self.scales[0], y, d=self.d, sign=self.sign, had=self.had)
        return y

    def experts(self, x, index, offsets):
        slots = x.shape[0] if index is None else index.shape[0]
        y = torch.empty((slots, self.out), dtype=torch.bfloat16, device="cuda")
        kq.kq_mxfp4_experts(x, index, offsets, self.codes, self.scales, y, d=self.d, sign=self.sign, had=self.had)
        return y


def route(x, router, top):
    """Slots sorted by expert: (token of each slot int32, first slot of each expert int32, weight)."""
    weight, chosen = torch.softmax(x.float() @ router, dim=1).topk(top, dim=1)
    expert, order = chosen.flatten().sort(stable=True)
    firsts = torch.searchsorted(expert, torch.arange(router.shape[1] + 1, device=x.device))
    return (order // top).int(), firsts.int(), weight.flatten()[order]


def gated(both):
    gate, up = both.float().chunk(2, dim=1)
    return (torch.nn.functional.silu(gate) * up).to(torch.bfloat16)


class Mixture:
    """shared [width, width], up [experts, 2 inner, width], down [experts, width, inner]."""

    def __init__(self, shared, up, down, router, top, calibration, processed=True):
        self.router, self.top = router, top
        self.shared = Layers(shared[None], calibration, processed)
        self.up = Layers(up, calibration, processed)
        index, offsets, _ = route(calibration, router, top)
        self.down = Layers(down, gated(self.up.experts(calibration, index, offsets)), processed)

    def __call__(self, x):
        index, offsets, weight = route(x, self.router, self.top)
        inner = gated(self.up.experts(x, index, offsets))
        y = self.down.experts(inner, None, offsets)
        out = self.shared.linear(x).float()
        return out.index_add_(0, index, y.float() * weight[:, None])


def plain(x, shared, up, down, router, top):
    """The same block in fp32 (its activations rounded to bf16 where the block's are)."""
    index, offsets, weight = route(x, router, top)
    out = x.float() @ shared.T
    first = offsets.tolist()
    for e in range(up.shape[0]):
        mine = slice(first[e], first[e + 1])
        inner = gated((x[index[mine]].float() @ up[e].T).to(torch.bfloat16))
        out.index_add_(0, index[mine], (inner.float() @ down[e].T) * weight[mine, None])
    return out


def make(tokens, width, inner, experts, seed=0):
    """(activations, shared, up, down, router) on the device."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")  # noqa: E731
    loud = torch.ones(width, device="cuda")
    loud[torch.randperm(width, generator=gen, device="cuda")[:max(1, width // 100)]] = 30.0
    x = (normal(tokens, width) * loud).to(torch.bfloat16)
    return (x, normal(width, width) / width ** 0.5, normal(experts, 2 * inner, width) / width ** 0.5,
            normal(experts, width, inner) / inner ** 0.5, normal(width, experts) / width ** 0.5)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    for name, value in (("tokens", 512), ("width", 2048), ("inner", 1408), ("experts", 16), ("top", 2)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    x, *weights = make(2 * a.tokens, a.width, a.inner, a.experts)
    calibration, x = x[:a.tokens], x[a.tokens:]
    want = plain(x, *weights, a.top)
    for processed in (False, True):
        block = Mixture(*weights, a.top, calibration, processed)
        error = (block(x) - want).norm() / want.norm()
        print(f"{'processed' if processed else 'as it is':10s} error against fp32 {float(error):.4f}")
    for tokens in (1, a.tokens):
        index, offsets, _ = route(x[:tokens], weights[3], a.top)
        inner = gated(block.up.experts(x[:tokens], index, offsets))
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        for turn in range(30):
            if turn == 10:
                begin.record()
            block.shared.linear(x[:tokens])
            block.up.experts(x[:tokens], index, offsets)
            block.down.experts(inner, None, offsets)
        end.record()
        end.synchronize()
        print(f"{tokens} token{'s' if tokens > 1 else ''}: the three products {begin.elapsed_time(end) / 20 * 1e3:.1f} us")


if __name__ == "__main__":
    main()
