"""Timed cases of what surrounds the products of a mixture of experts held in MXFP4: routing with
its balance loss, products with an epilogue, and the sum of the experts' rows.

The operators:
  route     logits l [T, E]: p = softmax(l); the k largest logits of a row (ties: the lowest index,
            none of -inf); weights p of the chosen, or these divided by their sum; choices in a
            stable order by expert: the slot of each choice, the row of each slot, each expert's
            first slot and count; the balance loss L = E sum_e f_e P_e, with f_e expert e's share of
            the choices and P_e its mean probability over the rows that have one.  With training,
            the gradient of the logits too, from those of the weights and of the loss.
  linear    y = act(Q(x~) W^T + b) + r for a layer W held in MXFP4; gated: W has twice the rows,
            y = act(first half) * second half + r
  experts   the same with the layer of the expert that a slot belongs to
  combine   y[t] = r[t] + sum_j w[t, j] z[slot[t, j]]; with training, the gradients of z and w too

MXFP4, its layout and the rotation x~ of the activations are those of `operators.py` beside this
file: blocks of 32 values with a scale 2^e and E2M1 elements; codes [N][Kp / 2] bytes, Kp = K rounded
up to 128, the even element of a pair in the low nibble; scales [Kp / 128][N][4] bytes of e + 127.
"""
import math

import torch

own = False

GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
LARGEST_PRODUCT = 16384 * 4096 * 22016
LARGEST_ROUTE = 131072 * 256
LARGEST_COMBINE = 32768 * 2048 * 6


def listed():
    return [
        # one token of a mixture of eight: launch latency
        dict(name="route_token", op="route", rows=1, experts=8, pad=0, top=2, normalize=True, masked=False, train=False, x="f32"),
        # a padded batch of prompts over many small experts, some of them closed
        dict(name="route_prompt", op="route", rows=4099, experts=64, pad=0, top=6, normalize=False, masked=True, train=False, x="bf16"),
        # a training step over a calibration stream: weights, balance loss and the logits' gradient
        dict(name="route_train", op="route", rows=131072, experts=256, pad=0, top=8, normalize=True, masked=False, train=True, x="f32"),
        # decoding one sequence: a gate and up projection in one
        dict(name="linear_token", op="linear", rows=1, n=4096, out=11008, had=4096, x="bf16", y="bf16", act="silu", gated=True, bias=False, residual=None),
        # odd sizes in every direction, single precision, everything in the epilogue
        dict(name="linear_ragged", op="linear", rows=77, n=1000, out=4099, had=8, x="f32", y="f32", act="gelu", gated=False, bias=True, residual="f32"),
        # a prompt through a down projection, added to the stream it came from
        dict(name="linear_prompt", op="linear", rows=2048, n=11008, out=4096, had=256, x="bf16", y="bf16", act="none", gated=False, bias=True, residual="bf16"),
        # many prompts through a gate and up projection
        dict(name="linear_large", op="linear", rows=16384, n=4096, out=11008, had=4096, x="bf16", y="bf16", act="silu", gated=True, bias=False, residual=None),
        # a small batch over many small experts: a few rows each, some with none
        dict(name="experts_batch", op="experts", tokens=96, top=6, experts=64, n=2048, out=1408, had=2048, x="bf16", y="bf16", act="silu", gated=True, bias=False, residual=None),
        # a prompt over eight experts of uneven popularity
        dict(name="experts_prompt", op="experts", tokens=4096, top=2, experts=8, n=4096, out=11008, had=4096, x="bf16", y="bf16", act="silu", gated=True, bias=True, residual=None),
        # one token's experts summed onto the shared layer's output: launch latency
        dict(name="combine_token", op="combine", rows=1, n=4096, pad=0, top=2, weighted=True, dropped=False, train=False, z="bf16", y="bf16", residual="bf16"),
        # a prompt's, in rows of a wider buffer, some choices without a slot
        dict(name="combine_prompt", op="combine", rows=4099, n=4100, pad=3, top=2, weighted=True, dropped=True, train=False, z="bf16", y="f32", residual="f32"),
        # a training step over a calibration stream: the sum and both gradients
        dict(name="combine_train", op="combine", rows=32768, n=2048, pad=0, top=6, weighted=True, dropped=False, train=True, z="bf16", y="bf16", residual="bf16"),
    ]


def _log(rng, low, high):
    """A whole number of [low, high], even over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A width: half of them multiples of 128 as layers mostly have, half of them any."""
    n = _log(rng, low, high)
    return max(128, n // 128 * 128) if rng.random() < 0.5 else n


def draw(rng):
    op = rng.choice(("route", "linear", "experts", "combine"))
    if op == "route":
        experts = rng.choice((_log(rng, 1, 1024), rng.choice((8, 16, 64, 128, 256))))
        rows = _log(rng, 1, min(131072, LARGEST_ROUTE // experts))
        return dict(op=op, rows=rows, experts=experts, pad=rng.choice((0, 1, 8)), top=min(experts, rng.choice((1, 2, 3, 4, 6, 8))),
                    normalize=rng.random() < 0.5, masked=rng.random() < 0.5, train=rng.random() < 0.5, x=rng.choice(("bf16", "f32")))
    if op == "combine":
        top, n = rng.choice((1, 2, 3, 4, 6, 8)), _width(rng, 64, 16384)
        rows = _log(rng, 1, min(32768, LARGEST_COMBINE // (top * n)))
        return dict(op=op, rows=rows, n=n, pad=rng.choice((0, 0, 3, 8)), top=top, weighted=rng.random() < 0.75, dropped=rng.random() < 0.5,
                    train=rng.random() < 0.5, z=rng.choice(("bf16", "f32")), y=rng.choice(("bf16", "f32")), residual=rng.choice((None, "bf16", "f32")))
    case = dict(op=op, x=rng.choice(("bf16", "f32")), y=rng.choice(("bf16", "f32")), act=rng.choice(ACTS), gated=rng.random() < 0.5,
                bias=rng.random() < 0.5, residual=rng.choice((None, "bf16", "f32")))
    wide = 1 + case["gated"]
    if op == "linear":
        n, out = _width(rng, 64, 16384), _width(rng, 64, 16384)
        while n * out * wide > 16384 * 16384:
            n, out = (n + 1) // 2, (out + 1) // 2
        case |= dict(rows=_log(rng, 1, min(16384, LARGEST_PRODUCT // (n * out * wide))), n=n, out=out)
    else:
        experts, n, out = _log(rng, 4, 128), _width(rng, 256, 8192), _width(rng, 256, 16384)
        while experts * n * out * wide > 8 * 4096 * 22016:
            n, out = max(64, n // 2), max(64, out // 2)
        top = rng.choice((1, 2, 4))
        case |= dict(tokens=_log(rng, 1, max(1, min(8192, LARGEST_PRODUCT // (top * n * out * wide)))), top=top, experts=experts, n=n, out=out)
    # the largest power of two that divides the width, as the incoherence processing takes it, or no rotation
    case["had"] = min(8192, case["n"] & -case["n"]) if rng.random() < 0.75 else 1
    return case


# ---- inputs ----

def _normal(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return g, lambda *s: torch.randn(*s, generator=g, device="cuda")


def _typed(normal, rows, n, pad, kind, scale=None):
    """A matrix in rows of a buffer that is `pad` wider."""
    v = normal(rows, n + pad)
    return (v if scale is None else v * scale).to(DTYPES[kind])[:, :n]


def _choose(logits, top):
    """(experts, logits) of the `top` largest, the lower index first among equal ones."""
    value, expert = logits.sort(dim=1, descending=True, stable=True)
    return expert[:, :top], value[:, :top]


def _order(expert, experts):
    """Choices (-1: none) in a stable order by expert: (row of each slot, first slots, slot of each choice, counts)."""
    flat, top = expert.reshape(-1), expert.shape[1]
    key = torch.where(flat < 0, experts, flat)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device).index_add_(0, key, torch.ones_like(key))[:experts]
    offsets = torch.cat((counts.new_zeros(1), counts.cumsum(0)))
    place = torch.arange(len(flat), device=flat.device)
    slot = torch.empty_like(order).scatter_(0, order, place)
    index = torch.where(place < offsets[-1], order // top, -1)
    return index.int(), offsets.int(), torch.where(flat < 0, -1, slot).view(expert.shape).int(), counts.int()


def _route_inputs(case, seed):
    """Router logits with experts of uneven popularity; masked: some experts closed, padding rows,
    rows with fewer open experts than choices, equal logits."""
    g, normal = _normal(seed)
    rows, experts = case["rows"], case["experts"]
    logits = normal(rows, experts + case["pad"]) + 0.5 * normal(experts + case["pad"])
    if case["masked"]:
        logits[:, torch.rand(experts + case["pad"], generator=g, device="cuda") < 0.1] = -math.inf
        kind = torch.rand(rows, generator=g, device="cuda")
        logits[kind < 0.1] = -math.inf
        some = torch.rand(logits.shape, generator=g, device="cuda") < 1.0 / experts
        logits = torch.where((kind > 0.95)[:, None] & ~some, -math.inf, logits)
        logits = torch.where(((kind > 0.9) & (kind < 0.92))[:, None], 0.25, logits)
    return logits.to(DTYPES[case["x"]])[:, :experts], normal(rows, case["top"]), 0.01 * normal(()).abs() * rows


def _combine_inputs(case, seed):
    """Experts' rows in slot order, the slots of each row's choices, and the gradient of the sum."""
    g, normal = _normal(seed)
    rows, n, top, pad = case["rows"], case["n"], case["top"], case["pad"]
    expert = torch.randint(0, 64, (rows, top), generator=g, device="cuda")
    if case["dropped"]:
        expert[torch.rand(rows, top, generator=g, device="cuda") < 0.1] = -1
    slot = _order(expert, 64)[2]
    z = _typed(normal, rows * top, n, pad, case["z"])
    weight = torch.softmax(normal(rows, top), dim=1) if case["weighted"] else None
    residual = _typed(normal, rows, n, pad, case["residual"]) if case["residual"] else None
    dy = _typed(normal, rows, n, pad, case["y"]) if case["train"] else None
    return z, slot, weight, residual, dy


def _product_inputs(case, seed):
    """Activations with log-normal channel scales, the rescale vector that evens them out in part,
    the rotation's signs; then, in this order, routing, weights, bias and residual."""
    g, normal = _normal(seed)
    rows, n = case.get("rows", case.get("tokens")), case["n"]
    scale = normal(n).exp()
    x = _typed(normal, rows, n, 0, case["x"], scale)
    d = (scale.sqrt() * (0.1 * normal(n)).exp()) if case["had"] > 1 else None
    sign = (torch.randint(0, 2, (n,), generator=g, device="cuda") * 2 - 1).to(torch.int8) if case["had"] > 1 else None
    experts, slots, index, offsets = case.get("experts", 1), rows * case.get("top", 1), None, None
    if case["op"] == "experts":
        popular = normal(experts)
        index, offsets, _, _ = _order(_choose(popular + normal(rows, experts), case["top"])[0], experts)
    wide = case["out"] * (1 + case["gated"])
    bias = 0.5 * normal(experts, wide) if case["bias"] else None
    residual = _typed(normal, slots, case["out"], 0, case["residual"]) if case["residual"] else None
    # weights that make sums of order one: |x~| is about the geometric mean of its channels' scales
    layers = (normal(wide, n) / math.sqrt(n) / 2 for _ in range(experts))
    return x, d, sign, index, offsets, bias, residual, layers


# ---- MXFP4 in 32 bits ----

def _blocks(n):
    """Columns of a quantised row of n values: whole groups of 128."""
    return (n + 127) // 128 * 128


def _encode(x):
    """Codes 0..15 [rows, Kp] and scale exponents [rows, Kp / 32] of finite x in 32 bits."""
    rows, n = x.shape
    v = torch.nn.functional.pad(x, (0, _blocks(n) - n)).view(rows, -1, 32)
    e = ((v.abs().amax(2).view(torch.int32) >> 23) - 129).clamp(min=-127)
    v = v * ((127 - e) << 23).view(torch.float32).unsqueeze(2)
    a = v.abs()
    code = (a > 0.25).to(torch.uint8)
    for limit in (0.75, 1.75, 3.5):
        code += a >= limit
    for limit in (1.25, 2.5, 5.0):
        code += a > limit
    return (code + 8 * (v < 0).to(torch.uint8)).view(rows, -1), e


def _decode(code, e):
    """The values in 32 bits: element times 2^e (two exact factors, since 2^-127 is no normal number)."""
    rows = code.shape[0]
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=code.device)
    scale = ((e.clamp(max=125) + 129) << 23).view(torch.float32)
    return (grid[code.int()].view(rows, -1, 32) * 0.25 * scale.unsqueeze(2)).view(rows, -1)


def _pack(code, e):
    """A layer as it is held: two codes in a byte, four blocks' scale bytes by 128 columns and row."""
    rows = code.shape[0]
    pair = code.view(rows, -1, 2)
    scales = (e + 127).to(torch.uint8).view(rows, -1, 4).transpose(0, 1).contiguous()
    return pair[..., 0] | (pair[..., 1] << 4), scales


def _unpack(codes, scales):
    """The values of a held layer, [rows, Kp]."""
    rows = codes.shape[0]
    code = torch.stack((codes & 15, codes >> 4), dim=2).view(rows, -1)
    return _decode(code, scales.transpose(0, 1).reshape(rows, -1).int() - 127)


def _rotate(x, d, sign, had):
    """P (x / d) / sqrt(b), in 32 bits: butterflies of the Sylvester matrix, strides ascending."""
    x = x.float()
    if d is not None:
        x = x * (sign.float() / d)
    h = 1
    while h < had:
        pair = x.reshape(x.shape[0], -1, 2, h)
        a, c = pair[:, :, 0], pair[:, :, 1]
        x = torch.stack((a + c, a - c), dim=2).view(x.shape[0], -1)
        h *= 2
    return x * (1.0 / math.sqrt(had)) if had > 1 else x


def _act(v, kind):
    if kind == "relu":
        return torch.clamp(v, min=0)
    if kind == "silu":
        return v / (1 + torch.exp(-v))
    if kind == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


# ---- a pass ----

def prepare(case, seed):
    s = dict(case=case)
    empty = lambda *shape, kind=torch.float32: torch.empty(*shape, dtype=kind, device="cuda")  # noqa: E731
    if case["op"] == "route":
        s["logits"], s["dweight"], s["dloss"] = _route_inputs(case, seed)
        rows, experts, top = case["rows"], case["experts"], case["top"]
        s["routes"] = dict(weight=empty(rows, top), expert=empty(rows, top, kind=torch.int32), slot=empty(rows, top, kind=torch.int32),
                           index=empty(rows * top, kind=torch.int32), offsets=empty(experts + 1, kind=torch.int32),
                           counts=empty(experts + 2, kind=torch.int32))
        if case["train"]:
            s["routes"]["loss"] = empty(1)
            s["dlogits"] = empty(rows, experts, kind=DTYPES[case["x"]])
        return s
    if case["op"] == "combine":
        s["z"], s["slot"], s["weight"], s["residual"], s["dy"] = _combine_inputs(case, seed)
        s["y"] = empty(case["rows"], case["n"], kind=DTYPES[case["y"]])
        if case["train"]:
            s["dz"] = torch.zeros(case["rows"] * case["top"], case["n"], dtype=DTYPES[case["z"]], device="cuda")
            s["dweight"] = empty(case["rows"], case["top"])
        return s
    s["x"], s["d"], s["sign"], s["index"], s["offsets"], s["bias"], s["residual"], layers = _product_inputs(case, seed)
    s["codes"], s["scales"] = (torch.stack(v) for v in zip(*(_pack(*_encode(w)) for w in layers)))
    if case["op"] == "linear":
        s["codes"], s["scales"] = s["codes"][0], s["scales"][0]
        s["bias"] = s["bias"][0] if case["bias"] else None
    rows, held = s["x"].shape[0], _blocks(case["n"])
    s["y"] = empty(rows * case.get("top", 1), case["out"], kind=DTYPES[case["y"]])
    s["ws"] = empty(held // 128 * 68 * rows, kind=torch.uint8)  # the quantised activations
    return s


def _plain_route(s):
    case, x = s["case"], s["logits"].float()
    experts, top = case["experts"], case["top"]
    expert, value = _choose(x, top)
    has = value[:, :1] > -math.inf  # rows with a softmax
    most = torch.where(has, value[:, :1], 0.0)
    p = torch.exp(x - most)
    total = p.sum(1, keepdim=True)
    p = p / torch.where(has, total, 1.0)
    chosen = value > -math.inf
    weight = torch.exp(value - most)
    weight = weight / torch.where(has, weight.sum(1, keepdim=True) if case["normalize"] else total, 1.0)
    expert = torch.where(chosen, expert, -1)
    index, offsets, slot, counts = _order(expert, experts)
    made, used = counts.sum(), has.sum()
    out = dict(weight=weight, expert=expert.int(), slot=slot, index=index, offsets=offsets, counts=torch.cat((counts, made[None].int(), used[None].int())))
    if not case["train"]:
        return out
    share, rows = counts / made.clamp(min=1).double(), used.clamp(min=1).double()
    out["loss"] = (experts * (share * p.sum(0, dtype=torch.float64) / rows).sum()).float()[None]
    balance = (s["dloss"].double() * experts * share / rows).float()
    dl = p * (balance - (p * balance).sum(1, keepdim=True))
    dw = torch.where(chosen, s["dweight"], 0.0)
    dot = (weight * dw).sum(1, keepdim=True)
    if not case["normalize"]:
        dl = dl - p * dot
    own_part = torch.where(chosen, weight * (dw - dot if case["normalize"] else dw), 0.0)
    out["dlogits"] = dl.scatter_add(1, expert.clamp(min=0), own_part).to(s["dlogits"].dtype)
    return out


def _plain_combine(s):
    case, top = s["case"], s["case"]["top"]
    there = s["slot"] >= 0
    weight = torch.where(there, 1.0 if s["weight"] is None else s["weight"], 0.0)
    rows = s["z"][s["slot"].clamp(min=0).view(-1).long()].view(case["rows"], top, -1).float()
    y = (rows * weight[:, :, None]).sum(1)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = dict(y=y.to(s["y"].dtype))
    if case["train"]:
        dy = s["dy"].float()
        out["dweight"] = torch.where(there, (rows * dy[:, None]).sum(2), 0.0)
        dz = (dy[:, None] * weight[:, :, None]).to(s["dz"].dtype)
        out["dz"] = torch.zeros_like(s["dz"])
        out["dz"][s["slot"][there].long()] = dz[there]
    return out


def _finish(v, bias, case, residual, dtype):
    if bias is not None:
        v = v + bias
    if case["gated"]:
        v = _act(v[:, :case["out"]], case["act"]) * v[:, case["out"]:]
    else:
        v = _act(v, case["act"])
    return (v if residual is None else v + residual.float()).to(dtype)


def _plain_product(s):
    case = s["case"]
    x = _decode(*_encode(_rotate(s["x"], s["d"], s["sign"], case["had"])))
    if case["op"] == "linear":
        return _finish(x @ _unpack(s["codes"], s["scales"]).T, s["bias"], case, s["residual"], s["y"].dtype)
    y = torch.empty_like(s["y"])
    first = s["offsets"].tolist()
    for e in range(case["experts"]):
        mine = slice(first[e], first[e + 1])
        if first[e] < first[e + 1]:
            v = x[s["index"][mine]] @ _unpack(s["codes"][e], s["scales"][e]).T
            y[mine] = _finish(v, s["bias"][e] if case["bias"] else None, case, s["residual"][mine] if case["residual"] else None, y.dtype)
    return y


def run(s):
    case = s["case"]
    if not own:
        return {"route": _plain_route, "combine": _plain_combine}.get(case["op"], _plain_product)(s)
    import post_quantization_syrk_amd as kq

    if case["op"] == "route":
        r = s["routes"]
        kq.kq_route(s["logits"], normalize=case["normalize"], **r)
        if not case["train"]:
            return r
        kq.kq_route_backward(s["logits"], s["dlogits"], r["weight"], r["expert"], r["counts"], dweight=s["dweight"], dloss=s["dloss"],
                             normalize=case["normalize"])
        return {**r, "dlogits": s["dlogits"]}
    if case["op"] == "combine":
        kq.kq_combine(s["z"], s["slot"], s["y"], weight=s["weight"], residual=s["residual"])
        if not case["train"]:
            return dict(y=s["y"])
        kq.kq_combine_backward(s["dy"], s["z"], s["slot"], s["dz"], weight=s["weight"], dweight=s["dweight"])
        return dict(y=s["y"], dweight=s["dweight"], dz=s["dz"])
    rest = dict(d=s["d"], sign=s["sign"], had=case["had"], bias=s["bias"], act=case["act"], gated=case["gated"], residual=s["residual"])
    if case["op"] == "linear":
        kq.kq_mxfp4_linear_epilogue(s["x"], s["codes"], s["scales"], s["y"], s["ws"], **rest)
    else:
        kq.kq_mxfp4_experts_epilogue(s["x"], s["index"], s["offsets"], s["codes"], s["scales"], s["y"], s["ws"], **rest)
    return s["y"]


def work(case):
    """Inputs once, outputs once; of the experts only those that a token can reach."""
    if case["op"] == "route":
        grid, choices = case["rows"] * case["experts"], case["rows"] * case["top"]
        size = SIZE[case["x"]]
        moved, flops = grid * size + 16 * choices + 8 * case["experts"], grid * (4 + case["top"])
        if case["train"]:
            moved, flops = moved + 2 * grid * size + 12 * choices, flops + 6 * grid
        return {"bytes": moved, "flops": flops}
    if case["op"] == "combine":
        row, choices = case["rows"] * case["n"], case["rows"] * case["top"]
        z, y, r = choices * case["n"] * SIZE[case["z"]], row * SIZE[case["y"]], row * SIZE[case["residual"]] if case["residual"] else 0
        moved, flops = z + y + r + 8 * choices, 2 * choices * case["n"]
        if case["train"]:
            moved, flops = moved + 2 * z + y + 12 * choices, 5 * choices * case["n"]
        return {"bytes": moved, "flops": flops}
    n, held, rows = case["n"], _blocks(case["n"]), case.get("rows", case.get("tokens"))
    slots, wide = rows * case.get("top", 1), case["out"] * (1 + case["gated"])
    used = min(case.get("experts", 1), slots)
    moved = rows * n * SIZE[case["x"]] + 5 * n * (case["had"] > 1) + used * wide * (held * 17 // 32 + 4 * case["bias"])
    moved += slots * case["out"] * (SIZE[case["y"]] + (SIZE[case["residual"]] if case["residual"] else 0))
    return {"bytes": moved, "flops": rows * n * (math.log2(case["had"]) + 2) + 2 * slots * n * wide}


# ---- the definitions in 64 bits ----

def _exact_values(x):
    """The MXFP4 values of x, in 64 bits: a rounding to multiples of the step at each magnitude."""
    rows, n = x.shape
    v = torch.nn.functional.pad(x, (0, -n % 32)).view(rows, -1, 32)
    top = v.abs().amax(2, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(min=-127).where(top > 0, torch.full_like(top, -127).int())
    scale = torch.ldexp(torch.ones_like(top), e)
    a = (v / scale).abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    return (torch.sign(v) * a * scale).view(rows, -1)[:, :n]


def _sylvester(b):
    h = torch.ones(1, 1, dtype=torch.float64, device="cuda")
    while h.shape[0] < b:
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    return h


def _exact_route(case, seed):
    logits, dweight, dloss = _route_inputs(case, seed)
    experts, top = case["experts"], case["top"]
    l64 = logits.double().requires_grad_(case["train"])
    with torch.set_grad_enabled(case["train"]):
        has = torch.isfinite(l64).any(1)
        live = l64[has]
        p = torch.softmax(live, dim=1)
        # one choice after another: the first of the largest that is left
        left, picks = live.detach().clone(), []
        for _ in range(top):
            best = left.amax(1, keepdim=True)
            pick = (left == best).int().argmax(1, keepdim=True)
            picks.append(torch.where(best > -math.inf, pick, -1))
            left.scatter_(1, pick, -math.inf)
        picks = torch.cat(picks, 1) if len(live) else torch.empty(0, top, dtype=torch.int64, device="cuda")
        w = torch.where(picks >= 0, p.gather(1, picks.clamp(min=0)), 0.0)
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True)
        counts = (picks[:, :, None] == torch.arange(experts, device="cuda")).sum((0, 1)) if len(live) * top * experts < 1 << 26 else \
            torch.bincount(picks[picks >= 0], minlength=experts)
        made, used = int(counts.sum()), len(live)
        loss = experts * (counts / max(made, 1) * p.sum(0) / max(used, 1)).sum()
        full = lambda v, fill: torch.full((case["rows"], top), fill, dtype=v.dtype, device="cuda").index_copy(0, has.nonzero()[:, 0], v)  # noqa: E731
        weight, expert = full(w, 0.0), full(picks, -1)
        if case["train"]:
            grad = torch.autograd.grad((weight * dweight.double()).sum() + dloss.double() * loss, l64)[0]
    flat = expert.reshape(-1)
    choice = (flat >= 0).nonzero()[:, 0]
    choice = choice[torch.sort(flat[choice], stable=True)[1]]
    index = torch.full_like(flat, -1)
    index[:made] = choice // top
    slot = torch.full_like(flat, -1)
    slot[choice] = torch.arange(made, device="cuda")
    offsets = torch.searchsorted(flat[choice].contiguous(), torch.arange(experts + 1, device="cuda"))
    out = dict(weight=weight.detach(), expert=expert, slot=slot.view(expert.shape), index=index, offsets=offsets,
               counts=torch.cat((counts, torch.tensor([made, used], device="cuda"))))
    if case["train"]:
        out |= dict(loss=loss.detach()[None], dlogits=grad)
    return out


def _exact_combine(case, seed):
    z, slot, weight, residual, dy = _combine_inputs(case, seed)
    y = torch.zeros(case["rows"], case["n"], dtype=torch.float64, device="cuda") if residual is None else residual.double()
    dw = torch.zeros(case["rows"], case["top"], dtype=torch.float64, device="cuda")
    dz = torch.zeros(z.shape, dtype=torch.float64, device="cuda")
    for j in range(case["top"]):
        t = (slot[:, j] >= 0).nonzero()[:, 0]
        at = slot[t, j].long()
        w = torch.ones(len(t), 1, dtype=torch.float64, device="cuda") if weight is None else weight[t, j, None].double()
        mine = z[at].double()
        y[t] += w * mine
        if case["train"]:
            dw[t, j] = (mine * dy[t].double()).sum(1)
            dz[at] = w * dy[t].double()
    return dict(y=y, dweight=dw, dz=dz) if case["train"] else dict(y=y)


def exact(case, seed):
    if case["op"] == "route":
        return _exact_route(case, seed)
    if case["op"] == "combine":
        return _exact_combine(case, seed)
    x, d, sign, index, offsets, bias, residual, layers = _product_inputs(case, seed)
    layers = list(layers)
    x = x.double()
    if case["had"] > 1:
        b = case["had"]
        x = x / d.double() * sign.double()
        x = ((x.reshape(-1, b) @ _sylvester(b)) / math.sqrt(b)).view(x.shape)
    x = _exact_values(x)

    def layer(rows, e, r):
        v = rows @ _exact_values(layers[e].double()).T
        if bias is not None:
            v = v + bias[e].double()
        half = v[:, :case["out"]]
        if case["act"] == "relu":
            half = torch.relu(half)
        elif case["act"] == "silu":
            half = half * torch.sigmoid(half)
        elif case["act"] == "gelu":
            half = half * torch.special.ndtr(half)
        elif case["act"] == "gelu_tanh":  # (1 + tanh u) / 2 = sigmoid(2 u)
            half = half * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (half + 0.044715 * half ** 3))
        v = half * v[:, case["out"]:] if case["gated"] else half
        return v if r is None else v + r.double()

    if case["op"] == "linear":
        return layer(x, 0, residual)
    y = torch.empty(len(index), case["out"], dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        mine = slice(int(offsets[e]), int(offsets[e + 1]))
        if int(offsets[e]) < int(offsets[e + 1]):
            y[mine] = layer(x[index[mine].long()], e, residual[mine] if residual is not None else None)
    return y
