"""The operators of layer-wise quantisation-aware training, as a user's program calls them, and their plain forms.

Four operators around the trellis kernels: 8-bit floating-point codes with one
power-of-two scale for each block of 128 (``fp8_quantise``), the matrix product
of two such operands (``fp8_matmul``), the Newton-Schulz orthogonalisation of
an update (``orthogonalise``), and the whole Muon step on the latent weights
(``muon_step``).  A case is one call of one of them.

With ``own`` false, ``run`` computes the operator in elementary torch
operations in fp32; with ``own`` true it calls ``bcjr_sum_product_b200.lib``.
``exact`` gives the same outputs in fp64 from the operators' definitions.
"""
import math

import torch

own = False

#: Muon's quintic: x -> 3.4445 x - 4.7750 x^3 + 2.0315 x^5, five times, on the update over its Frobenius norm.
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
MU = 0.95
LR = 1e-3
DECAY = 0.01

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
#: Largest finite value of each 8-bit type: 0.875 * 2^TOP.
TOP = {"e4m3": 9, "e5m2": 16}
BLOCK = 128

#: Work of the largest listed cases; draws stay below.
MOST_QUANTISED = 8192 * 8192
MOST_MULTIPLIED = 8192 * 8192 * 2048
MOST_ORTHOGONALISED = 8192 * 2048 * 2048


def listed():
    return [
        # serving: the activations of one small decoding batch, before the first projection
        {"name": "quantise_decode", "op": "quantise", "rows": 16, "cols": 2048, "x": "bf16", "q": "e4m3", "block_rows": 1, "layout": "rows", "minus": False},
        # a calibration batch of activations of odd length, needed along both axes (forward and weight gradient)
        {"name": "quantise_tokens", "op": "quantise", "rows": 4003, "cols": 2048, "x": "bf16", "q": "e4m3", "block_rows": 1, "layout": "both", "minus": False},
        # what the trellis code leaves of the largest matrix of a decoder layer: soft codeword minus target, in 128 x 128 blocks
        {"name": "quantise_residual", "op": "quantise", "rows": 8192, "cols": 8192, "x": "fp32", "q": "e4m3", "block_rows": 128, "layout": "both", "minus": True},
        # serving: one token through a gate or up projection
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": 8192, "k": 2048, "a": "e4m3", "b": "e4m3", "a_rows": 1, "b_rows": 128, "out": "bf16", "alpha": 1.0},
        # serving: a ragged decoding batch through a key projection whose inner length is not a multiple of 128
        {"name": "matmul_batch", "op": "matmul", "m": 37, "n": 512, "k": 2000, "a": "e4m3", "b": "e4m3", "a_rows": 1, "b_rows": 128, "out": "bf16", "alpha": 1.0},
        # training: a batch of tokens through the up projection
        {"name": "matmul_forward", "op": "matmul", "m": 8192, "n": 8192, "k": 2048, "a": "e4m3", "b": "e4m3", "a_rows": 1, "b_rows": 128, "out": "bf16", "alpha": 1.0},
        # training: the gradient of a square projection's weights, summed over the tokens, the upstream gradient in e5m2
        {"name": "matmul_weight_grad", "op": "matmul", "m": 2048, "n": 2048, "k": 8192, "a": "e5m2", "b": "e4m3", "a_rows": 1, "b_rows": 1, "out": "fp32", "alpha": 2.0},
        # the update of a key or value projection
        {"name": "orthogonalise_key", "op": "orthogonalise", "batch": 1, "rows": 512, "cols": 2048, "g": "fp32", "out": "bf16"},
        # the updates of sixteen small matrices of one shape at once, rows the longer side, sizes odd
        {"name": "orthogonalise_batch", "op": "orthogonalise", "batch": 16, "rows": 333, "cols": 130, "g": "bf16", "out": "bf16"},
        # the update of a down projection
        {"name": "orthogonalise_down", "op": "orthogonalise", "batch": 1, "rows": 2048, "cols": 8192, "g": "bf16", "out": "bf16"},
        # one training step on a square projection
        {"name": "muon_square", "op": "muon", "rows": 2048, "cols": 2048, "g": "fp32", "nesterov": True},
        # one training step on an up projection: rows the longer side
        {"name": "muon_up", "op": "muon", "rows": 8192, "cols": 2048, "g": "fp32", "nesterov": True},
    ]


def _size(rng, low, high):
    """A size spread over the logarithm of its range; every other one near a multiple of 128 or of 16."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    step = rng.choice((1, 1, 16, 128))
    return min(high, max(low, n - n % step))


def draw(rng):
    op = rng.choice(("quantise", "matmul", "matmul", "orthogonalise", "muon"))
    if op == "quantise":
        rows, cols = _size(rng, 1, 8192), _size(rng, 1, 8192)
        return {"op": op, "rows": rows, "cols": cols, "x": rng.choice(("fp32", "bf16", "fp16")), "q": rng.choice(("e4m3", "e4m3", "e5m2")),
                "block_rows": rng.choice((1, 128)), "layout": rng.choice(("rows", "cols", "both")), "minus": rng.random() < 0.3}
    if op == "matmul":
        while True:
            m, n, k = _size(rng, 1, 8192), _size(rng, 16, 8192), _size(rng, 16, 8192)
            if m * n * k <= MOST_MULTIPLIED:
                break
        return {"op": op, "m": m, "n": n, "k": k, "a": rng.choice(("e4m3", "e4m3", "e5m2")), "b": rng.choice(("e4m3", "e4m3", "e5m2")),
                "a_rows": rng.choice((1, 1, 128)), "b_rows": rng.choice((1, 128, 128)), "out": rng.choice(("bf16", "fp16", "fp32")), "alpha": rng.choice((1.0, 2.0))}
    while True:
        rows, cols = _size(rng, 16, 8192), _size(rng, 16, 8192)
        batch = 1 if op == "muon" else rng.choice((1, 1, 1, 4, 7))
        if batch * rows * cols * min(rows, cols) <= MOST_ORTHOGONALISED:
            break
    if op == "orthogonalise":
        return {"op": op, "batch": batch, "rows": rows, "cols": cols, "g": rng.choice(("fp32", "bf16", "fp16")), "out": rng.choice(("bf16", "bf16", "fp16"))}
    return {"op": op, "rows": rows, "cols": cols, "g": rng.choice(("fp32", "fp32", "bf16")), "nesterov": rng.random() < 0.7}


# ---------------------------------------------------------------- inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _activations(g, rows, cols):
    """Unit normal rows with a few large channels, and one row in sixteen empty (padding)."""
    x = _randn(g, rows, cols)
    x *= 1.0 + 19.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01).float()
    x *= (torch.rand(rows, 1, generator=g, device="cuda") > 1.0 / 16 if rows > 1 else torch.ones(1, 1, device="cuda")).float()
    return x


def _update(g, *shape):
    """A gradient: a few strong directions over noise, at a gradient's magnitude."""
    rank = min(8, shape[-2], shape[-1])
    strong = torch.arange(1, rank + 1, device="cuda").float().reciprocal()
    u, v = _randn(g, *shape[:-1], rank), _randn(g, *shape[:-2], rank, shape[-1])
    return 1e-3 * (_randn(g, *shape) + (u * strong) @ v)


def _padded(codes, multiple=16):
    """The same values in rows that start at multiples of 16 bytes, as the kernels take and give them."""
    rows, cols = codes.shape
    room = torch.zeros(rows, -(-cols // multiple) * multiple, dtype=torch.uint8, device=codes.device)
    room[:, :cols] = codes.view(torch.uint8)
    return room.view(codes.dtype)[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "quantise":
        x = _activations(g, case["rows"], case["cols"])
        s["x"] = x.to(TYPES[case["x"]])
        s["minus"] = x + 0.1 * _randn(g, case["rows"], case["cols"]) if case["minus"] else None
    elif case["op"] == "matmul":
        for name, rows, x in (("a", "m", _activations(g, case["m"], case["k"])), ("b", "n", _randn(g, case["n"], case["k"]))):
            q, scale = _quantise(x, case[name + "_rows"], case[name])
            s[name], s["scale_" + name] = _padded(q), scale
    elif case["op"] == "orthogonalise":
        s["g"] = _update(g, case["batch"], case["rows"], case["cols"]).to(TYPES[case["g"]])
    else:
        s["w"] = _randn(g, case["rows"], case["cols"])
        s["momentum"] = 4.0 * _update(g, case["rows"], case["cols"])
        s["g"] = _update(g, case["rows"], case["cols"]).to(TYPES[case["g"]])
    return s


# ---------------------------------------------------------------- plain forms

def _blocks(x, rows):
    """[rows of blocks, rows, blocks, 128], zeros behind the end."""
    r, c = x.shape
    x = torch.nn.functional.pad(x, (0, -c % BLOCK, 0, -r % rows))
    return x.reshape(x.shape[0] // rows, rows, -1, BLOCK)


def _quantise(x, rows, kind):
    """Codes, and for each block the smallest power of two (at least 2^-127) that brings its values into the type's range."""
    x = x.float()
    b = _blocks(x, rows)
    most = b.abs().amax(dim=(1, 3))
    m, e = torch.frexp(most)
    e = torch.where(m > 0.875, e - TOP[kind] + 1, e - TOP[kind]).clamp_min(-127)
    e = torch.where(most == 0, torch.zeros_like(e), e)
    scale = torch.where(torch.isfinite(most), e + 127, torch.full_like(e, 255)).to(torch.uint8)
    factor = torch.where(torch.isfinite(most), torch.ldexp(torch.ones_like(most), -e), torch.full_like(most, math.nan))
    q = (b * factor[:, None, :, None]).to(TYPES[kind])
    q = q.view(torch.uint8).reshape(q.shape[0] * rows, -1)[: x.shape[0], : x.shape[1]].view(TYPES[kind])
    return q, scale.view(torch.float8_e8m0fnu)


def _values(q, scale, rows):
    """What codes and scales stand for, in fp32."""
    s = scale.float().repeat_interleave(rows, 0)[: q.shape[0]].repeat_interleave(BLOCK, 1)[:, : q.shape[1]]
    return q.float() * s


def _newton_schulz(x):
    """Of [..., rows, cols] in fp32."""
    flip = x.shape[-2] > x.shape[-1]
    x = x.mT if flip else x
    x = x / (x.square().sum(dim=(-2, -1), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFS
    for _ in range(STEPS):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if flip else x


def _scale(rows, cols):
    return math.sqrt(max(1.0, rows / cols))


def _plain(s):
    if s["op"] == "quantise":
        x = s["x"].float()
        x = x if s["minus"] is None else x - s["minus"]
        out = []
        if s["layout"] in ("rows", "both"):
            out += _quantise(x, s["block_rows"], s["q"])
        if s["layout"] in ("cols", "both"):
            out += _quantise(x.mT, s["block_rows"], s["q"])
        return out
    if s["op"] == "matmul":
        y = _values(s["a"], s["scale_a"], s["a_rows"]) @ _values(s["b"], s["scale_b"], s["b_rows"]).mT
        return (y * s["alpha"]).to(TYPES[s["out"]])
    if s["op"] == "orthogonalise":
        return _newton_schulz(s["g"].float()).to(TYPES[s["out"]])
    g = s["g"].float()
    s["momentum"].mul_(MU).add_(g)
    u = g + MU * s["momentum"] if s["nesterov"] else s["momentum"]
    s["w"].mul_(1.0 - LR * DECAY).sub_(_newton_schulz(u), alpha=LR * _scale(*g.shape))
    return s["w"], s["momentum"]


def run(state):
    s = state
    if not own:
        return _plain(s)
    from bcjr_sum_product_b200 import lib
    if s["op"] == "quantise":
        return lib.fp8_quantise(s["x"], block_rows=s["block_rows"], dtype=TYPES[s["q"]], minus=s["minus"], layout=s["layout"])
    if s["op"] == "matmul":
        return lib.fp8_matmul(s["a"], s["scale_a"], s["b"], s["scale_b"], alpha=s["alpha"], out_dtype=TYPES[s["out"]])
    if s["op"] == "orthogonalise":
        return lib.orthogonalise(s["g"], out_dtype=TYPES[s["out"]])
    return lib.muon_step(s["w"], s["g"], s["momentum"], LR, mu=MU, nesterov=s["nesterov"], weight_decay=DECAY)


def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2, "e4m3": 1, "e5m2": 1}
    if case["op"] == "quantise":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["x"]] + (4 if case["minus"] else 0) + (2 if case["layout"] == "both" else 1)), "flops": 2 * n}
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": (m + n) * k + m * n * size[case["out"]], "flops": 2 * m * n * k}
    # the two symmetric products need half of their entries
    m, n = sorted((case["rows"], case["cols"]))
    flops = case.get("batch", 1) * STEPS * (m * m * n + m * m * m + 2 * m * m * n)
    if case["op"] == "orthogonalise":
        return {"bytes": case["batch"] * m * n * (size[case["g"]] + 2), "flops": flops}
    return {"bytes": m * n * (size[case["g"]] + 16), "flops": flops}


# ---------------------------------------------------------------- 64 bits

def _exact_codes(x, rows, kind):
    """Codes and scales of a 64-bit matrix from the definition: scale 2^e with the least e >= -127 for which |x| <= largest * 2^e over the
    block, codes rounded to the nearest of the type's values, ties to the even one."""
    largest, digits, lowest = {"e4m3": (448.0, 3, -6), "e5m2": (57344.0, 2, -14)}[kind]
    r, c = x.shape
    full = torch.zeros(-(-r // rows) * rows, -(-c // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:r, :c] = x
    tall, wide = full.shape[0] // rows, full.shape[1] // BLOCK
    most = full.abs().view(tall, rows, wide, BLOCK).amax(dim=3).amax(dim=1)
    e = torch.ceil(torch.log2(most / largest))
    for step in (-1.0, 1.0):  # a logarithm may be off by an ulp next to a whole number
        other = e + step
        fits, other_fits = most <= largest * torch.exp2(e), most <= largest * torch.exp2(other)
        e = torch.where(other_fits & ((other < e) | ~fits), other, e)
    e = torch.where(most == 0, torch.zeros_like(e), e.clamp_min(-127.0))
    scale = torch.exp2(e)
    y = full / scale.repeat_interleave(rows, 0).repeat_interleave(BLOCK, 1)
    unit = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** lowest))).clamp_min(lowest) - digits)
    return (torch.round(y / unit) * unit)[:r, :c], scale


def _exact_polar(u):
    """The odd polynomial of Muon five times over, from u's definition: on the side with the shorter Gram matrix."""
    x = u / (torch.linalg.vector_norm(u, dim=(-2, -1), keepdim=True) + EPS)
    a, b, c = COEFFS
    one = torch.eye(min(x.shape[-2:]), dtype=torch.float64, device=x.device)
    for _ in range(STEPS):
        if x.shape[-2] > x.shape[-1]:
            t = torch.matmul(x.transpose(-2, -1), x)
            x = torch.matmul(x, a * one + torch.matmul(t, b * one + c * t))
        else:
            t = torch.matmul(x, x.transpose(-2, -1))
            x = torch.matmul(a * one + torch.matmul(t, b * one + c * t), x)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantise":
        # the subtraction is one of fp32 values, rounded to fp32: the operator's definition
        x = (s["x"].double() if s["minus"] is None else (s["x"].float() - s["minus"]).double())
        out = []
        if case["layout"] != "cols":
            out += _exact_codes(x, case["block_rows"], case["q"])
        if case["layout"] != "rows":
            out += _exact_codes(x.t().contiguous(), case["block_rows"], case["q"])
        return out
    if case["op"] == "matmul":
        wide = []
        for name in ("a", "b"):
            q, scale, rows = s[name].double(), s["scale_" + name].double(), case[name + "_rows"]
            i = torch.arange(q.shape[0], device=q.device) // rows
            j = torch.arange(q.shape[1], device=q.device) // BLOCK
            wide.append(q * scale[i][:, j])
        return case["alpha"] * torch.einsum("mk,nk->mn", *wide)
    if case["op"] == "orthogonalise":
        return _exact_polar(s["g"].double())
    g = s["g"].double()
    momentum = MU * s["momentum"].double() + g
    u = g + MU * momentum if case["nesterov"] else momentum
    rows, cols = case["rows"], case["cols"]
    w = s["w"].double() * (1.0 - LR * DECAY) - LR * math.sqrt(max(1.0, rows / cols)) * _exact_polar(u)
    return w, momentum
