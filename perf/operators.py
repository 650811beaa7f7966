"""The products with operands held in 4 and 8 bits, as cases to be timed.

Four operators:

w4_product   C = A W^T with W in 4-bit codes and one scale for each group of
             `group` weights of a row: serving, from one token to a prompt
w4_values    a weight matrix quantised to 4 bits, and the values that it then
             stands for: what a program does once when it loads a model
q8_values    activations stored in 8 bits (a scale for each 32 neighbours of a
             row), and read back: a checkpoint saved and restored
q8_gradient  C = A^T X with X such a checkpoint: a layer's weight gradient

Storage.  4 bits: `words` int32 [N/16, K/128, 64, 4] (both rounded up, absent
weights zero).  Word j of lane l of tile (b, t) holds the eight weights of row
16 b + l % 16 at columns 128 t + 32 j + 8 (l / 16) + i, i = 0..7: code + 8 in
the four bits from 16 (i % 2) + 4 (i / 2).  `scales` fp16 [N/16, columns of the
tiles / group, 16], each of at most 8 significant bits, so that a scale times a
code is exact in fp16.  8 bits: `codes` int8 [T, N up to a multiple of 32] and
`scales` fp16 [T, N/32], of at most 4 significant bits.

A group's scale is the smallest such number (a multiple of 2^-24) that reaches
the group's largest magnitude with the largest code: 7 (at most 9344) or 127.
Codes are quotients rounded to nearest, ties to even, and one lower in
magnitude where their value would pass fp16's largest.
"""
import math

import torch

own = False

GROUP8 = 32


def listed():
    return [
        # the least work that a call does: a small projection for one token
        dict(name="w4 one token, small", op="w4_product", m=1, n=1024, k=1024, group=32),
        # one token through a large projection: reading the weights is all
        dict(name="w4 one token", op="w4_product", m=1, n=4096, k=14336, group=128),
        # a few sequences at once, and sizes that fill no tile
        dict(name="w4 few tokens, ragged", op="w4_product", m=5, n=7001, k=4160, group=64),
        # a full decoding batch
        dict(name="w4 batch", op="w4_product", m=48, n=16384, k=16384, group=128),
        # a prompt of ordinary length
        dict(name="w4 prompt", op="w4_product", m=333, n=4096, k=14336, group=128),
        # a long prompt, or many at once: bound by the matrix units
        dict(name="w4 long prompt", op="w4_product", m=4096, n=8192, k=8192, group=128),
        # a small layer's weights, and a large one's, quantised when a model is loaded
        dict(name="w4 values, small", op="w4_values", n=256, k=256, group=32),
        dict(name="w4 values", op="w4_values", n=8192, k=8192, group=128),
        # activations of a few tokens, and of a training step with ragged sizes, saved and restored
        dict(name="q8 values, small", op="q8_values", t=64, n=4096),
        dict(name="q8 values, ragged", op="q8_values", t=4999, n=7001),
        # the gradient of a low-rank adapter, and of a whole layer over a ragged batch of tokens
        dict(name="q8 gradient, adapter", op="q8_gradient", m=16, n=4096, t=8192),
        dict(name="q8 gradient, layer", op="q8_gradient", m=8192, n=4160, t=4999),
    ]


def _between(rng, low, high):
    """A whole number, its logarithm uniform."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(("w4_product", "w4_product", "w4_product", "w4_values", "q8_values", "q8_gradient", "q8_gradient"))
    while True:
        if op == "w4_product":
            case = dict(op=op, m=_between(rng, 1, 4096), n=_between(rng, 16, 16384), k=_between(rng, 32, 16384), group=rng.choice((32, 64, 128)))
            if rng.random() < 0.6:  # most models' sizes are multiples of 64
                case.update(n=max(64, case["n"] // 64 * 64), k=max(64, case["k"] // 64 * 64))
        elif op == "w4_values":
            case = dict(op=op, n=_between(rng, 16, 8192), k=_between(rng, 32, 8192), group=rng.choice((32, 64, 128)))
        elif op == "q8_values":
            case = dict(op=op, t=_between(rng, 1, 8192), n=_between(rng, 32, 14336))
        else:
            case = dict(op=op, m=_between(rng, 8, 8192), n=_between(rng, 64, 8192), t=_between(rng, 1, 8192))
            if rng.random() < 0.6:
                case.update(m=max(16, case["m"] // 16 * 16), n=max(64, case["n"] // 64 * 64))
        w = work(case)
        if w["flops"] <= 2 * 4096 * 8192 * 8192 // 2 and w["bytes"] <= 3e8:
            return case


def work(case):
    op = case["op"]
    if op == "w4_product":
        m, n, k = case["m"], case["n"], case["k"]
        weights = n * k / 2 + 2 * n * -(-k // case["group"])
        return {"bytes": weights + 2 * (m * k + m * n), "flops": 2 * m * n * k}
    if op == "w4_values":
        n, k = case["n"], case["k"]
        weights = n * k / 2 + 2 * n * -(-k // case["group"])
        return {"bytes": 2 * n * k + weights + 2 * n * k, "flops": 4 * n * k}
    t, n = case["t"], case["n"]
    stored = t * n + 2 * t * -(-n // GROUP8)
    if op == "q8_values":
        return {"bytes": 2 * t * n + stored + 2 * t * n, "flops": 4 * t * n}
    return {"bytes": 2 * t * case["m"] + stored + 2 * case["m"] * n, "flops": 2 * case["m"] * n * t}


# ---- inputs ------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, t, n):
    """Normal values with some channels far larger than the rest, and a few
    tokens that are padding."""
    x = _normal(g, t, n)
    x *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    x *= (torch.rand(t, 1, generator=g, device="cuda") >= 0.02)
    return x.half()


def _keep_bits(x, drop):
    """fp16 values without the last `drop` bits of their significand."""
    return (x.half().view(torch.int16) & -(1 << drop)).view(torch.float16)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = dict(case)
    if op == "w4_product":
        m, n, k, group = case["m"], case["n"], case["k"], case["group"]
        nb, kt = -(-n // 16), -(-k // 128)
        codes = torch.zeros(16 * nb, 128 * kt, device="cuda", dtype=torch.int32)
        codes[:n, :k] = (2.5 * _normal(g, n, k)).round_().clamp_(-8, 7).int()
        # [b, r, t, j, q, h, p]: row r of block b; column 32 j + 8 q + 2 h + p of tile t
        codes = codes.add_(8).view(nb, 16, kt, 4, 4, 4, 2)
        words = torch.zeros(nb, 16, kt, 4, 4, device="cuda", dtype=torch.int32)
        for h in range(4):
            for p in range(2):
                words |= codes[..., h, p] << (16 * p + 4 * h)
        del codes
        state["words"] = words.permute(0, 2, 4, 1, 3).contiguous().view(nb, kt, 64, 4)
        groups = -(-k // group)
        scales = torch.zeros(nb * 16, 128 * kt // group, device="cuda", dtype=torch.float16)
        scales[:n, :groups] = _keep_bits((0.5 + torch.rand(n, groups, generator=g, device="cuda")) / (2.5 * math.sqrt(k)), 3)
        state["scales"] = scales.view(nb, 16, -1).permute(0, 2, 1).contiguous()
        state["a"] = _normal(g, m, k).half()
    elif op == "w4_values":
        state["w"] = (_normal(g, case["n"], case["k"]) / math.sqrt(case["k"])).half()
    elif op == "q8_values":
        state["x"] = _activations(g, case["t"], case["n"])
    else:
        t, n = case["t"], case["n"]
        groups = -(-n // GROUP8)
        codes = torch.zeros(t, groups * GROUP8, device="cuda", dtype=torch.int8)
        codes[:, :n] = (45 * _normal(g, t, n)).round_().clamp_(-127, 127).to(torch.int8)
        state["codes"] = codes
        state["scales"] = _keep_bits((0.5 + torch.rand(t, groups, generator=g, device="cuda")) / 45, 7)
        state["a"] = (_normal(g, t, case["m"]) / math.sqrt(t)).half()
    if own:  # the handles that a program keeps: the same tensors, with their sizes
        import dense_fp16_gemm_amd as lib

        if op == "w4_product":
            state["handle"] = lib.W4Matrix(state["words"], state["scales"], case["n"], case["k"], case["group"])
        elif op == "q8_gradient":
            state["handle"] = lib.Q8Matrix(state["codes"], state["scales"], case["n"])
    return state


# ---- one pass ----------------------------------------------------------------
def run(state):
    op = state["op"]
    if own:
        import dense_fp16_gemm_amd as lib

        if op == "w4_product":
            return lib.gemm_nt_w4(state["a"], state["handle"])
        if op == "w4_values":
            return lib.dequantize_w4(lib.quantize_w4(state["w"], state["group"]))
        if op == "q8_values":
            return lib.dequantize_q8(lib.quantize_q8(state["x"]))
        return lib.gemm_tn_q8(state["a"], state["handle"])
    if op == "w4_product":
        return (state["a"].float() @ _plain_w4(state).t()).half()
    if op == "w4_values":
        return _plain_round(state["w"], state["group"], 8, 7, 9344.0)
    if op == "q8_values":
        return _plain_round(state["x"], GROUP8, 4, 127, 576.0)
    n = state["n"]
    x = state["codes"].float().view(state["t"], -1, GROUP8) * state["scales"].float()[:, :, None]
    return (state["a"].float().t() @ x.view(state["t"], -1)[:, :n]).half()


def _plain_w4(state):
    """W in fp32 from its words and scales."""
    words, scales = state["words"], state["scales"]
    nb, kt = words.shape[:2]
    at = torch.tensor([16 * (i % 2) + 4 * (i // 2) for i in range(8)], device=words.device, dtype=torch.int32)
    codes = ((words[..., None] >> at) & 15) - 8                     # [b, t, lane, j, i]
    codes = codes.view(nb, kt, 4, 16, 4, 8).permute(0, 3, 1, 4, 2, 5)  # [b, r, t, j, q, i]
    w = codes.reshape(nb * 16, -1, state["group"]).float() * scales.permute(0, 2, 1).reshape(nb * 16, -1, 1).float()
    return w.view(nb * 16, -1)[: state["n"], : state["k"]]


def _plain_round(x, group, bits, top, most):
    """x rounded to codes of up to `top` and back: the scale is found among all
    the numbers of so many bits."""
    rows, cols = x.shape
    few = torch.arange(1, 2 ** bits, device=x.device, dtype=torch.float32) * 2.0 ** -24
    more = torch.arange(2 ** (bits - 1), 2 ** bits, device=x.device, dtype=torch.float32)
    exponents = torch.tensor([2.0 ** e for e in range(-23, 9)], device=x.device, dtype=torch.float32)
    scales = torch.cat([few, (exponents[:, None] * more).view(-1)])
    scales = scales[scales <= most]
    v = torch.nn.functional.pad(x.float(), (0, -cols % group)).view(rows, -1, group)
    largest = v.abs().amax(-1)
    s = scales[torch.searchsorted(scales * top, largest).clamp_(max=scales.numel() - 1)]
    limit = torch.floor(65504.0 / s).clamp(max=top)[:, :, None]
    code = (v.double() / s[:, :, None].double()).round().float()  # in 64 bits: quotients lie on ties
    code = torch.minimum(torch.maximum(code, -limit), limit)
    return (code * s[:, :, None]).view(rows, -1)[:, :cols].half()


# ---- the definition, in 64 bits ----------------------------------------------
def _exact_values(x, group, bits, top, most):
    rows, cols = x.shape
    x = x.double()
    out = torch.empty_like(x)
    for first in range(0, cols, group):
        v = x[:, first : first + group]
        need = v.abs().max(dim=1, keepdim=True).values / top
        _, exponent = torch.frexp(need.clamp(min=2.0 ** -24))       # need = m 2^exponent, 1/2 <= m < 1
        step = (exponent.long() - bits + 1023 << 52).view(torch.float64).clamp(min=2.0 ** -24)
        s = (torch.ceil(need / step) * step).clamp(2.0 ** -24, most)
        code = torch.round(v / s)
        code = torch.where((code * s).abs() > 65504, code - torch.sign(code), code)
        out[:, first : first + group] = code * s
    return out


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "w4_values":
        return _exact_values(state["w"], case["group"], 8, 7, 9344.0)
    if op == "q8_values":
        return _exact_values(state["x"], GROUP8, 4, 127, 576.0)
    if op == "w4_product":
        n, k = case["n"], case["k"]
        kt = -(-k // 128)
        row = torch.arange(n, device="cuda")[:, None]
        col = torch.arange(k, device="cuda")[None, :]
        word = ((row // 16 * kt + col // 128) * 64 + col % 32 // 8 * 16 + row % 16) * 4 + col % 128 // 32
        w = state["words"].reshape(-1)[word] >> (col % 2 * 16 + col % 8 // 2 * 4)
        w = (w & 15).double() - 8
        del word
        groups = state["scales"].shape[1]
        w *= state["scales"].reshape(-1)[(row // 16 * groups + col // case["group"]) * 16 + row % 16].double()
        return torch.matmul(state["a"].double(), w.t())
    out = torch.zeros(case["m"], case["n"], device="cuda", dtype=torch.float64)
    for first in range(0, case["t"], 1024):
        part = slice(first, first + 1024)
        x = state["codes"][part, : case["n"]].double()
        x *= state["scales"][part].double().repeat_interleave(GROUP8, 1)[:, : case["n"]]
        out += torch.matmul(state["a"][part].double().t().contiguous(), x)
    return out
