"""Products in 8-bit floating point and the experts' layers that use them, as
cases to be timed.

Four operators, each forward and backward:

product   Y = X W^T, W in e4m3 with a scale for each 128 x 128 block, X in fp16
          and quantised in the pass with a scale for each 128 values of a row;
          backward: dX and dW of the fp16 dY, from W's transpose and from the
          X that the forward pass kept, quantised along the tokens
route     a token's experts and their weights from its logits, and the order
          that brings each expert's rows together; backward: the logits'
          gradient from the weights'
experts   the same product for rows that each go to their own expert's W;
          backward: the rows' gradient and each expert's dW
combine   a token's output from its experts' rows and weights; backward: the
          rows' and the weights' gradients

Storage.  A matrix [R, K] in F8: `codes` e4m3 [R, K up to a multiple of 128],
zero past K, and `scales` uint8 [ceil(K / 512), ceil(R / block), 4], block 1 or
128: byte j of [i, b] is the exponent + 127 of the scale of columns
128 (4 i + j) .. + 127 of rows block b .. .  A stack of matrices has one more
dimension in front of both.

A scale is the smallest power of two, and at least 2^-32, that reaches its
block's largest magnitude with 448.  Codes are quotients rounded to nearest,
ties to even.

A token's choice is made with scores in 64 bits, ties to the lowest index: the
scores of two experts are often closer than 32 bits tell apart.  An expert
whose logit is -inf is never chosen; where fewer than k remain, the others are
-1 with a weight of zero.  Slot t k + j is token t's j-th choice: `rows` lists the
slots by expert, -1 past the last; `places` is its inverse, -1 for no expert;
`offsets` says where each expert's rows begin.  Rows past the last are zeros.
"""
import math

import torch

own = False

GROUP = 128


def listed():
    return [
        # one token through a large projection: reading the weights is all
        dict(name="product one token", op="product", backward=False, m=1, n=4096, k=14336),
        # a few sequences at once, and sizes that fill no tile
        dict(name="product few tokens, ragged", op="product", backward=False, m=5, n=7001, k=4160),
        # a long prompt, or many at once: bound by the matrix units
        dict(name="product long prompt", op="product", backward=False, m=4096, n=8192, k=8192),
        # the gradients of a small layer, and of a large one over a ragged batch of tokens
        dict(name="product gradients, small", op="product", backward=True, m=256, n=1024, k=1024),
        dict(name="product gradients, ragged", op="product", backward=True, m=4999, n=8192, k=4160),
        # one token's choice among many experts in groups: the least work that a call does
        dict(name="route one token", op="route", backward=False, t=1, e=256, top=8, scores="sigmoid", groups=8, top_groups=4, bias=True, half=True, padded=False),
        # a training step's tokens, some of them padding, with the gradient
        dict(name="route training", op="route", backward=True, t=8191, e=128, top=6, scores="softmax", groups=1, top_groups=1, bias=False, half=False, padded=True),
        # one token through its experts: reading their weights is all
        dict(name="experts one token", op="experts", backward=False, t=1, e=64, top=8, n=2048, k=4096, padded=False),
        # a prompt of a few hundred tokens: every expert has some rows, none many
        dict(name="experts prompt", op="experts", backward=False, t=333, e=64, top=6, n=2048, k=4096, padded=False),
        # a training step's gradients, some tokens of it padding
        dict(name="experts gradients", op="experts", backward=True, t=4099, e=32, top=4, n=1408, k=2048, padded=True),
        # one token's output, and a training step's with its gradients
        dict(name="combine one token", op="combine", backward=False, t=1, e=64, top=8, n=4096, padded=False),
        dict(name="combine gradients", op="combine", backward=True, t=4999, e=128, top=6, n=4160, padded=True),
    ]


def _between(rng, low, high):
    """A whole number, its logarithm uniform."""
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(("product", "product", "product", "route", "experts", "experts", "combine"))
    while True:
        backward = rng.random() < 0.4
        e = rng.choice((8, 16, 32, 64, 96, 128, 160, 256))
        top = rng.randint(2, 8)
        t = _between(rng, 1, 8192)
        if op == "product":
            case = dict(op=op, backward=backward, m=t, n=_between(rng, 16, 16384), k=_between(rng, 32, 16384))
            if rng.random() < 0.6:  # most models' sizes are multiples of 64
                case.update(n=max(64, case["n"] // 64 * 64), k=max(64, case["k"] // 64 * 64))
        elif op == "route":
            groups = rng.choice((1, 1, 4, 8))
            groups = groups if e // groups >= 4 else 1
            case = dict(op=op, backward=backward, t=t, e=e, top=min(top, e // groups), scores=rng.choice(("softmax", "sigmoid")), groups=groups,
                        top_groups=rng.randint(1, groups), bias=rng.random() < 0.5, half=rng.random() < 0.5, padded=rng.random() < 0.3)
        elif op == "experts":
            case = dict(op=op, backward=backward, t=t, e=e, top=top, n=_between(rng, 64, 4096), k=_between(rng, 64, 4096), padded=rng.random() < 0.3)
            if rng.random() < 0.8:
                case.update(n=max(64, case["n"] // 64 * 64), k=max(64, case["k"] // 64 * 64))
        else:
            case = dict(op=op, backward=backward, t=t, e=e, top=top, n=_between(rng, 64, 8192), padded=rng.random() < 0.3)
        w = work(case)
        if w["flops"] <= 2 * 4096 * 8192 * 8192 and w["bytes"] <= 1.2e9 and (op != "experts" or case["e"] * case["n"] * case["k"] <= 6e8):
            return case


def _stored(r, k, block=1):
    return r * k + -(-k // GROUP) * -(-r // block)


def work(case):
    op, back = case["op"], case["backward"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        if back:
            return {"bytes": 2 * m * n + _stored(k, n, 128) + _stored(k, m) + 2 * m * k + 2 * n * k, "flops": 4 * m * n * k}
        return {"bytes": 2 * m * k + _stored(n, k, 128) + 2 * m * n, "flops": 2 * m * n * k}
    t, e, top = case["t"], case["e"], case["top"]
    slots = t * top
    order = 4 * (2 * slots + e + 1)
    if op == "route":
        logits = (2 if case["half"] else 4) * t * e
        return {"bytes": logits * (2 if back else 1) + 8 * slots + order + (4 * slots if back else 0), "flops": 20 * t * e}
    if op == "experts":
        n, k = case["n"], case["k"]
        used = e * (1 - (1 - top / e) ** t)  # experts with rows, on average
        weights = used * _stored(n, k, 128)
        if back:
            return {"bytes": 2 * slots * n + weights + 2 * t * k + 2 * slots * k + 2 * e * n * k + order, "flops": 4 * slots * n * k}
        return {"bytes": 2 * t * k + weights + 2 * slots * n + order, "flops": 2 * slots * n * k}
    n = case["n"]
    if back:
        return {"bytes": 2 * t * n * (2 + 2 * top) + 12 * slots, "flops": 5 * slots * n}
    return {"bytes": 2 * t * n * (1 + top) + 8 * slots, "flops": 2 * slots * n}


# ---- inputs ------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, t, n):
    """Normal values with some channels far larger than the rest."""
    x = _normal(g, t, n)
    x *= torch.where(torch.rand(n, generator=g, device="cuda") < 0.01, 20.0, 1.0)
    return x.half()


def _weights(g, count, r, k, block):
    """(codes, scales) of a stack of matrices in F8 whose values are about
    normal / sqrt(k)."""
    groups = -(-k // GROUP)
    codes = torch.zeros(count, r, groups * GROUP, device="cuda", dtype=torch.float8_e4m3fn)
    for i in range(count):
        codes[i, :, :k] = (100 * _normal(g, r, k)).clamp_(-448, 448).to(torch.float8_e4m3fn)
    exponent = 127 - round(math.log2(100 * math.sqrt(k)))
    bytes_ = torch.randint(exponent - 1, exponent + 2, (count, -(-r // block), groups), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return codes, _scales_stored(bytes_)


def _scales_stored(s):
    """uint8 [count, blocks of rows, groups] to the stored order."""
    count, blocks, groups = s.shape
    s = torch.nn.functional.pad(s, (0, -groups % 4), value=127)
    return s.view(count, blocks, -1, 4).transpose(1, 2).contiguous()


def _padding(g, t):
    """Which tokens are padding: some in the middle and the end of the batch."""
    pad = torch.rand(t, generator=g, device="cuda") < 0.02
    pad[t - t // 16:] = True
    return pad


def _some_routing(g, case):
    """Experts of each token by random scores, some experts more sought than
    others, and all that follows from them."""
    t, e, top = case["t"], case["e"], case["top"]
    score = _normal(g, t, e) + 0.5 * _normal(g, e)
    experts = score.sort(dim=1, descending=True, stable=True).indices[:, :top].int().contiguous()
    weights = torch.rand(t, top, generator=g, device="cuda") + 0.1
    weights /= weights.sum(1, keepdim=True)
    if case["padded"]:
        pad = _padding(g, t)
        experts[pad] = -1
        weights[pad] = 0
    return (experts, weights) + _plain_order(experts, e)


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    state = dict(case)
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        if case["backward"]:
            state["dy"] = (_normal(g, m, n) / math.sqrt(m)).half()
            state["wt"] = _weights(g, 1, k, n, 128)
            state["xt"] = _weights(g, 1, k, m, 1)
        else:
            state["x"] = _activations(g, m, k)
            state["w"] = _weights(g, 1, n, k, 128)
    elif op == "route":
        t, e = case["t"], case["e"]
        logits = 1.5 * _normal(g, t, e)
        if case["padded"]:
            logits[_padding(g, t)] = -math.inf
        state["logits"] = logits.half() if case["half"] else logits
        state["bias_values"] = 0.1 * _normal(g, e) if case["bias"] else None
        if case["backward"]:
            state["dweights"] = _normal(g, t, case["top"])
    else:
        t, n = case["t"], case["n"]
        state["routing"] = _some_routing(g, case)
        offsets = state["bounds"] = state["routing"][4].tolist()
        slots = t * case["top"]
        if op == "experts":
            k, e = case["k"], case["e"]
            if case["backward"]:
                state["dy"] = (_normal(g, slots, n) / math.sqrt(slots / e)).half()
                state["x"] = _activations(g, t, k)
                state["wt"] = _weights(g, e, k, n, 128)
            else:
                state["x"] = _activations(g, t, k)
                state["w"] = _weights(g, e, n, k, 128)
        else:
            state["y"] = _normal(g, slots, n).half()
            state["y"][offsets[-1]:] = 0
            if case["backward"]:
                state["dout"] = _normal(g, t, n).half()
    if own:  # the handles that a program keeps: the same tensors, with their sizes
        import dense_fp16_gemm_amd as lib

        if op == "product":
            if case["backward"]:
                state["wt8"] = lib.F8Matrix(state["wt"][0][0], state["wt"][1][0], case["n"], 128)
                state["xt8"] = lib.F8Matrix(state["xt"][0][0], state["xt"][1][0], case["m"], 1)
            else:
                state["w8"] = lib.F8Matrix(state["w"][0][0], state["w"][1][0], case["k"], 128)
        elif op != "route":
            state["route"] = lib.Routing(*state["routing"])
            if op == "experts" and case["backward"]:
                state["wt8"] = lib.F8Matrix(*state["wt"], case["n"], 128)
            elif op == "experts":
                state["w8"] = lib.F8Matrix(*state["w"], case["k"], 128)
    return state


# ---- one pass ----------------------------------------------------------------
def run(state):
    op = state["op"]
    return (_own if own else _plain)[op](state)


def _own_product(state):
    import dense_fp16_gemm_amd as lib

    if not state["backward"]:
        return lib.gemm_nt_f8(state["x"], state["w8"])
    dy = state["dy"]
    return lib.gemm_nt_f8(dy, state["wt8"]), lib.gemm_nt_f8(lib.quantize_f8(dy, transposed=True), state["xt8"])


def _own_route(state):
    import dense_fp16_gemm_amd as lib

    r = lib.route(state["logits"], state["top"], scores=state["scores"], bias=state["bias_values"], groups=state["groups"], top_groups=state["top_groups"], scale=2.5)
    out = r.experts, r.weights, r.rows, r.places, r.offsets
    return out + (lib.route_backward(state["logits"], r, state["dweights"]),) if state["backward"] else out


def _own_experts(state):
    import dense_fp16_gemm_amd as lib

    r = state["route"]
    if not state["backward"]:
        return lib.gemm_nt_f8_experts(state["x"], state["w8"], r, gather=True)
    dx = lib.gemm_nt_f8_experts(state["dy"], state["wt8"], r)
    dy8, x8 = lib.quantize_f8_experts(state["dy"], r), lib.quantize_f8_experts(state["x"], r, gather=True)
    return dx, lib.gemm_nt_f8_experts_grad(dy8, x8, r)


def _own_combine(state):
    import dense_fp16_gemm_amd as lib

    r = state["route"]
    if not state["backward"]:
        return lib.combine_experts(state["y"], r)
    return (lib.combine_experts(state["y"], r),) + lib.combine_experts_backward(state["dout"], state["y"], r)


_own = dict(product=_own_product, route=_own_route, experts=_own_experts, combine=_own_combine)


def _plain_round(x):
    """x [rows, k] in the values that its quantised form stands for, a scale for
    each 128 of a row."""
    rows, k = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -k % GROUP)).view(rows, -1, GROUP)
    m, e = torch.frexp(v.abs().amax(-1).clamp(min=2.0 ** -24))   # 448 = 0.875 2^9
    s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).int())[:, :, None]
    return ((v / s).to(torch.float8_e4m3fn).float() * s).view(rows, -1)[:, :k]


def _plain_values(stored, k, block):
    """A stored matrix [R, k] in fp32."""
    codes, scales = stored
    s = scales.transpose(0, 1).reshape(scales.shape[1], -1)[:, : codes.shape[1] // GROUP]
    s = torch.ldexp(torch.ones_like(s, dtype=torch.float32), s.int() - 127).repeat_interleave(block, 0)[: codes.shape[0]]
    return (codes.float().view(codes.shape[0], -1, GROUP) * s[:, :, None]).view(codes.shape[0], -1)[:, :k]


def _plain_product(state):
    m, n, k = state["m"], state["n"], state["k"]
    if not state["backward"]:
        return (_plain_round(state["x"]) @ _plain_values([v[0] for v in state["w"]], k, 128).t()).half()
    wt, xt = _plain_values([v[0] for v in state["wt"]], n, 128), _plain_values([v[0] for v in state["xt"]], m, 1)
    dx = _plain_round(state["dy"]) @ wt.t()
    dw = _plain_round(state["dy"].t()) @ xt.t()
    return dx.half(), dw.half()


def _plain_order(experts, e):
    t, top = experts.shape
    flat = experts.reshape(-1).long()
    order = torch.where(flat < 0, e, flat).sort(stable=True)
    offsets = torch.searchsorted(order.values, torch.arange(e + 1, device=flat.device)).int()
    here = order.values < e
    rows = torch.where(here, order.indices, -1).int()
    places = torch.full_like(rows, -1)
    places[order.indices] = torch.where(here, torch.arange(t * top, device=flat.device), -1).int()
    return rows, places.view(t, top), offsets


def _plain_route(state):
    e, top, groups = state["e"], state["top"], state["groups"]
    x = state["logits"].double()
    masked = x == -math.inf
    if state["scores"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
        total = p.sum(1, keepdim=True)
        score = p / torch.where(total > 0, total, 1.0)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score if state["bias_values"] is None else score + state["bias_values"].double()
    choice = torch.where(masked, -math.inf, choice)
    if groups > 1:
        best = choice.view(-1, groups, e // groups).sort(dim=2, descending=True).values[:, :, :2]
        best = torch.where(torch.isinf(best[:, :, :1]), best[:, :, 0:1], torch.where(torch.isinf(best), 0.0, best)).sum(2)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : state["top_groups"]]
        inside = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(inside.repeat_interleave(e // groups, 1), choice, -math.inf)
    order = choice.sort(dim=1, descending=True, stable=True)
    experts = order.indices[:, :top]
    none = order.values[:, :top] == -math.inf
    chosen = torch.where(none, 0.0, score.gather(1, experts))
    total = chosen.sum(1, keepdim=True) + 1e-20
    weights = (2.5 * chosen / total).float()
    experts = torch.where(none, -1, experts).int()
    out = (experts, weights) + _plain_order(experts, e)
    if not state["backward"]:
        return out
    dw = state["dweights"].double()
    ds = 2.5 / total * (dw - (dw * chosen).sum(1, keepdim=True) / total)
    ds = torch.zeros_like(score).scatter_add_(1, experts.clamp(min=0).long(), torch.where(none, 0.0, ds))
    if state["scores"] == "softmax":
        dx = score * (ds - (score * ds).sum(1, keepdim=True))
    else:
        dx = ds * score * (1 / (1 + torch.exp(x)))
    return out + (dx.to(state["logits"].dtype),)


def _plain_experts(state):
    top, bounds = state["top"], state["bounds"]
    rows = state["routing"][2]
    tokens = rows[: bounds[-1]].long() // top
    if not state["backward"]:
        x = _plain_round(state["x"])[tokens]
        y = torch.zeros(rows.numel(), state["n"], device="cuda", dtype=torch.float16)
        for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
            if b > a:
                y[a:b] = (x[a:b] @ _plain_values([v[e] for v in state["w"]], state["k"], 128).t()).half()
        return y
    dy = _plain_round(state["dy"])
    dx = torch.zeros(rows.numel(), state["k"], device="cuda", dtype=torch.float16)
    dw = torch.zeros(state["e"], state["n"], state["k"], device="cuda", dtype=torch.float16)
    for e, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            dx[a:b] = (dy[a:b] @ _plain_values([v[e] for v in state["wt"]], state["n"], 128).t()).half()
            dw[e] = (_plain_round(state["dy"][a:b].t()) @ _plain_round(state["x"][tokens[a:b]].t()).t()).half()
    return dx, dw


def _plain_combine(state):
    experts, weights, _, places, _ = state["routing"]
    t, top = weights.shape
    at = places.clamp(min=0).long()
    w = weights[:, :, None]
    y = state["y"][at].float() * (places >= 0)[:, :, None]
    out = (w * y).sum(1).half()
    if not state["backward"]:
        return out
    dout = state["dout"].float()[:, None, :]
    dy = torch.zeros(t * top + 1, state["n"], device="cuda", dtype=torch.float16)
    dy[torch.where(places < 0, t * top, places).long()] = (w * dout * (places >= 0)[:, :, None]).half()
    dw = (dout.double() * y.double()).sum(2).float()
    return out, dy[: t * top], dw


_plain = dict(product=_plain_product, route=_plain_route, experts=_plain_experts, combine=_plain_combine)


# ---- the definition, in 64 bits ----------------------------------------------
def _exact_round(x):
    """Rows quantised and read back, group by group and with the rounding to a
    multiple of the code's last place written out."""
    x = x.double()
    out = torch.empty_like(x)
    for first in range(0, x.shape[1], GROUP):
        v = x[:, first: first + GROUP]
        s = torch.exp2(torch.ceil(torch.log2(v.abs().max(dim=1, keepdim=True).values.clamp(min=2.0 ** -24) / 448)))
        q = v / s
        place = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        out[:, first: first + GROUP] = torch.round(q / place) * place * s
    return out


def _exact_values(codes, scales, k, block):
    r = torch.arange(codes.shape[0], device=codes.device)[:, None] // block
    group = torch.arange(k, device=codes.device)[None, :] // GROUP
    return codes[:, :k].double() * torch.exp2(scales[group // 4, r, group % 4].double() - 127)


def _times(a, b):
    return torch.matmul(a, b.t().contiguous())


def _exact_choice(x, score, bias, case):
    """Experts of each token, by taking the highest over and over."""
    t, e = x.shape
    per = e // case["groups"]
    c = score if bias is None else score + bias.double()
    c = torch.where(x == -math.inf, -math.inf, c)
    index = torch.arange(e, device=x.device)[None, :]

    def take(values, places):
        highest = values.max(dim=1, keepdim=True).values
        first = torch.where(values == highest, places, values.shape[1]).min(dim=1, keepdim=True).values
        return highest, first

    if case["groups"] > 1:
        total = torch.zeros(t, case["groups"], device=x.device, dtype=torch.float64)
        for group in range(case["groups"]):
            part = c[:, group * per: group * per + per]
            high, at = take(part, index[:, :per])
            second = take(torch.where(index[:, :per] == at, -math.inf, part), index[:, :per])[0]
            total[:, group: group + 1] = high + torch.where(second == -math.inf, 0.0, second)
        keep = torch.zeros(t, e, device=x.device, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            at = take(total, index[:, : case["groups"]])[1]
            keep |= index // per == at
            total = torch.where(index[:, : case["groups"]] == at, -math.inf, total)
        c = torch.where(keep, c, -math.inf)
    experts = torch.full((t, case["top"]), -1, device=x.device, dtype=torch.int64)
    for j in range(case["top"]):
        high, at = take(c, index)
        experts[:, j: j + 1] = torch.where(high == -math.inf, -1, at)
        c = torch.where(index == at, -math.inf, c)
    return experts


def _exact_route(state):
    x = state["logits"].double()
    masked = x == -math.inf
    if state["scores"] == "softmax":
        top = torch.where(masked, -1e4, x).max(dim=1, keepdim=True).values
        score = torch.where(masked, 0.0, torch.exp(x - top))
        score = score / score.sum(dim=1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1 / (1 + torch.exp(-x))
    experts = _exact_choice(x, score, state["bias_values"], state)
    picked = torch.zeros_like(score).scatter(1, experts.clamp(min=0), 1.0)
    picked = torch.where((experts < 0).all(1, keepdim=True), 0.0, picked)   # in these cases all or none are -1
    some = (experts >= 0).double()
    total = (score * picked).sum(1, keepdim=True) + 1e-20
    w = 2.5 * score * picked / total
    weights = w.gather(1, experts.clamp(min=0)) * some
    flat = experts.reshape(-1)
    slots = torch.arange(flat.numel(), device=x.device)
    key = torch.where(flat < 0, state["e"], flat) * flat.numel() + slots
    rows = key.argsort()
    here = flat[rows] >= 0
    places = torch.empty_like(rows)
    places[rows] = torch.where(here, slots, -1)
    offsets = torch.zeros(state["e"] + 1, device=x.device, dtype=torch.int64)
    offsets[1:] = torch.bincount(flat[flat >= 0], minlength=state["e"]).cumsum(0)
    out = experts.int(), weights, torch.where(here, rows, -1).int(), places.view_as(experts).int(), offsets.int()
    if not state["backward"]:
        return out
    dw = torch.zeros_like(score).scatter(1, experts.clamp(min=0), state["dweights"].double()) * picked
    ds = 2.5 * picked * (dw / total - (dw * score).sum(1, keepdim=True) / total ** 2)
    if state["scores"] == "softmax":
        dx = ds * score - score * (ds * score).sum(1, keepdim=True)
    else:
        dx = ds * score / (1 + torch.exp(x))
    return out + (torch.where(masked, 0.0, dx),)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        return _exact_route(state)
    n = case["n"]
    if op == "product":
        m, k = case["m"], case["k"]
        if not case["backward"]:
            return _times(_exact_round(state["x"]), _exact_values(state["w"][0][0], state["w"][1][0], k, 128))
        dx = _times(_exact_round(state["dy"]), _exact_values(state["wt"][0][0], state["wt"][1][0], n, 128))
        dw = _times(_exact_round(state["dy"].t()), _exact_values(state["xt"][0][0], state["xt"][1][0], m, 1))
        return dx, dw
    experts, weights, _, places, _ = state["routing"]
    flat = experts.reshape(-1).long()
    top = case["top"]
    if op == "experts":
        slots, k = flat.numel(), case["k"]
        where = places.reshape(-1).long()
        y = torch.zeros(slots, k if case["backward"] else n, device="cuda", dtype=torch.float64)
        dw = torch.zeros(case["e"], n, k, device="cuda", dtype=torch.float64) if case["backward"] else None
        x8 = None if case["backward"] else _exact_round(state["x"])
        for e in range(case["e"]):
            mine = (flat == e).nonzero()[:, 0]   # slots of this expert, ascending
            if not mine.numel():
                continue
            if case["backward"]:
                dy = state["dy"][where[mine]]
                y[where[mine]] = _times(_exact_round(dy), _exact_values(state["wt"][0][e], state["wt"][1][e], n, 128))
                dw[e] = _times(_exact_round(dy.t()), _exact_round(state["x"][mine // top].t()))
            else:
                y[where[mine]] = _times(x8[mine // top], _exact_values(state["w"][0][e], state["w"][1][e], k, 128))
        return (y, dw) if case["backward"] else y
    t = case["t"]
    out = torch.zeros(t, n, device="cuda", dtype=torch.float64)
    dy = torch.zeros(t * top, n, device="cuda", dtype=torch.float64)
    dw = torch.zeros(t, top, device="cuda", dtype=torch.float64)
    for j in range(top):
        some = (experts[:, j] >= 0).nonzero()[:, 0]
        place = places[some, j].long()
        w = weights[some, j].double()[:, None]
        y = state["y"][place].double()
        out[some] += w * y
        if case["backward"]:
            dout = state["dout"][some].double()
            dy[place] = w * dout
            dw[some, j] = (dout * y).sum(1)
    return (out, dy, dw) if case["backward"] else out
