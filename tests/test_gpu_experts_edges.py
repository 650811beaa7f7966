"""8-bit products and layers of experts as programs use them: at the edges of what
their headers allow, on other streams, saved and read back, all steps together."""
import copy
import os
import pickle
import subprocess
import sys

import numpy as np
import pytest
import torch

import f8_ref as ref
from test_gpu_experts import layer, layer_inputs
from test_gpu_f8 import dev, g, host  # noqa: F401  (g: the fixture)

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- rows of nearly 2^31 columns -------------------------------------------------
WIDEST = 2 ** 31 - 8     # the last of a wave's steps of 2048 columns ends past 2^31


def widest_row():
    """One row of small whole numbers."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    part = torch.randint(-2, 3, (2 ** 28,), device="cuda", generator=gen).half()
    x = torch.empty(1, WIDEST, dtype=torch.float16, device="cuda")
    for at in range(0, WIDEST, 2 ** 28):
        x[0, at:at + 2 ** 28] = part[: WIDEST - at]
    return x


def guarded_row():
    """A row's memory, and what lies around it."""
    memory = torch.full((WIDEST + 8192,), 3.0, dtype=torch.float16, device="cuda")
    return memory[4096:4096 + WIDEST].view(1, WIDEST), (memory[:4096], memory[4096 + WIDEST:])


def test_combine_widest(g):
    """One token, one choice, as many columns as a call takes: both directions."""
    x = widest_row()
    r = g.route(torch.zeros(1, 1, device="cuda"), 1, scale=0.5)
    assert r.places.tolist() == [[0]] and r.weights.tolist() == [[0.5]]
    out, around = guarded_row()
    g.combine_experts(x, r, out=out)
    half = x * 0.5
    assert torch.equal(out, half)
    # the inner product: of the first and the last columns, so that it is a small whole number
    y = torch.zeros_like(x)
    ends = (slice(0, 4096), slice(WIDEST - 4096, WIDEST))
    for part in ends:
        y[0, part] = x[0, part]
    out.fill_(9.0)
    dw = torch.zeros(1, 1, device="cuda")
    g.gemm_f16_combine_backward(1, 1, WIDEST, x.data_ptr(), y.data_ptr(), r.weights.data_ptr(), r.rows.data_ptr(),
                                r.places.data_ptr(), out.data_ptr(), dw.data_ptr(), stream())
    assert torch.equal(out, half)
    assert dw.item() == sum((x[0, part].double() ** 2).sum().item() for part in ends)
    assert all((v == 3).all() for v in around)


def test_combine_widest_of_no_expert(g):
    """The same for a token without an expert: a row of zeros."""
    x = torch.ones(1, WIDEST, dtype=torch.float16, device="cuda")
    r = g.route(torch.full((1, 1), -torch.inf, device="cuda"), 1)
    assert r.places.tolist() == [[-1]] and r.rows.tolist() == [-1]
    out, around = guarded_row()
    g.gemm_f16_combine_backward(1, 1, WIDEST, x.data_ptr(), 0, 0, r.rows.data_ptr(), r.places.data_ptr(),
                                out.data_ptr(), 0, stream())
    assert torch.count_nonzero(out).item() == 0
    out.fill_(9.0)
    g.combine_experts(x, r, out=out)
    assert torch.count_nonzero(out).item() == 0
    assert all((v == 3).all() for v in around)


# ---- nothing, and more than 32 bits ----------------------------------------------------
@pytest.mark.parametrize("t,top", [(0, 1), (0, 3), (5, 2)])
def test_layer_of_nothing(g, t, top):
    """No tokens, or none that has an expert: gradients of weights are 0, the rest is
    empty or 0."""
    e, n, k = 4, 130, 200
    logits = torch.full((t, e), -torch.inf, device="cuda")
    x = torch.ones(t, k, dtype=torch.float16, device="cuda")
    w8 = g.quantize_f8(torch.ones(e, n, k, dtype=torch.float16, device="cuda"), 128)
    wt8 = g.quantize_f8(torch.ones(e, n, k, dtype=torch.float16, device="cuda"), 128, transposed=True)
    r = g.route(logits, top)
    assert r.experts.shape == r.weights.shape == r.places.shape == (t, top) and r.rows.shape == (t * top,)
    assert r.offsets.tolist() == [0] * (e + 1)
    for a in (x, g.quantize_f8(x)):
        y = g.gemm_nt_f8_experts(a, w8, r, gather=True)
        assert y.shape == (t * top, n) and (y == 0).all()
    out = g.combine_experts(y, r)
    assert out.shape == (t, n) and (out == 0).all()
    dout = torch.ones(t, n, dtype=torch.float16, device="cuda")
    dy, dw = g.combine_experts_backward(dout, y, r)
    assert dy.shape == y.shape and (dy == 0).all() and dw.shape == (t, top) and (dw == 0).all()
    dlogits = g.route_backward(logits, r, dw)
    assert dlogits.shape == (t, e) and (dlogits == 0).all()
    dx = g.combine_experts(g.gemm_nt_f8_experts(dy, wt8, r), r, weighted=False)
    assert dx.shape == (t, k) and (dx == 0).all()
    dy8, x8 = g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True)
    grad = g.gemm_nt_f8_experts_grad(dy8, x8, r, out=torch.full((e, n, k), 9.0, dtype=torch.float16, device="cuda"))
    assert (grad == 0).all()


def test_rows_beyond_32_bits(g):
    """Experts' rows past 2^32 bytes, and past 2^32 codes: combined, their gradients, and
    the products' operands and outputs."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    t, e, top, n, k = 300000, 8, 4, 4160, 96
    r = g.route(torch.randn(t, e, device="cuda", generator=gen), top)
    assert t * top * n > 2 ** 32
    some = torch.cat((torch.arange(0, 200), torch.arange(t - 200, t))).cuda()
    w = torch.randint(-2, 3, (e, k, n), device="cuda", generator=gen).half()
    y = torch.empty(t * top, n, dtype=torch.float16, device="cuda")
    for part in y.split(2 ** 16):
        part.copy_(torch.randint(-2, 3, part.shape, generator=gen, device="cuda", dtype=torch.int8))
    # a token's rows together: whole numbers
    sums = y[r.places[some].long()].double().sum(1)
    assert torch.equal(g.combine_experts(y, r, weighted=False)[some].double(), sums)
    # the rows' products, K past 2^32 codes
    c = g.gemm_nt_f8_experts(y, g.quantize_f8(w, 128), r)
    experts, places = r.experts[some].long(), r.places[some].long()
    want = torch.stack([torch.matmul(w[i].double(), v.double()) for i, v in
                        zip(experts.view(-1).tolist(), y[places.view(-1)])])
    assert torch.equal(c[places.view(-1)], want.half())
    del c
    # the weights' gradients, of few rows that are not zero
    dc = torch.zeros(t * top, k, dtype=torch.float16, device="cuda")
    on = places[::40].reshape(-1)
    dc[on] = torch.randint(-2, 3, (on.numel(), k), generator=gen, device="cuda").half()
    y8 = g.quantize_f8_experts(y, r)
    assert y8.codes.numel() > 2 ** 32
    grad = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dc, r), y8, r)
    want = torch.zeros(e, k, n, dtype=torch.float64, device="cuda")
    for at, i in zip(on.tolist(), experts[::40].reshape(-1).tolist()):
        want[i] += dc[at].double()[:, None] * y[at].double()
    assert torch.equal(grad, want.half())
    del y8
    # outputs past 2^32 bytes, and the gradients of the combination
    wt8 = g.quantize_f8(w, 128, transposed=True)
    rows = g.gemm_nt_f8_experts(dc, wt8, r)
    want = torch.stack([torch.matmul(w[i].double().t().contiguous(), dc[at].double()) for at, i in
                        zip(on.tolist(), experts[::40].reshape(-1).tolist())])
    assert torch.equal(rows[on], want.half())
    del rows
    dout = torch.randint(-2, 3, (t, n), device="cuda", generator=gen, dtype=torch.int8).half()
    dy, dw = g.combine_experts_backward(dout, y, r)
    weights = r.weights[some].double()
    want = weights[..., None] * dout[some][:, None].double()
    # a product in fp32, then in fp16: 2^-24 and 2^-11, 2^-25 among the subnormals
    assert ((dy[places].double() - want).abs() <= want.abs() * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()
    assert torch.equal(dw[some].double(), (dout[some][:, None].double() * y[places].double()).sum(2))


# ---- streams ----------------------------------------------------------------------
class ElsewhereStream:
    """A stream of another device."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_streams_of_another_device_are_refused(g):
    """By every function, whether it allocates its output or is given it."""
    f16 = dict(dtype=torch.float16, device="cuda")
    t, e, top, n, k = 4, 3, 2, 20, 130
    x, dy, w = torch.ones(t, k, **f16), torch.ones(t * top, n, **f16), torch.ones(e, n, k, **f16)
    logits = torch.zeros(t, e, device="cuda")
    r, w8, one = g.route(logits, top), g.quantize_f8(w, 128), g.quantize_f8(w[0], 128)
    dy8, x8 = g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True)
    s = ElsewhereStream()
    calls = [
        lambda: g.quantize_f8(x, stream=s), lambda: g.quantize_f8(w, 128, stream=s),
        lambda: g.route(logits, top, stream=s), lambda: g.route_backward(logits, r, r.weights, stream=s),
        lambda: g.quantize_f8_experts(x, r, gather=True, stream=s), lambda: g.combine_experts_backward(x, None, r, weighted=False, stream=s),
    ]
    for fn, args, shape in ((g.dequantize_f8, (one,), (n, k)), (g.dequantize_f8, (w8,), (e, n, k)),
                            (g.gemm_nt_f8, (x, one), (t, n)), (g.gemm_nt_f8_experts, (x, w8, r, True), (t * top, n)),
                            (g.gemm_nt_f8_experts_grad, (dy8, x8, r), (e, n, k)), (g.combine_experts, (dy, r), (t, n))):
        fn(*args, out=torch.empty(shape, **f16))      # what is wrong is the stream alone
        for out in (None, torch.empty(shape, **f16)):
            calls.append(lambda fn=fn, args=args, out=out: fn(*args, out=out, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="stream is on"):
            call()


LIVES = ["quantize rows", "quantize transposed", "quantize blocks", "dequantize", "product of few halves",
         "product, workspace", "product of codes", "route", "route_backward", "experts of few halves", "experts, gathered",
         "experts, workspace", "quantize_f8_experts", "experts' gradients", "combine", "combine_backward", "combine_backward, unweighted"]


def operands_and_call(g, what):
    """(call(**kw) giving tensors, the tensors that it is given, each its own memory)."""
    rng = np.random.default_rng(3)
    t, e, top, n, k = 700, 16, 2, 520, 768

    def halves(*shape):
        return dev(rng.standard_normal(shape).astype(np.float16))

    def codes(q):
        return q.codes.view(torch.uint8), q.scales

    cus = g.gemm_f16_device_cus()
    if what.startswith("quantize "):
        x = halves(1024, 2048)
        how = {"quantize rows": (1, False), "quantize transposed": (1, True), "quantize blocks": (128, False)}[what]
        return lambda **kw: codes(g.quantize_f8(x, *how, **kw)), [x]
    if what == "dequantize":
        q = g.quantize_f8(halves(1024, 2048))
        return lambda **kw: (g.dequantize_f8(q, **kw),), [q.codes, q.scales]
    if what.startswith("product"):
        w = g.quantize_f8(halves(1024, 2048), 128)
        a = halves(7 if what == "product of few halves" else 300, 2048)
        if what == "product of codes":
            q = g.quantize_f8(a)
            return lambda **kw: (g.gemm_nt_f8(q, w, **kw),), [q.codes, q.scales, w.codes, w.scales]
        need = g.gemm_f16_nt_f8_plan(len(a), 1024, 2048, 128, True, cus).workspace_bytes
        if what == "product of few halves":
            assert need == 0
            return lambda **kw: (g.gemm_nt_f8(a, w, **kw),), [a, w.codes, w.scales]
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        return lambda **kw: (g.gemm_nt_f8(a, w, workspace=ws, **kw),), [a, w.codes, w.scales, ws]
    few = what == "experts of few halves"
    t = 3 if few else t
    logits, bias = dev(rng.standard_normal((t, e)).astype(np.float32)), dev(rng.standard_normal(e).astype(np.float32))
    if what == "route":
        def call(**kw):
            r = g.route(logits, top, "sigmoid", bias, **kw)
            return r.experts, r.weights, r.rows, r.places, r.offsets
        return call, [logits, bias]
    r = g.route(logits, top)
    r = g.Routing(*(x.clone() for x in (r.experts, r.weights, r.rows, r.places, r.offsets)))   # each its own memory
    y, x = halves(t * top, n), halves(t, k)
    if what == "route_backward":
        dw = dev(rng.standard_normal((t, top)).astype(np.float32))
        return lambda **kw: (g.route_backward(logits, r, dw, **kw),), [logits, r.experts, r.weights, dw]
    if what == "quantize_f8_experts":
        used = sum(-(-c // 128) for c in r.offsets.diff().tolist())     # groups that are written

        def call(**kw):
            q = g.quantize_f8_experts(x, r, gather=True, **kw)
            return q.codes.view(torch.uint8)[:, :128 * used], q.scales[:used // 4]
        return call, [x, r.rows, r.offsets]
    if what == "experts' gradients":
        a, b = g.quantize_f8_experts(y, r), g.quantize_f8_experts(x, r, gather=True)
        return lambda **kw: (g.gemm_nt_f8_experts_grad(a, b, r, **kw),), [a.codes, a.scales, b.codes, b.scales, r.offsets]
    if what.startswith("experts"):
        w = g.quantize_f8(halves(e, n, k), 128)
        given = [x, w.codes, w.scales, r.rows, r.offsets]
        need = g.gemm_f16_nt_f8_experts_plan(t * top, e, n, k, top, True, cus).workspace_bytes
        assert (need == 0) == few
        if what != "experts, workspace":
            return lambda **kw: (g.gemm_nt_f8_experts(x, w, r, True, **kw),), given
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        return lambda **kw: (g.gemm_nt_f8_experts(x, w, r, True, workspace=ws, **kw),), given + [ws]
    if what == "combine":
        return lambda **kw: (g.combine_experts(y, r, **kw),), [y, r.weights, r.places]
    dout = halves(t, n)
    if what == "combine_backward":
        return lambda **kw: g.combine_experts_backward(dout, y, r, **kw), [dout, y, r.weights, r.rows, r.places]
    return lambda **kw: g.combine_experts_backward(dout, None, r, False, **kw)[:1], [dout, r.rows, r.places]


@pytest.mark.parametrize("what", LIVES)
def test_operands_dropped_at_once(g, what):
    """Operands (and a workspace) of the default stream, used on a busy stream and
    dropped at once: their memory goes to no other tensor before they are read."""
    want = [host(t) for t in operands_and_call(g, what)[0]()]
    s, done = torch.cuda.Stream(), torch.cuda.Event()
    filler = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    # torch's memory for what both streams allocate later: new memory from the
    # driver would wait for s
    operands_and_call(g, what)[0](stream=s)
    s.synchronize()
    call, given = operands_and_call(g, what)
    ranges = [(t.data_ptr(), t.numel() * t.element_size()) for t in given]
    spare = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in ranges for _ in range(8)]
    del spare
    torch.cuda.synchronize()     # the operands are made
    with torch.cuda.stream(s):
        for _ in range(200):   # some 40 ms
            filler[:1 << 29].copy_(filler[1 << 29:])
    got = call(stream=s)
    done.record(s)
    del call, given
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in ranges for _ in range(4)]
    # (asked before the default stream gets work: it may share a hardware queue with s)
    assert not done.query(), "the stream was not busy for long enough to show anything"
    for t in later:
        for at, size in ranges:
            assert t.data_ptr() + t.numel() <= at or at + size <= t.data_ptr()
        t.fill_(0x55)
    s.synchronize()
    for t, w in zip(got, want):
        np.testing.assert_array_equal(host(t), w)


def test_layer_on_another_stream(g):
    """A layer and its gradients on a stream that waits for their inputs, against the
    same on the default stream."""
    rng = np.random.default_rng(11)
    x, wr, up, down = layer_inputs(g, rng, 90, 256, 128, 8)
    up8, down8 = g.quantize_f8(up, 128), g.quantize_f8(down, 128)
    logits, r, h, y, out = layer(g, x, wr, up8, down8, 2)

    def steps(logits, h, dout, **kw):
        r = g.route(logits, 2, "sigmoid", groups=2, top_groups=1, scale=1.5, **kw)
        y = g.gemm_nt_f8_experts(h, down8, r, **kw)
        out = g.combine_experts(y, r, **kw)
        dy, dw = g.combine_experts_backward(dout, y, r, **kw)
        dlogits = g.route_backward(logits, r, dw, **kw)
        ddown = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r, **kw), g.quantize_f8_experts(h, r, **kw), r, **kw)
        single = g.gemm_nt_f8(g.quantize_f8(h, **kw), g.quantize_f8(down[0], 128, **kw), **kw)
        return out, dlogits, ddown, single, g.dequantize_f8(up8, **kw)

    want = steps(logits, h, out)
    s = torch.cuda.Stream()
    copies = logits.clone(), h.clone(), out.clone()
    s.wait_stream(torch.cuda.current_stream())
    got = steps(*copies, stream=s)
    del copies
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ---- all steps together ------------------------------------------------------------
@pytest.mark.parametrize("t", [1, 7, 150])
@pytest.mark.parametrize("scores,renormalize", [("sigmoid", True), ("softmax", True), ("softmax", False)])
def test_layer_step_by_step(g, t, scores, renormalize):
    """A layer of experts and all its gradients, some tokens padding: each step's output
    against 64 bits on the inputs that it was given."""
    rng = np.random.default_rng(t)
    d, f, e, top, scale = 256, 200, 8, 3, 1.5
    x, wr, up, down = layer_inputs(g, rng, t, d, f, e)
    logits = g.gemm_nt(x, wr)
    if t > 1:
        logits[t // 2] = -torch.inf
        logits[0, 2:] = -torch.inf        # fewer experts than choices
    r = g.route(logits, top, scores, renormalize=renormalize, scale=scale)
    h = torch.relu(g.gemm_nt_f8_experts(x, g.quantize_f8(up, 128), r, gather=True))
    y = g.gemm_nt_f8_experts(h, g.quantize_f8(down, 128), r)
    out = g.combine_experts(y, r)
    dout = dev(rng.standard_normal((t, d)).astype(np.float16))
    dy, dweights = g.combine_experts_backward(dout, y, r)
    dlogits = g.route_backward(logits, r, dweights)
    dh = torch.where(h > 0, g.gemm_nt_f8_experts(dy, g.quantize_f8(down, 128, transposed=True), r), 0)
    dxs = g.gemm_nt_f8_experts(dh, g.quantize_f8(up, 128, transposed=True), r)
    dx = g.combine_experts(dxs, r, weighted=False)
    dx_router = g.matmul(dlogits, wr)
    dwr = g.matmul(dlogits.t(), x)

    lg = host(logits).astype(np.float64)
    experts, weights = ref.route(host(logits), top, scores, renormalize=renormalize, scale=scale)
    np.testing.assert_array_equal(host(r.experts), experts)
    w = host(r.weights).astype(np.float64)
    # one rounding to fp32, and sums of 64-bit scores in another order
    assert (np.abs(w - weights) <= np.abs(weights) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150).all()
    rows, places, offsets = ref.order(experts, e)
    for a, b in ((r.rows, rows), (r.places, places), (r.offsets, offsets)):
        np.testing.assert_array_equal(host(a), b)

    there = (places >= 0)[..., None]

    def of_tokens(v):
        return np.where(there, host(v)[np.maximum(places, 0)].astype(np.float64), 0.0)

    def summed(got, factor, v):
        """Sums over a token's choices in fp32 (a rounding each), rounded to fp16."""
        terms = factor[..., None] * of_tokens(v)
        exact, size = terms.sum(1), np.abs(terms).sum(1)
        off = size * (top + 1) * 2.0 ** -24
        assert (np.abs(host(got) - exact) <= off + (np.abs(exact) + off) * 2.0 ** -11 + 2.0 ** -25).all()

    summed(out, w, y)
    summed(dx, np.ones_like(w), dxs)

    do = host(dout).astype(np.float64)
    want = np.zeros((t * top, d))
    for i, j in zip(*np.nonzero(places >= 0)):
        want[places[i, j]] = w[i, j] * do[i]
    # a product in fp32, then in fp16: 2^-24 and 2^-11, 2^-25 among the subnormals
    assert (np.abs(host(dy) - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()
    terms = do[:, None] * of_tokens(y)
    # products and sums of d terms in fp32, a rounding each and 16 to join
    assert (np.abs(host(dweights) - terms.sum(2)) <= np.abs(terms).sum(2) * (d + 16) * 2.0 ** -24).all()

    dw = host(dweights).astype(np.float64)
    want = ref.route_gradient(lg, experts, dw, scores, renormalize, scale)
    # one rounding to fp16; 64-bit sums of at most top + e terms of 4 scale dw / (least sum) in size
    size = 4 * scale * np.abs(dw).max(1, keepdims=True) * (top + e + 40) * 2.0 ** -52 * 2.0 ** 10
    assert (np.abs(host(dlogits) - want) <= np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size).all()

    def near(got, a, b):
        """A product in 8-bit codes within the bound."""
        exact = a @ b.T
        bound = ref.product_bound(np.abs(a) @ np.abs(b).T, exact, a.shape[1])
        assert (np.abs(host(got).astype(np.float64) - exact) <= bound).all()

    dl, q = host(dlogits).astype(np.float64), ref.quantized
    ddown = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(h, r), r)
    dup = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dh, r), g.quantize_f8_experts(x, r, gather=True), r)
    for i in range(e):
        a, b = offsets[i], offsets[i + 1]
        if a == b:
            assert (host(dup[i]) == 0).all() and (host(ddown[i]) == 0).all()
            continue
        xi = host(x)[rows[a:b] // top]
        near(y[a:b], q(host(h[a:b]), 1), q(host(down[i]), 128))
        near(dxs[a:b], q(host(dh[a:b]), 1), q(host(up[i]), 128).T)
        near(ddown[i], q(host(dy[a:b]).T.copy(), 1), q(host(h[a:b]).T.copy(), 1))
        near(dup[i], q(host(dh[a:b]).T.copy(), 1), q(xi.T.copy(), 1))
    for v in (y, dy, dxs):
        assert (host(v[offsets[-1]:]) == 0).all()
    for got, a, b in ((dx_router, dl, host(wr).astype(np.float64)), (dwr, dl.T, host(x).astype(np.float64))):
        exact, size = a @ b, np.abs(a) @ np.abs(b)
        off = size * (a.shape[1] + 16) * 2.0 ** -23          # fp32 sums
        assert (np.abs(host(got) - exact) <= off + (np.abs(exact) + off) * 2.0 ** -11 + 2.0 ** -25).all()


# ---- saved and read back -----------------------------------------------------------
READ_BACK = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, dense_fp16_gemm_amd as g
safe = sys.argv[3] == "safe"
if safe:
    torch.serialization.add_safe_globals([g.F8Matrix, g.Routing])
stored = torch.load(sys.argv[2], weights_only=safe)
def same(a, b):
    assert torch.equal(a, b)
if "gemm_nt_f8" in stored:
    a, w, stack, y, values = stored["gemm_nt_f8"]
    assert (a.shape, a.block, w.shape, w.block, stack.shape) == ((3, 200), 1, (50, 200), 128, (4, 50, 200))
    same(g.gemm_nt_f8(a, w), y)
    same(g.dequantize_f8(stack), values)
else:
    r, logits, x, w, y, out, dlogits = stored["route"]
    assert (r.tokens, r.top, r.n_experts, r.scores, r.renormalize, r.scale) == (30, 2, 4, "sigmoid", False, 2.5)
    same(g.combine_experts(y, r), out)
    same(g.gemm_nt_f8_experts(x, w, r, gather=True), y)
    same(g.route_backward(logits, r, torch.ones_like(r.weights)), dlogits)
print("same")
"""


@pytest.mark.parametrize("how", ["safe", "any"])
@pytest.mark.parametrize("what", ["gemm_nt_f8", "route"])
def test_saved_in_a_new_process(g, how, what, tmp_path):
    """Matrices and a routing, saved whole: in a process whose first use of the package
    is of what it read back."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def halves(*shape):
        return torch.randn(shape, generator=gen, device="cuda").half()

    stack = g.quantize_f8(halves(4, 50, 200), 128)
    if what == "gemm_nt_f8":
        a, w = g.quantize_f8(halves(3, 200)), g.quantize_f8(halves(50, 200), 128)
        stored = a, w, stack, g.gemm_nt_f8(a, w), g.dequantize_f8(stack)
    else:
        logits, x = torch.randn(30, 4, generator=gen, device="cuda"), halves(30, 200)
        r = g.route(logits, 2, "sigmoid", renormalize=False, scale=2.5)
        y = g.gemm_nt_f8_experts(x, stack, r, gather=True)
        stored = r, logits, x, stack, y, g.combine_experts(y, r), g.route_backward(logits, r, torch.ones_like(r.weights))
    path = str(tmp_path / "stored.pt")
    torch.save({what: stored}, path)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", READ_BACK, root, path, how], timeout=100, capture_output=True)
    assert done.returncode == 0 and done.stdout == b"same\n", done.stderr.decode()[-2000:]


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_copies(g, how):
    """Copies hold the same and are checked as what a program makes itself."""
    x = torch.randn(7, 130, device="cuda").half()
    q = g.quantize_f8(x)
    again = how(q)
    assert (again.shape, again.block) == (q.shape, q.block)
    assert torch.equal(g.dequantize_f8(again), g.dequantize_f8(q))
    r = g.route(torch.randn(7, 5, device="cuda"), 2, scale=0.5)
    s = how(r)
    assert (s.scores, s.renormalize, s.scale, s.n_experts) == (r.scores, r.renormalize, r.scale, r.n_experts)
    assert torch.equal(g.combine_experts(x.repeat(2, 1), s), g.combine_experts(x.repeat(2, 1), r))
    assert (s.weights.data_ptr() == r.weights.data_ptr()) == (how is copy.copy)
