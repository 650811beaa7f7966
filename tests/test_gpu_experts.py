"""Routing, the experts' products and their combination on the GPU, against plain
64-bit references (f8_ref.py)."""
import numpy as np
import pytest
import torch

import f8_ref as ref
from test_gpu_f8 import dev, f8, g, host, whole  # noqa: F401  (g: the fixture)

pytestmark = pytest.mark.gpu


def check_route(r, experts, weights, e):
    np.testing.assert_array_equal(host(r.experts), experts)
    w = host(r.weights).astype(np.float64)
    assert (np.isnan(w) == np.isnan(weights)).all()
    fine = ~np.isnan(weights)
    # one rounding to fp32, and sums of 64-bit scores in another order
    assert (np.abs(w - weights)[fine] <= np.abs(weights[fine]) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150).all()
    rows, places, offsets = ref.order(experts, e)
    np.testing.assert_array_equal(host(r.rows), rows)
    np.testing.assert_array_equal(host(r.places), places)
    np.testing.assert_array_equal(host(r.offsets), offsets)


ROUTES = [(1, 1, 1, 1, 1), (1, 8, 2, 1, 1), (3, 5, 5, 1, 1), (7, 64, 6, 1, 1), (1, 256, 8, 8, 4),
          (65, 65, 3, 1, 1), (100, 128, 8, 4, 2), (33, 160, 6, 8, 3), (20, 384, 8, 1, 1),
          (9, 1024, 32, 64, 5), (5, 1000, 10, 8, 8), (300, 16, 2, 4, 1), (12, 96, 4, 3, 2)]


@pytest.mark.parametrize("t,e,top,groups,top_groups", ROUTES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("half", [True, False])
def test_route(g, t, e, top, groups, top_groups, scores, half):
    rng = np.random.default_rng(t * 1000 + e)
    x = (2 * rng.standard_normal((t, e))).astype(np.float16 if half else np.float32)
    for bias, norm, scale, how in ((None, True, 1.0, "top2"), (rng.standard_normal(e).astype(np.float32) * 0.2, True, 2.5, "top2"),
                                   (rng.standard_normal(e).astype(np.float32) * 0.2, False, 0.7, "max")):
        r = g.route(dev(x), top, scores, None if bias is None else dev(bias), groups, top_groups,
                    how, norm, scale)
        check_route(r, *ref.route(x, top, scores, bias, groups, top_groups, how, norm, scale), e)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masks_ties_and_not_finite(g, scores, groups):
    """Rows with all experts masked, with fewer left than wanted, with equal
    logits, with the type's lowest value, with infinities and NaN."""
    rng = np.random.default_rng(1)
    t, e, top = 40, 32, 6
    x = np.round(rng.standard_normal((t, e)) * 2).astype(np.float16)     # many ties
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2] = 1.0
    x[3, 5] = np.nan
    x[4, 6] = np.inf
    x[5] = -65504
    x[6] = 65504
    x[7, ::2] = -np.inf
    x[8, 8:] = -65504
    x[9, :24] = -np.inf
    bias = np.zeros(e, dtype=np.float32)
    bias[9] = -np.inf
    for b in (None, bias):
        for how in ("top2", "max"):
            r = g.route(dev(x), top, scores, None if b is None else dev(b), groups, 2 if groups > 1 else 1, how)
            check_route(r, *ref.route(x, top, scores, b, groups, 2 if groups > 1 else 1, how), e)
    bias[4] = np.nan
    r = g.route(dev(x), top, scores, dev(bias), groups, groups)
    check_route(r, *ref.route(x, top, scores, bias, groups, groups), e)


def test_route_by_close_scores(g):
    """Scores that 32 bits do not tell apart are told apart."""
    x = np.full((2, 70), 20.0, dtype=np.float32)
    x[0, 69], x[0, 33] = 20.5, 20.25
    x[1, 1] = np.nextafter(np.float32(20), np.float32(21))
    r = g.route(dev(x), 3, "sigmoid")
    np.testing.assert_array_equal(host(r.experts), [[69, 33, 0], [1, 0, 2]])
    check_route(r, *ref.route(x, 3, "sigmoid"), 70)


@pytest.mark.parametrize("t", [0, 1, 2, 63, 64, 65, 511, 1025, 5000])
@pytest.mark.parametrize("e,top", [(8, 2), (130, 7), (1024, 1)])
def test_order(g, t, e, top):
    """The order of many tokens; some experts have none, some tokens no expert."""
    rng = np.random.default_rng(t + e)
    x = rng.standard_normal((t, e)).astype(np.float32) + 2 * rng.standard_normal(e).astype(np.float32)
    x[rng.random(t) < 0.1] = -np.inf
    x[:, rng.random(e) < 0.3] -= 50
    r = g.route(dev(x), top)
    experts = host(r.experts)
    s = ref.scores_of(x.astype(np.float64), "softmax")
    want = np.argsort(-s, axis=1, kind="stable")[:, :top] if t else np.zeros((0, top), int)
    np.testing.assert_array_equal(experts, np.where(np.isneginf(x).all(1, keepdims=True), -1, want))
    flat = experts.reshape(-1)
    keep = np.nonzero(flat >= 0)[0]
    rows = keep[np.argsort(flat[keep], kind="stable")]
    np.testing.assert_array_equal(host(r.rows), np.concatenate([rows, np.full(flat.size - rows.size, -1)]))
    places = np.full(flat.size, -1)
    places[rows] = np.arange(rows.size)
    np.testing.assert_array_equal(host(r.places).reshape(-1), places)
    np.testing.assert_array_equal(host(r.offsets), np.concatenate([[0], np.cumsum(np.bincount(flat[keep], minlength=e))]))


@pytest.mark.parametrize("t,e,top", [(1, 1, 1), (1, 64, 8), (5, 3, 2), (30, 100, 6), (11, 300, 8), (4, 1024, 32), (200, 32, 4)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_backward(g, t, e, top, scores, norm):
    rng = np.random.default_rng(e + t)
    x = (1.5 * rng.standard_normal((t, e))).astype(np.float32)
    x[rng.random((t, e)) < 0.05] = -np.inf
    if t > 3:
        x[2] = -np.inf
    dw = rng.standard_normal((t, top)).astype(np.float32)
    for dtype in (np.float32, np.float16):
        xx = x.astype(dtype)
        r = g.route(dev(xx), top, scores, renormalize=norm, scale=1.7)
        got = host(g.route_backward(dev(xx), r, dev(dw))).astype(np.float64)
        want = ref.route_gradient(xx.astype(np.float64), host(r.experts), dw.astype(np.float64), scores, norm, 1.7)
        # one rounding; the 64-bit sums of at most top + E terms of this size
        size = np.abs(dw).max(1, keepdims=True) * 1.7 * (4 if norm else 1)
        half = 2.0 ** -24 if dtype == np.float32 else 2.0 ** -11
        tiny = 2.0 ** -150 if dtype == np.float32 else 2.0 ** -25
        assert (np.abs(got - want) <= np.abs(want) * half + tiny + size * (top + e + 40) * 2.0 ** -52).all()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("norm", [True, False])
def test_route_backward_by_differences(g, scores, norm):
    rng = np.random.default_rng(3)
    t, e, top, h = 3, 12, 4, 2.0 ** -17
    x = rng.standard_normal((t, e)).astype(np.float32)
    dw = rng.standard_normal((t, top)).astype(np.float32)
    r = g.route(dev(x), top, scores, renormalize=norm, scale=2.0)
    got = host(g.route_backward(dev(x), r, dev(dw))).astype(np.float64)
    experts = host(r.experts)
    for i in range(t):
        for j in range(e):
            up, down = x.astype(np.float64), x.astype(np.float64)
            up[i, j] += h
            down[i, j] -= h
            d = ((ref.weights_of(up, experts, scores, norm, 2.0) - ref.weights_of(down, experts, scores, norm, 2.0)) * dw).sum() / (2 * h)
            # the third derivative's share (h^2, times at most 10) and roundings of 2^-52 / h
            assert abs(d - got[i, j]) <= 10 * h * h + 2.0 ** -52 / h * 10 + abs(d) * 2.0 ** -24


def test_route_backward_without_value(g):
    """A token with NaN weights gets NaN, one without experts zeros whatever
    dweights holds for it."""
    x = np.zeros((4, 8), dtype=np.float32)
    x[1, 2], x[2], x[3, 4:] = np.nan, -np.inf, -np.inf
    dw = np.full((4, 6), 2.0, dtype=np.float32)
    dw[2], dw[3, 4:] = np.nan, np.inf
    r = g.route(dev(x), 6)
    got = host(g.route_backward(dev(x), r, dev(dw)))
    assert np.isnan(got[1]).all() and (got[2] == 0).all() and np.isfinite(got[3]).all() and (got[3, 4:] == 0).all()


# ---- the experts' products -------------------------------------------------------
def routing(g, rng, t, e, top, drop=0.0, only=None):
    """Random experts, distinct for a token; some slots without one."""
    pool = np.arange(e) if only is None else np.asarray(only)
    experts = np.stack([rng.permutation(pool)[:top] for _ in range(t)]) if t else np.zeros((0, top), int)
    experts = np.where(rng.random(experts.shape) < drop, -1, experts)
    weights = rng.random(experts.shape).astype(np.float32)
    weights[experts < 0] = 0
    rows, places, offsets = ref.order(experts, e)
    i32 = lambda v: dev(v.astype(np.int32))  # noqa: E731
    r = g.Routing(i32(experts), dev(weights), i32(rows), i32(places), i32(offsets))
    return r, experts, weights, rows, places, offsets


EXPERTS = [(1, 1, 1, 16, 128), (1, 8, 2, 100, 300), (1, 64, 8, 256, 640), (3, 4, 2, 130, 200),
           (16, 8, 3, 64, 512), (50, 5, 2, 200, 129), (100, 64, 6, 128, 256), (130, 3, 1, 300, 128),
           (200, 2, 2, 96, 1000), (333, 16, 4, 136, 384), (40, 200, 8, 32, 130), (700, 6, 2, 264, 256)]


@pytest.mark.parametrize("t,e,top,n,k", EXPERTS)
@pytest.mark.parametrize("gather", [True, False])
def test_experts_exact(g, t, e, top, n, k, gather):
    rng = np.random.default_rng(t + e + n)
    wc, ws, w = zip(*(whole(rng, n, k, 128) for _ in range(e)))
    w8 = g.F8Matrix(dev(np.stack(wc)).view(torch.float8_e4m3fn), dev(np.stack(ws)), k, 128)
    for drop, only in ((0.0, None), (0.2, None), (0.0, list(range(top)) if e > top else None)):
        r, _, _, rows, _, offsets = routing(g, rng, t, e, top, drop, only)
        ac, as_, a = whole(rng, t if gather else t * top, k, 1)
        y = host(g.gemm_nt_f8_experts(f8(g, ac, as_, k, 1), w8, r, gather=gather))
        want = np.zeros((t * top, n))
        for i in range(e):
            p = np.arange(offsets[i], offsets[i + 1])
            want[p] = a[rows[p] // top if gather else p] @ w[i].T
        np.testing.assert_array_equal(y, want.astype(np.float16))


@pytest.mark.parametrize("t,e,top,n,k", [(1, 16, 4, 200, 300), (9, 4, 2, 128, 256), (150, 8, 3, 130, 640)])
def test_experts_of_halves(g, t, e, top, n, k):
    """A in fp16: what quantize_f8 gives, bit for bit; one expert's rows are the
    dense product's."""
    rng = np.random.default_rng(t)
    w8 = g.quantize_f8(dev(rng.standard_normal((e, n, k)).astype(np.float16)), 128)
    r, _, _, rows, _, offsets = routing(g, rng, t, e, top)
    x = dev(rng.standard_normal((t, k)).astype(np.float16))
    y = g.gemm_nt_f8_experts(x, w8, r, gather=True)
    x8 = g.quantize_f8(x)
    assert torch.equal(y, g.gemm_nt_f8_experts(x8, w8, r, gather=True))
    sorted_x = x[dev(rows // top)]
    assert torch.equal(y, g.gemm_nt_f8_experts(sorted_x, w8, r))
    wq = [ref.quantized(host(g.dequantize_f8(g.F8Matrix(w8.codes[i], w8.scales[i], k, 128))), 128) for i in range(e)]
    xq = ref.quantized(host(sorted_x), 1)
    for i in range(e):
        p = slice(offsets[i], offsets[i + 1])
        exact = xq[p] @ wq[i].T
        assert (np.abs(host(y)[p] - exact) <= ref.product_bound(np.abs(xq[p]) @ np.abs(wq[i]).T, exact, k)).all()


@pytest.mark.parametrize("t,e,top,n,k", [(1, 8, 2, 16, 32), (5, 3, 2, 130, 64), (100, 4, 2, 128, 256), (300, 7, 3, 200, 140), (1000, 2, 1, 300, 40)])
def test_experts_gradient_exact(g, t, e, top, n, k):
    """Whole numbers with the same largest one in every group quantise without a
    rounding: each expert's dW is exact."""
    rng = np.random.default_rng(t + n)
    for drop in (0.0, 0.3):
        r, _, _, rows, _, offsets = routing(g, rng, t, e, top, drop)
        dy, x = rng.integers(-7, 8, (t * top, n)), rng.integers(-7, 8, (t, k))
        dyt = g.quantize_f8_experts(dev(dy.astype(np.float16)), r)
        xt = g.quantize_f8_experts(dev(x.astype(np.float16)), r, gather=True)
        xs = g.quantize_f8_experts(dev(x[np.maximum(rows, 0) // top].astype(np.float16)), r)
        dw = g.gemm_nt_f8_experts_grad(dyt, xt, r)
        want = np.stack([dy[a:b].T @ x[rows[a:b] // top] for a, b in zip(offsets, offsets[1:])])
        np.testing.assert_array_equal(host(dw), want.astype(np.float16))
        assert torch.equal(dw, g.gemm_nt_f8_experts_grad(dyt, xs, r))


def test_experts_columns(g):
    """The columns of quantize_f8_experts: each expert's from a multiple of 128."""
    rng = np.random.default_rng(5)
    t, e, top, n = 200, 5, 2, 150
    r, _, _, rows, _, offsets = routing(g, rng, t, e, top, 0.1)
    x = rng.standard_normal((t * top, n)).astype(np.float16)
    q = g.quantize_f8_experts(dev(x), r)
    got = ref.code_values()[host(q.codes.view(torch.uint8))]
    scales = host(q.scales)
    at = 0
    for a, b in zip(offsets, offsets[1:]):
        want, exps = ref.encode(x[a:b].T, 1)
        np.testing.assert_array_equal(got[:, at:at + want.shape[1]], want)
        for i in range(want.shape[1] // 128):
            group = at // 128 + i
            np.testing.assert_array_equal(scales[group // 4, :, group % 4], exps[:, i] + 127)
        at += want.shape[1]
    assert at <= q.k == g.gemm_f16_f8_experts_columns(t * top, e)


def test_experts_handles_of_any_numbers(g):
    """Whatever numbers rows, places and offsets hold, nothing outside the
    outputs is written."""
    rng = np.random.default_rng(6)
    t, e, top, n, k = 20, 6, 2, 130, 256
    x = dev(rng.standard_normal((t, k)).astype(np.float16))
    w8 = g.quantize_f8(dev(rng.standard_normal((e, n, k)).astype(np.float16)), 128)
    good, experts, weights, *_ = routing(g, rng, t, e, top)
    for i in range(4):
        far = lambda *s: dev(rng.integers(-2 ** 31, 2 ** 31, s).astype(np.int32))  # noqa: E731
        near = lambda *s: dev(rng.integers(-3, 45, s).astype(np.int32))  # noqa: E731
        some = far if i < 2 else near
        r = g.Routing(good.experts, good.weights, some(t * top), some(t, top), some(e + 1))
        buf = torch.full((t * top + 2, n), 5.0, dtype=torch.float16, device="cuda")
        y = g.gemm_nt_f8_experts(x, w8, r, gather=True, out=buf[1:-1])
        assert (buf[0] == 5).all() and (buf[-1] == 5).all()
        dyt, xt = g.quantize_f8_experts(y, r), g.quantize_f8_experts(x, r, gather=True)
        buf = torch.full((e * n + 2, k), 5.0, dtype=torch.float16, device="cuda")
        g.gemm_nt_f8_experts_grad(dyt, xt, r, out=buf[1:-1].view(e, n, k))
        assert (buf[0] == 5).all() and (buf[-1] == 5).all()
        g.combine_experts(y, r)
        g.combine_experts_backward(torch.ones(t, n, dtype=torch.float16, device="cuda"), y, r)
    torch.cuda.synchronize()


# ---- combination -------------------------------------------------------------------
@pytest.mark.parametrize("t,top,n", [(1, 1, 1), (1, 8, 4096), (3, 2, 7), (17, 6, 130), (200, 4, 1000), (64, 32, 9), (5, 3, 8192)])
@pytest.mark.parametrize("weighted", [True, False])
def test_combine(g, t, top, n, weighted):
    rng = np.random.default_rng(n)
    r, experts, weights, rows, places, offsets = routing(g, rng, t, max(top, 40), top, 0.15)
    y = rng.standard_normal((t * top, n)).astype(np.float16)
    y[offsets[-1]:] = np.nan                      # rows of no slot are not read
    w = weights.astype(np.float64) if weighted else np.ones((t, top))
    there = places >= 0
    rowsof = np.where(there[..., None], y[np.maximum(places, 0)].astype(np.float64), 0.0)
    out = host(g.combine_experts(dev(y), r, weighted)).astype(np.float64)
    want = (w[..., None] * rowsof).sum(1)
    size = (np.abs(w)[..., None] * np.abs(rowsof)).sum(1)
    assert (np.abs(out - want) <= np.abs(want) * 2.0 ** -11 + 2.0 ** -25 + size * (top + 1) * 2.0 ** -24 * 1.01).all()

    dout = rng.standard_normal((t, n)).astype(np.float16)
    dy, dw = g.combine_experts_backward(dev(dout), dev(y), r, weighted)
    want = np.zeros((t * top, n))
    for i in range(t):
        for j in range(top):
            if there[i, j]:
                want[places[i, j]] = w[i, j] * dout[i].astype(np.float64)   # 35 bits: exact
    # the product in fp32 (2^-24 off at most, or exact), then in fp16 (2^-11, or
    # 2^-25 among the subnormals)
    assert (np.abs(host(dy) - want) <= np.abs(want) * (2.0 ** -11 + 2.0 ** -23) + 2.0 ** -25).all()
    if not weighted:
        assert dw is None
        return
    exact = (dout[:, None].astype(np.float64) * rowsof).sum(2)
    size = np.abs(dout[:, None].astype(np.float64) * rowsof).sum(2)
    assert (np.abs(host(dw) - exact) <= (size * (n + 16) * 2.0 ** -24)).all()
    assert (host(dw)[~there] == 0).all()


def test_combine_not_finite(g):
    """A NaN weight reaches its token, also where its slot has no expert."""
    rng = np.random.default_rng(2)
    r, *_ = routing(g, rng, 3, 4, 2)
    r.places[1, 0] = -1
    r.weights[1, 0] = float("nan")
    out = host(g.combine_experts(torch.ones(6, 20, dtype=torch.float16, device="cuda"), r))
    assert np.isnan(out[1]).all() and np.isfinite(out[[0, 2]]).all()


# ---- together ------------------------------------------------------------------------
def layer(g, x, wr, up, down, top):
    logits = g.gemm_nt(x, wr)
    r = g.route(logits, top, "sigmoid", groups=2, top_groups=1, scale=1.5)
    h = torch.relu(g.gemm_nt_f8_experts(x, up, r, gather=True))
    y = g.gemm_nt_f8_experts(h, down, r)
    return logits, r, h, y, g.combine_experts(y, r)


def layer_inputs(g, rng, t, d, f, e):
    x = dev(rng.standard_normal((t, d)).astype(np.float16))
    wr = dev((rng.standard_normal((e, d)) / np.sqrt(d)).astype(np.float16))
    up = dev((rng.standard_normal((e, f, d)) / np.sqrt(d)).astype(np.float16))
    down = dev((rng.standard_normal((e, d, f)) / np.sqrt(f)).astype(np.float16))
    return x, wr, up, down


@pytest.mark.parametrize("t", [1, 7, 150])
def test_layer_of_experts(g, t):
    """A layer of experts forward and backward, each step against 64 bits on the
    inputs that it was given."""
    rng = np.random.default_rng(t)
    d, f, e, top = 256, 200, 8, 3
    x, wr, up, down = layer_inputs(g, rng, t, d, f, e)
    up8, down8 = g.quantize_f8(up, 128), g.quantize_f8(down, 128)
    logits, r, h, y, out = layer(g, x, wr, up8, down8, top)
    check_route(r, *ref.route(host(logits), top, "sigmoid", groups=2, top_groups=1, scale=1.5), e)
    rows, offsets = host(r.rows), host(r.offsets)

    def near(got, a, b):
        exact = a @ b.T
        assert (np.abs(host(got).astype(np.float64) - exact) <= ref.product_bound(np.abs(a) @ np.abs(b).T, exact, a.shape[1])).all()

    dout = dev(rng.standard_normal((t, d)).astype(np.float16))
    dy, dw = g.combine_experts_backward(dout, y, r)
    dlogits = g.route_backward(logits, r, dw)
    dh = g.gemm_nt_f8_experts(dy, g.quantize_f8(down, 128, transposed=True), r)
    dh = torch.where(h > 0, dh, 0)
    dxs = g.gemm_nt_f8_experts(dh, g.quantize_f8(up, 128, transposed=True), r)
    dx = g.combine_experts(dxs, r, weighted=False)
    ddown = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(h, r), r)
    dup = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dh, r), g.quantize_f8_experts(x, r, gather=True), r)
    dwr = g.matmul(dlogits.t(), x)
    assert dwr.shape == wr.shape and dx.shape == x.shape
    q = ref.quantized
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


@pytest.mark.parametrize("t", [1, 64, 700])
def test_layer_captured(g, t):
    """A captured layer, replayed on inputs that route otherwise."""
    rng = np.random.default_rng(t)
    x, wr, up, down = layer_inputs(g, rng, t, 256, 128, 8)
    up8, down8 = g.quantize_f8(up, 128), g.quantize_f8(down, 128)
    layer(g, x, wr, up8, down8, 2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(g, x, wr, up8, down8, 2)
    for i in range(4):
        x.copy_(dev(rng.standard_normal(tuple(x.shape)).astype(np.float16)))
        graph.replay()
        torch.cuda.synchronize()
        want = layer(g, x, wr, up8, down8, 2)
        for name in ("experts", "weights", "rows", "places", "offsets"):
            assert torch.equal(getattr(got[1], name), getattr(want[1], name))
        assert torch.equal(got[3], want[3]) and torch.equal(got[4], want[4])


def test_experts_on_another_stream(g):
    rng = np.random.default_rng(11)
    x, wr, up, down = layer_inputs(g, rng, 90, 256, 128, 8)
    up8, down8 = g.quantize_f8(up, 128), g.quantize_f8(down, 128)
    logits, r, h, y, out = layer(g, x, wr, up8, down8, 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    r2 = g.route(logits.clone(), 2, "sigmoid", groups=2, top_groups=1, scale=1.5, stream=s)
    y2 = g.gemm_nt_f8_experts(h.clone(), down8, r2, stream=s)
    out2 = g.combine_experts(y2, r2, stream=s)
    dy2, dw2 = g.combine_experts_backward(out2, y2, r2, stream=s)
    dl2 = g.route_backward(logits, r2, dw2, stream=s)
    grad2 = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy2, r2, stream=s), g.quantize_f8_experts(h, r2, stream=s), r2, stream=s)
    s.synchronize()
    assert torch.equal(out2, out)
    dy, dw = g.combine_experts_backward(out, y, r)
    assert torch.equal(dl2, g.route_backward(logits, r, dw))
    assert torch.equal(grad2, g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(h, r), r))


def test_refusals(g):
    x = torch.zeros(4, 128, dtype=torch.float16, device="cuda")
    logits = torch.zeros(4, 8, dtype=torch.float32, device="cuda")
    w = g.quantize_f8(torch.zeros(8, 64, 128, dtype=torch.float16, device="cuda"), 128)
    r = g.route(logits, 2)
    for bad in (dict(top=0), dict(top=9), dict(groups=3), dict(groups=4, top_groups=5), dict(scores="relu"),
                dict(group_score="sum"), dict(bias=torch.zeros(7, device="cuda")), dict(bias=torch.zeros(8))):
        with pytest.raises(ValueError):
            g.route(logits, **{"top": 2, **bad})
    with pytest.raises(TypeError):
        g.route(logits.bfloat16(), 2)
    with pytest.raises(ValueError):
        g.route(logits.cpu(), 2)
    with pytest.raises(ValueError):
        g.route(logits.t(), 2)
    with pytest.raises(ValueError):
        g.gemm_nt_f8_experts(x, w, r)                     # wants the slots' rows
    with pytest.raises(ValueError):
        g.gemm_nt_f8_experts(x.repeat(2, 1), w, r, gather=True)
    with pytest.raises(ValueError):
        g.gemm_nt_f8_experts(x, g.quantize_f8(x, 128), r, gather=True)
    with pytest.raises(ValueError):
        g.gemm_nt_f8_experts(x, g.F8Matrix(w.codes[:7], w.scales[:7], 128, 128), r, gather=True)
    with pytest.raises(TypeError):
        g.gemm_nt_f8_experts(x, w, (r.rows, r.offsets), gather=True)
    with pytest.raises(ValueError):
        g.combine_experts(x, r)
    with pytest.raises(ValueError):
        g.combine_experts_backward(x.repeat(2, 1), x.repeat(2, 1), r)
    with pytest.raises(ValueError):
        g.route_backward(logits, r, torch.zeros(4, 3, device="cuda"))
    with pytest.raises(ValueError):
        g.route_backward(torch.zeros(4, 9, device="cuda"), r, torch.zeros(4, 2, device="cuda"))
    q = g.quantize_f8_experts(x, r, gather=True)
    with pytest.raises(ValueError):
        g.gemm_nt_f8_experts_grad(g.quantize_f8(x), q, r)
    with pytest.raises(TypeError):
        g.Routing(r.experts.long(), r.weights, r.rows, r.places, r.offsets)
    with pytest.raises(ValueError):
        g.Routing(r.experts, r.weights, r.rows[:-1], r.places, r.offsets)
