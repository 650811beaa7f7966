"""Products in 8-bit floating point at the edges of what their header allows."""
import numpy as np
import pytest
import torch

import f8_ref as ref
from test_gpu_f8 import g, host  # noqa: F401  (g: the fixture)
from test_gpu_f8_tiles import generator, guarded, product, uneven, whole, whole_halves

pytestmark = pytest.mark.gpu


# ---- A in fp16 and in F8 ----------------------------------------------------------
@pytest.mark.parametrize("m,k", [(1, 1500), (1, 2560), (7, 4096), (16, 2048), (40, 2560), (300, 2560)])
def test_sums_in_another_order(g, m, k):
    """Sums whose terms cancel from far above the result: A in fp16 and A in F8 are the
    same codes, which kernels may add in another order, each within the bound."""
    gen = generator(m + k)
    n = 200
    x = torch.randint(-2, 3, (m, k), device="cuda", generator=gen).half()
    w = torch.randint(-2, 3, (n, k), device="cuda", generator=gen).half()
    x[:, :128] = 0
    x[:, k - 128:] = 0
    x[:, 0], x[:, k - 1] = 2.0 ** 15, -2.0 ** 15      # in groups of their own: 2^25 comes and goes
    w[:, 0] = w[:, k - 1] = 2.0 ** 10
    w[:, 1:128] = 0
    w[:, k - 128:k - 1] = 0
    w8 = g.quantize_f8(w)
    a, b = host(x).astype(np.float64), host(w).astype(np.float64)
    exact, size = a @ b.T, np.abs(a) @ np.abs(b).T
    bound = ref.product_bound(size, exact, k)
    halves, codes = g.gemm_nt_f8(x, w8), g.gemm_nt_f8(g.quantize_f8(x), w8)
    for got in (halves, codes):
        assert (np.abs(host(got).astype(np.float64) - exact) <= bound).all()
    # without those columns every sum is a small whole number: the same whatever the order
    x[:, 0] = x[:, k - 1] = 0
    assert torch.equal(g.gemm_nt_f8(x, w8), g.gemm_nt_f8(g.quantize_f8(x), w8))


# ---- every kernel ------------------------------------------------------------------
# (rows and columns of a tile, waves): the kernels that a plan can name
STREAMS = {(16, 16, 8), (16, 16, 16)}
TILES = {(32, 64, 2), (64, 64, 4), (64, 128, 4), (128, 128, 4), (256, 192, 4), (256, 256, 4)}


def named(plan):
    return plan.block_m, plan.block_n, plan.waves


def compute_units(g):
    cus = g.gemm_f16_device_cus()
    if cus != 256:
        pytest.skip("the sizes are for 256 compute units")
    return cus


# m, n, k: A in fp16, up to 16 rows of it, by 8 and by 16 waves
STREAMED = [(1, 22, 2827), (2, 300, 4100), (5, 130, 3300), (7, 300, 4600), (13, 65, 1700), (16, 70, 2048),
            (1, 17, 65), (2, 300, 1536), (7, 31, 600), (16, 100, 1500), (3, 130, 9000), (1, 4097, 32768)]


def test_streams_are_reached(g):
    cus = compute_units(g)
    rows = {}
    for m, n, k in STREAMED:
        rows.setdefault(named(g.gemm_f16_nt_f8_plan(m, n, k, 128, True, cus)), set()).add(m)
    assert set(rows) == STREAMS
    assert all({1, 2, 7, 16} <= of for of in rows.values())


@pytest.mark.parametrize("m,n,k", STREAMED)
@pytest.mark.parametrize("block", [1, 128])
def test_streamed(g, m, n, k, block):
    gen = generator(m + n + k)
    x = whole_halves(gen, m, k)
    bc, bs, b = whole(gen, n, k, block)
    out, around = guarded((m, n))
    g.gemm_nt_f8(x, g.F8Matrix(bc, bs, k, block), out=out)
    assert torch.equal(out, product(x.double(), b))
    assert all((v == 3).all() for v in around)


# t, e, top, n, k, A in fp16
EXPERTS = [(13, 2, 2, 34, 279, True), (20, 8, 3, 100, 1000, True), (5, 4, 2, 130, 3400, True),
           (40, 16, 2, 37, 1800, True), (7, 2, 1, 17, 4224, True), (362, 16, 5, 21, 77, True),
           (100, 32, 2, 70, 500, False), (2748, 8, 3, 22, 67, True), (3015, 16, 3, 19, 258, False),
           (1131, 4, 1, 775, 88, True), (34, 32, 5, 515, 64, False), (460, 16, 2, 1538, 97, True),
           (5905, 4, 3, 20, 64, False), (7079, 32, 1, 911, 128, True), (8230, 8, 5, 147, 138, False),
           (506, 32, 5, 1689, 131, True), (2795, 8, 5, 1905, 65, False)]


@pytest.mark.parametrize("gather", [True, False])
def test_experts_reach_every_kernel(g, gather):
    cus = compute_units(g)
    reached = {True: set(), False: set()}
    for t, e, top, n, k, f16 in EXPERTS:
        plan = g.gemm_f16_nt_f8_experts_plan(t * top, e, n, k, top if gather else 0, f16, cus)
        reached[f16].add(named(plan))
    assert reached == {True: STREAMS | TILES, False: TILES}


@pytest.mark.parametrize("t,e,top,n,k,f16", EXPERTS)
@pytest.mark.parametrize("gather", [True, False])
def test_experts(g, t, e, top, n, k, f16, gather):
    gen = generator(t + e)
    r = g.route(uneven(gen, t, e, top), top)
    bounds = r.offsets.tolist()
    x = whole_halves(gen, t if gather else t * top, k)
    wc, ws, w = whole(gen, n, k, 128, count=e)
    out, around = guarded((t * top, n))
    g.gemm_nt_f8_experts(x if f16 else g.quantize_f8(x), g.F8Matrix(wc, ws, k, 128), r, gather=gather, out=out)
    a = x.double()
    if gather:
        a = a[r.rows.long().clamp(min=0) // top]
    for i in range(e):
        lo, hi = bounds[i: i + 2]
        assert torch.equal(out[lo:hi], product(a[lo:hi], w[i])), i
    assert (out[bounds[-1]:] == 0).all()
    assert all((v == 3).all() for v in around)


# t, e, top, n, k
GRADIENTS = [(34, 8, 2, 30, 81), (9, 4, 4, 1042, 77), (20, 16, 2, 33, 539), (29, 64, 1, 16, 263), (300, 16, 3, 515, 64),
             (200, 2, 2, 259, 3648), (700, 32, 4, 134, 1035), (312, 64, 6, 156, 782)]


def test_gradients_reach_every_kernel(g):
    cus = compute_units(g)
    assert {named(g.gemm_f16_nt_f8_experts_grad_plan(t * top, e, n, k, cus)) for t, e, top, n, k in GRADIENTS} == TILES


@pytest.mark.parametrize("t,e,top,n,k", GRADIENTS)
def test_experts_gradient(g, t, e, top, n, k):
    gen = generator(t + n)
    r = g.route(uneven(gen, t, e, top), top)
    bounds = r.offsets.tolist()
    dy, x = whole_halves(gen, t * top, n), whole_halves(gen, t, k)
    out, around = guarded((e, n, k))
    g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True), r, out=out)
    xs = x[r.rows.long().clamp(min=0) // top].double()
    for i in range(e):
        lo, hi = bounds[i: i + 2]
        assert torch.equal(out[i], product(dy[lo:hi].double().t().contiguous(), xs[lo:hi].t().contiguous())), i
    assert all((v == 3).all() for v in around)
