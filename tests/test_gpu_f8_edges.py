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


# ---- every code --------------------------------------------------------------------
def every_code(gen, r, k):
    """Random codes, the subnormal ones as often as others, no NaN: (codes, values)."""
    codes = torch.randint(0, 127, (r, -(-k // 128) * 128), generator=gen, device="cuda").to(torch.uint8)
    codes |= torch.randint(0, 2, codes.shape, generator=gen, device="cuda").to(torch.uint8) << 7
    codes[:, k:] = 0
    table = torch.from_numpy(ref.code_values()).cuda()
    return codes.view(torch.float8_e4m3fn), table[codes.long()][:, :k]


def ones(r, k):
    """Rows that have a one each, row i in column 7 i mod k."""
    x = torch.zeros(r, -(-k // 128) * 128, device="cuda")
    column = torch.arange(r, device="cuda") * 7 % k
    x[torch.arange(r, device="cuda"), column] = 1.0
    return x.to(torch.float8_e4m3fn), column


def unscaled(g, codes, k, block):
    blocks = -(-codes.shape[0] // block)
    return g.F8Matrix(codes, torch.full((-(-k // 512), blocks, 4), 127, dtype=torch.uint8, device="cuda"), k, block)


@pytest.mark.parametrize("m,n,k", [(1, 300, 1100), (7, 300, 600), (16, 300, 1700), (70, 300, 200), (300, 264, 2048),
                                   (333, 1001, 4000), (1000, 2050, 300), (4097, 2050, 130), (3001, 4096, 130)])
def test_every_code(g, m, n, k):
    """A code times one is that code's number, as A's operand and as B's, in every kernel."""
    gen = generator(m + n)
    codes, values = every_code(gen, m, k)
    one, column = ones(n, k)
    c = g.gemm_nt_f8(unscaled(g, codes, k, 1), unscaled(g, one, k, 128))
    assert torch.equal(c.double(), values[:, column])
    codes, values = every_code(gen, n, k)
    one, column = ones(m, k)
    for block in (1, 128):
        w = unscaled(g, codes, k, block)
        for a in (unscaled(g, one, k, 1), one[:, :k].half()):
            assert torch.equal(g.gemm_nt_f8(a, w).double(), values[:, column].t())


# ---- beyond 32 bits ------------------------------------------------------------------
def big_codes(gen, *shape):
    """Codes of small whole numbers, one in eight not zero."""
    codes = torch.zeros(shape, dtype=torch.uint8, device="cuda")
    table = torch.zeros(32, dtype=torch.uint8, device="cuda")
    table[:4] = torch.tensor([0xc0, 0xb8, 0x38, 0x40], dtype=torch.uint8)
    for part in codes.view(-1).split(2 ** 28):
        part.copy_(table[torch.randint(0, 32, part.shape, generator=gen, device="cuda", dtype=torch.uint8).int()])
    return codes.view(torch.float8_e4m3fn)


def test_stack_beyond_32_bits(g):
    """A stack of experts' matrices past 2^32 bytes of codes: quantised, read back and
    multiplied, forward and both gradients; its first and last matrices as by themselves."""
    gen = generator(1)
    e, n, k, top = 160, 4096, 7168, 2
    w8 = g.F8Matrix(big_codes(gen, e, n, k), torch.randint(126, 129, (e, k // 512, n // 128, 4), generator=gen,
                                                           device="cuda", dtype=torch.uint8), k, 128)
    assert w8.codes.numel() > 2 ** 32
    some = (0, e // 2, e - 1)
    w = g.dequantize_f8(w8)
    alone = {i: g.dequantize_f8(g.F8Matrix(w8.codes[i], w8.scales[i], k, 128)) for i in some}
    assert all(torch.equal(w[i], alone[i]) for i in some)
    again, turned = g.quantize_f8(w, 128), g.quantize_f8(w, 128, transposed=True)
    del w
    for i in some:
        for stack, transposed in ((again, False), (turned, True)):
            one = g.quantize_f8(alone[i], 128, transposed)
            assert torch.equal(stack.codes[i].view(torch.uint8), one.codes.view(torch.uint8))
            assert torch.equal(stack.scales[i], one.scales)
    del again
    for t in (1, 40, 3000):
        logits = torch.randn(t, e, generator=gen, device="cuda")
        logits[:, 0] += 2
        logits[:, e - 1] += 2
        logits[0, e - 1] = 50
        r = g.route(logits, top)
        bounds = r.offsets.tolist()
        assert bounds[e] > bounds[e - 1]
        x, dy = whole_halves(gen, t, k), whole_halves(gen, t * top, n)
        tokens = r.rows.long() // top
        y = g.gemm_nt_f8_experts(x, w8, r, gather=True)
        dx = g.gemm_nt_f8_experts(dy, turned, r)
        dw = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True), r)
        assert dw.numel() * 2 > 2 ** 32
        for i in some:
            lo, hi = bounds[i: i + 2]
            xi, dyi = x[tokens[lo:hi]].double(), dy[lo:hi].double()
            assert torch.equal(y[lo:hi], product(xi, alone[i].double()))
            assert torch.equal(dx[lo:hi], product(dyi, alone[i].double().t()))
            assert torch.equal(dw[i], product(dyi.t().contiguous(), xi.t()))
        del y, dx, dw


def test_matrix_beyond_32_bits(g):
    """Rows of activations past 2^32 codes, and their transpose, whose groups run along
    the rows: a layer's product and its weight's gradient."""
    gen = generator(2)
    t, k, n = 2 ** 20 + 37, 4160, 96
    x = torch.zeros(t, k, dtype=torch.float16, device="cuda")
    for part in x.split(2 ** 16):
        part.copy_(torch.randint(-2, 3, part.shape, generator=gen, device="cuda", dtype=torch.int8))
    x8 = g.quantize_f8(x)
    assert x8.codes.numel() > 2 ** 32
    w = whole_halves(gen, n, k)
    for part in (slice(0, 300), slice(t - 300, t)):
        want = product(x[part].double(), w.double())
        one = g.quantize_f8(x[part].contiguous())
        assert torch.equal(x8.codes[part].view(torch.uint8), one.codes.view(torch.uint8))
        for a in (x, x8):
            assert torch.equal(g.gemm_nt_f8(a, g.quantize_f8(w, 128))[part], want)
    back = g.dequantize_f8(x8)
    assert torch.equal(back[-300:], x[-300:]) and torch.equal(back[:300], x[:300])
    del x8, back
    xt = g.quantize_f8(x, transposed=True)
    assert xt.codes.numel() > 2 ** 32
    # one row in 64 has a gradient, so that sums of whole numbers stay far below 2^24
    dy = torch.zeros(t, n, dtype=torch.float16, device="cuda")
    dy[::64] = whole_halves(gen, len(range(0, t, 64)), n)
    dy[-1] = 1
    want = torch.zeros(n, k, dtype=torch.float64, device="cuda")
    on = dy.any(1).nonzero()[:, 0]
    for part in on.split(4096):
        want += torch.matmul(dy[part].double().t().contiguous(), x[part].double())
    assert want.abs().max() < 2 ** 20
    assert torch.equal(g.gemm_nt_f8(g.quantize_f8(dy, transposed=True), xt), want.half())


def test_output_beyond_32_bits(g):
    """C past 2^32 bytes: its first, middle and last rows."""
    gen = generator(3)
    m, n, k = 36000, 65500, 130
    ac, as_, a = whole(gen, m, k, 1)
    bc, bs, b = whole(gen, n, k, 128)
    c = g.gemm_nt_f8(g.F8Matrix(ac, as_, k, 1), g.F8Matrix(bc, bs, k, 128))
    assert c.numel() * 2 > 2 ** 32
    for part in (slice(0, 260), slice(m // 2, m // 2 + 260), slice(m - 260, m)):
        assert torch.equal(c[part], product(a[part], b))


# ---- what sums keep ------------------------------------------------------------------
def one_row(values, k, scales=None):
    """A row of F8 with the given values by column and, by group, exponents of scales."""
    x = torch.zeros(1, k)
    for column, v in values.items():
        x[0, column] = v
    s = torch.full((-(-k // 512), 1, 4), 127, dtype=torch.uint8)
    for group, e in (scales or {}).items():
        s[group // 4, 0, group % 4] = 127 + e
    return x.to(torch.float8_e4m3fn).cuda(), s.cuda()


@pytest.mark.parametrize("m", [1, 64, 2000])
def test_what_sums_keep(g, m):
    """Of eight neighbouring products all that reaches 2^-13 of the largest; of the sums
    of eight, and from one group to another, what fp32 does.  A large product comes and
    goes, and a small one is left."""
    n = 16 if m < 2000 else 2048

    def left(k, values, scales=None):
        codes, s = one_row(values, k, scales)
        a = g.F8Matrix(codes.repeat(m, 1), s.repeat(1, m, 1), k, 1)
        c = g.gemm_nt_f8(a, g.quantize_f8(torch.ones(n, k, dtype=torch.float16, device="cuda"), 128))
        assert (c == c[0, 0]).all()
        return c[0, 0].item()

    for column in (1, 5, 7):
        assert left(128, {0: 256.0, column: 2.0 ** -5, 120: -256.0}) == 2.0 ** -5
    for column in (8, 31, 32, 64, 119):
        assert left(128, {0: 256.0, column: 2.0 ** -9, 120: -256.0}) == 2.0 ** -9
    for e in (0, 7, 15):
        assert left(384, {0: 256.0, 128: 1.0, 256: -256.0}, {0: e, 2: e}) == 1.0
