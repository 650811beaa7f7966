"""The 4-bit and 8-bit forms and their products on the GPU, against plain
64-bit references (lowbit_ref.py)."""
import numpy as np
import pytest

import lowbit_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import torch

    import dense_fp16_gemm_amd as lib

    lib.load()
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return lib


def dev(x):
    import torch

    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def host(t):
    return t.cpu().numpy()


def spread(rng, shape):
    """fp16 values over all magnitudes, signs, zeros and subnormals."""
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-26, 14, (shape[0], 1)).astype(float))
    return np.clip(x, -65504, 65504).astype(np.float16)


# ---- quantising ---------------------------------------------------------------
W4_SHAPES = [(16, 128, 128), (1, 1, 32), (1, 128, 64), (17, 129, 64), (37, 300, 32), (37, 300, 64),
             (37, 301, 128), (15, 31, 32), (100, 4160, 128), (250, 97, 64), (33, 1000, 32)]


@pytest.mark.parametrize("n,k,group", W4_SHAPES)
def test_w4_quantize_exact(g, n, k, group):
    rng = np.random.default_rng(n * 1000 + k)
    w = spread(rng, (n, k))
    q = g.quantize_w4(dev(w), group)
    codes, scales = ref.encode(w, group, **ref.W4)
    assert (host(q.words) == ref.w4_words(codes[:, :k])).all()
    want = ref.w4_scales(scales, n, k, group, 2.0 ** -24)
    assert (host(q.scales).astype(np.float64) == want).all()
    got = host(g.dequantize_w4(q)).astype(np.float64)
    assert (got == ref.values(codes, scales, group, k)).all()


def test_w4_quantize_every_half(g):
    """All finite fp16 numbers as the largest of a group, with smaller ones
    that fall on and next to ties."""
    rng = np.random.default_rng(5)
    top = np.arange(0, 0x7c00, dtype=np.uint16).view(np.float16)
    w = (top[:, None].astype(np.float64) * rng.uniform(-1, 1, (top.size, 32))).astype(np.float16)
    w[:, 7] = top
    w[:, 8] = -top
    s = ref.encode(w, 32, **ref.W4)[1][:, 0]
    for i, tie in enumerate((0.5, 1.5, 2.5, 3.5, 4.5, 5.5, 6.5)):
        t = s * tie
        w[:, 10 + i] = np.where(t <= top, t, 0).astype(np.float16)
    codes, scales = ref.encode(w, 32, **ref.W4)
    q = g.quantize_w4(dev(w), 32)
    assert (host(q.words) == ref.w4_words(codes)).all()
    assert (host(g.dequantize_w4(q)).astype(np.float64) == ref.values(codes, scales, 32, 32)).all()


def test_q8_quantize_every_half(g):
    rng = np.random.default_rng(6)
    top = np.arange(0, 0x7c00, dtype=np.uint16).view(np.float16)
    x = (top[:, None].astype(np.float64) * rng.uniform(-1, 1, (top.size, 32))).astype(np.float16)
    x[:, 3] = top
    x[:, 4] = -top
    s = ref.encode(x, 32, **ref.Q8)[1][:, 0]
    for i, tie in enumerate((0.5, 1.5, 2.5, 62.5, 63.5, 100.5, 113.5, 125.5, 126.5)):
        t = s * tie
        x[:, 10 + i] = np.where(t <= top, t, 0).astype(np.float16)
    codes, scales = ref.encode(x, 32, **ref.Q8)
    q = g.quantize_q8(dev(x))
    assert (host(q.codes) == codes).all()
    assert (host(q.scales).astype(np.float64) == scales).all()
    got = host(g.dequantize_q8(q)).astype(np.float64)
    assert np.isfinite(got).all() and (got == ref.values(codes, scales, 32, 32)).all()


@pytest.mark.parametrize("r,n", [(1, 1), (1, 32), (3, 33), (5, 8), (64, 512), (65, 513), (7, 1000),
                                 (300, 70), (1000, 31), (129, 4160), (2, 20001)])
def test_q8_quantize_exact(g, r, n):
    rng = np.random.default_rng(r * 1000 + n)
    x = spread(rng, (r, n))
    q = g.quantize_q8(dev(x))
    codes, scales = ref.encode(x, 32, **ref.Q8)
    assert q.shape == (r, n)
    assert (host(q.codes) == codes).all()
    assert (host(q.scales).astype(np.float64) == scales).all()
    assert (host(g.dequantize_q8(q)).astype(np.float64) == ref.values(codes, scales, 32, n)).all()


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_non_finite_groups(g, value):
    rng = np.random.default_rng(8)
    x = rng.standard_normal((20, 300)).astype(np.float16)
    x[3, 70] = value
    x[19, 299] = value
    for group, quant, back, form in ((64, lambda t: g.quantize_w4(t, 64), g.dequantize_w4, ref.W4),
                                     (32, g.quantize_q8, g.dequantize_q8, ref.Q8)):
        codes, scales = ref.encode(x, group, **form)
        want = ref.values(codes, scales, group, 300)
        got = host(back(quant(dev(x)))).astype(np.float64)
        nan = np.zeros((20, 300), bool)
        for r, c in ((3, 70), (19, 299)):
            nan[r, c // group * group:(c // group + 1) * group] = True
        assert (np.isnan(got) == nan).all()
        assert (got[~nan] == want[~nan]).all()


@pytest.mark.parametrize("n,k,group", W4_SHAPES)
def test_w4_pack(g, n, k, group):
    rng = np.random.default_rng(n + k)
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    scales = (rng.uniform(-1, 1, (n, -(-k // group))) *
              np.exp2(rng.integers(-26, 12, (n, 1)).astype(float))).astype(np.float16)
    q = g.pack_w4(dev(codes), dev(scales), group)
    r = ref.round8(scales)
    assert (host(q.words) == ref.w4_words(codes)).all()
    assert (host(q.scales).astype(np.float64) == ref.w4_scales(r, n, k, group, 0.0)).all()
    full = np.zeros((n, -(-k // group) * group), np.int64)
    full[:, :k] = codes
    assert (host(g.dequantize_w4(q)).astype(np.float64) == ref.values(full, r, group, k)).all()


def test_group_from_numpy(g):
    """A group size out of an array or a configuration is as good as an int."""
    q = g.quantize_w4(dev(np.full((5, 70), 7, np.float16)), np.int64(64))
    p = g.pack_w4(dev(np.full((5, 70), 7, np.int8)), dev(np.ones((5, 2), np.float16)), np.int32(64))
    assert q.group == p.group == 64
    assert (host(g.dequantize_w4(q)) == 7).all() and (host(g.dequantize_w4(p)) == 7).all()


def test_w4_pack_refuses_groups(g):
    """What four bits or fp16 do not hold makes its group NaN, and no other."""
    codes = np.ones((16, 256), np.int8)
    scales = np.ones((16, 4), np.float16)
    codes[0, 5] = 8
    codes[1, 70] = -9
    codes[2, 130] = 127
    codes[3, 255] = -128
    scales[4, 0] = np.inf
    scales[5, 1] = np.nan
    scales[6, 2], codes[6, 128] = 8192.0, -8     # 65536 passes fp16
    scales[7, 3], codes[7, 192] = 8160.0, -8     # 65280 does not
    scales[8, 0] = 65504.0                       # rounds to 65536
    got = host(g.dequantize_w4(g.pack_w4(dev(codes), dev(scales), 64))).astype(np.float64)
    nan = np.zeros((16, 4), bool)
    for r, c in ((0, 0), (1, 1), (2, 2), (3, 3), (4, 0), (5, 1), (6, 2), (8, 0)):
        nan[r, c] = True
    assert (np.isnan(got).reshape(16, 4, 64) == nan[:, :, None]).all()
    assert got[7, 192] == -65280.0 and got[7, 193] == 8160.0


@pytest.mark.parametrize("off", [1, 3])
def test_unaligned_matrices(g, off):
    """fp16 matrices at 2-byte offsets, and nothing written around the outputs."""
    import torch

    rng = np.random.default_rng(off)
    n, k = 37, 203
    x = rng.standard_normal((n, k)).astype(np.float16)
    buf = torch.zeros(n * k + 16, dtype=torch.float16, device="cuda")
    src = buf[off:off + n * k].view(n, k)
    src.copy_(dev(x))
    for quant, back in ((lambda t: g.quantize_w4(t, 32), g.dequantize_w4),
                        (g.quantize_q8, g.dequantize_q8)):
        q, q0 = quant(src), quant(dev(x))
        out = torch.full((n * k + 16,), 7.0, dtype=torch.float16, device="cuda")
        back(q, out=out[off:off + n * k].view(n, k))
        assert (host(out[off:off + n * k].view(n, k)) == host(back(q0))).all()
        assert (host(out[:off]) == 7).all() and (host(out[off + n * k:]) == 7).all()


# ---- products -------------------------------------------------------------------
def w4_case(rng, n, k, group, integers):
    codes = rng.integers(-8, 8, (n, k)).astype(np.int8)
    if integers:
        scales = np.exp2(rng.integers(-2, 2, (n, -(-k // group))).astype(float)).astype(np.float16)
    else:
        scales = ref.round8((rng.uniform(0.5, 1.5, (n, -(-k // group))) / np.sqrt(k))
                            .astype(np.float16)).astype(np.float16)
    full = np.zeros((n, -(-k // group) * group), np.int64)
    full[:, :k] = codes
    return codes, scales, ref.values(full, scales, group, k)


def check_product(got, a, b, k, integers):
    """got against a @ b (float64 operands)."""
    want = a @ b
    got = got.astype(np.float64)
    if integers:
        # every partial sum is exact in fp32; rounded once to fp16
        with np.errstate(over="ignore"):
            assert (got == want.astype(np.float16).astype(np.float64)).all()
        return
    bound = ref.product_bound(np.abs(a) @ np.abs(b), want, k)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size}, worst {np.abs(got - want).max()}"


PRODUCT_M = [1, 2, 3, 5, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 100, 128, 129, 200, 300, 513]
PRODUCT_NK = [(16, 32, 32), (1, 1, 64), (7, 130, 64), (64, 128, 128), (130, 257, 32),
              (100, 1000, 128), (272, 2048, 64), (33, 4160, 128)]


@pytest.mark.parametrize("n,k,group", PRODUCT_NK)
@pytest.mark.parametrize("m", PRODUCT_M)
def test_nt_w4(g, m, n, k, group):
    for integers in (False, True):
        rng = np.random.default_rng(m * 7919 + n * 31 + k)
        codes, scales, w = w4_case(rng, n, k, group, integers)
        a = rng.integers(-3, 4, (m, k)) if integers else rng.standard_normal((m, k))
        a = a.astype(np.float16)
        got = host(g.gemm_nt_w4(dev(a), g.pack_w4(dev(codes), dev(scales), group)))
        check_product(got, a.astype(np.float64), w.T, k, integers)


@pytest.mark.parametrize("m,n,k,group", [(1, 4096, 14336, 128), (16, 1024, 16384, 32),
                                         (5, 7001, 4160, 64), (64, 2048, 8192, 128),
                                         (333, 1111, 4096, 64), (1500, 2048, 2048, 128)])
def test_nt_w4_large(g, m, n, k, group):
    rng = np.random.default_rng(m + n + k)
    codes, scales, w = w4_case(rng, n, k, group, False)
    a = rng.standard_normal((m, k)).astype(np.float16)
    got = host(g.gemm_nt_w4(dev(a), g.pack_w4(dev(codes), dev(scales), group)))
    check_product(got, a.astype(np.float64), w.T, k, False)


def q8_case(rng, r, n, integers):
    groups = -(-n // 32)
    codes = np.zeros((r, groups * 32), np.int8)
    codes[:, :n] = rng.integers(-4, 5, (r, n)) if integers else rng.integers(-127, 128, (r, n))
    if integers:
        scales = np.exp2(rng.integers(-1, 2, (r, groups)).astype(float)).astype(np.float16)
    else:
        m = rng.integers(8, 16, (r, groups)) * np.exp2(rng.integers(-11, -8, (r, groups)))
        scales = m.astype(np.float16)
    return codes, scales, ref.values(codes, scales, 32, n)


@pytest.mark.parametrize("n,k", [(32, 1), (1, 40), (33, 64), (70, 100), (256, 31), (257, 33),
                                 (300, 1024), (512, 333), (1000, 2000), (100, 5000)])
@pytest.mark.parametrize("m", [1, 2, 7, 8, 15, 16, 17, 32, 33, 48, 64, 65, 128, 200])
def test_tn_q8(g, m, n, k):
    for integers in (False, True):
        rng = np.random.default_rng(m * 7919 + n * 31 + k)
        codes, scales, x = q8_case(rng, k, n, integers)
        a = rng.integers(-3, 4, (k, m)) if integers else rng.standard_normal((k, m))
        a = a.astype(np.float16)
        got = host(g.gemm_tn_q8(dev(a), g.Q8Matrix(dev(codes), dev(scales), n)))
        check_product(got, a.astype(np.float64).T, x, k, integers)


@pytest.mark.parametrize("m,n,k", [(16, 4096, 8192), (64, 1024, 4999), (1024, 1056, 3000),
                                   (2048, 512, 1111), (5, 14336, 8192), (24, 2000, 8000),
                                   (256, 1000, 4097), (400, 256, 3001)])
def test_tn_q8_large(g, m, n, k):
    rng = np.random.default_rng(m + n + k)
    codes, scales, x = q8_case(rng, k, n, False)
    a = (rng.standard_normal((k, m)) / np.sqrt(k)).astype(np.float16)
    got = host(g.gemm_tn_q8(dev(a), g.Q8Matrix(dev(codes), dev(scales), n)))
    check_product(got, a.astype(np.float64).T, x, k, False)


def check_on_gpu(got, a, b, k):
    """check_product for large sizes: the 64-bit product on the GPU."""
    import torch

    a, b = a.double(), b.double()
    want = torch.matmul(a, b)
    fp32 = (k / 4 + k / 32 + 72) * 2.0 ** -24 * torch.matmul(a.abs(), b.abs())   # see product_bound
    bound = fp32 + (want.abs() + fp32) * 2.0 ** -11 + 2.0 ** -25
    bad = ~((got.double() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}"


# a shape for each kernel of the planner's table on 256 compute units, unsplit
# and split: (kernel, rows, columns, waves), then M, N, K
W4_KERNELS = [((1, 4, 16, 8), 3, 500, 1000), ((1, 8, 16, 8), 5, 500, 3000),
              ((1, 8, 32, 8), 7, 6500, 700), ((1, 16, 16, 8), 12, 500, 3000),
              ((1, 16, 32, 8), 16, 6500, 700), ((1, 16, 64, 8), 9, 12800, 520),
              ((1, 32, 16, 8), 17, 70, 32), ((1, 32, 16, 8), 30, 1000, 3000),
              ((1, 32, 32, 4), 24, 6500, 700), ((1, 32, 32, 4), 32, 6500, 2001),
              ((1, 32, 64, 8), 17, 12800, 700), ((1, 32, 64, 8), 29, 12801, 4001),
              ((1, 48, 16, 8), 40, 70, 700), ((1, 48, 16, 8), 48, 1000, 2100),
              ((1, 48, 32, 4), 33, 6500, 700), ((1, 48, 32, 4), 45, 6500, 2048),
              ((1, 48, 64, 4), 40, 12800, 2048), ((1, 48, 64, 4), 47, 12801, 3000),
              ((2, 32, 128, 4), 40, 70, 32), ((2, 32, 128, 4), 60, 1000, 700),
              ((2, 48, 256, 8), 333, 6500, 32), ((2, 48, 256, 8), 40, 6500, 8000),
              ((2, 64, 128, 8), 80, 12800, 700), ((2, 64, 128, 8), 60, 6500, 2048),
              ((2, 64, 128, 8), 333, 1000, 2000), ((2, 64, 128, 8), 500, 4001, 4100),
              ((2, 64, 256, 8), 200, 16384, 32), ((2, 64, 256, 8), 60, 12800, 8000),
              ((2, 96, 128, 8), 160, 12800, 700), ((2, 96, 128, 8), 80, 6500, 4096),
              ((2, 96, 256, 8), 333, 12800, 32), ((2, 96, 256, 8), 80, 12800, 8000),
              ((2, 112, 256, 8), 512, 12800, 32), ((2, 112, 256, 8), 112, 6500, 8000),
              ((2, 128, 256, 8), 512, 16384, 32), ((2, 128, 256, 8), 120, 12800, 8000),
              ((0,), 1500, 14336, 4096), ((0,), 2200, 7001, 4001)]


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("kernel,m,n,k", W4_KERNELS)
def test_nt_w4_every_kernel(g, kernel, m, n, k, group):
    import torch

    plan = g.gemm_f16_nt_w4_plan(m, n, k, group, 256)
    assert (plan.kernel, plan.block_m, plan.block_n, plan.waves)[:len(kernel)] == kernel
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    codes = torch.randint(-8, 8, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    # one row's scales past 2720, where the tile kernels unpack otherwise
    scales = torch.rand(n, -(-k // group), generator=gen, device="cuda") + 0.5
    scales[n // 2] *= 4000.0
    q = g.pack_w4(codes, scales.half(), group)
    a = (torch.randn(m, k, generator=gen, device="cuda") / k).half()
    check_on_gpu(g.gemm_nt_w4(a, q), a, g.dequantize_w4(q).t(), k)


# the same for the 8-bit product, and the ranges that its rows are split into
Q8_KERNELS = [((1, 16, 128, 4), 1, 7, 1000, 5), ((1, 16, 128, 4), 1, 16, 300, 500),
              ((1, 16, 128, 4), 28, 40, 300, 8000), ((1, 16, 256, 4), 4, 10, 14336, 8192),
              ((1, 16, 256, 4), 1, 7, 60000, 33), ((1, 32, 128, 4), 16, 30, 2000, 8000),
              ((1, 32, 128, 4), 1, 1500, 333, 40), ((1, 64, 128, 4), 2, 130, 4096, 4000),
              ((1, 64, 128, 4), 3, 1069, 463, 2357), ((1, 64, 128, 4), 2, 1001, 999, 8001),
              ((1, 64, 128, 4), 1, 100, 14337, 33), ((0,), 1, 1600, 1608, 3000),
              ((0,), 1, 1601, 1608, 2357), ((0,), 1, 1600, 1603, 1500), ((0,), 1, 1601, 1603, 2357),
              ((0,), 3, 3000, 300, 2357), ((0,), 4, 333, 4096, 8000), ((0,), 5, 1500, 999, 8000),
              ((1, 64, 128, 4), 1, 3001, 1999, 70), ((1, 32, 128, 4), 1, 1500, 300, 3),
              ((1, 16, 256, 4), 1, 130, 7001, 45)]


@pytest.mark.parametrize("kernel,splits,m,n,k", Q8_KERNELS)
def test_tn_q8_every_kernel(g, kernel, splits, m, n, k):
    import torch

    plan = g.gemm_f16_tn_q8_plan(m, n, k, 256)
    assert plan.splits == splits
    assert (plan.kernel, plan.block_m, plan.block_n, plan.waves)[:len(kernel)] == kernel
    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    x = g.quantize_q8(torch.randn(k, n, generator=gen, device="cuda").half())
    a = (torch.randn(k, m, generator=gen, device="cuda") / k).half()
    check_on_gpu(g.gemm_tn_q8(a, x), a.t().contiguous(), g.dequantize_q8(x), k)


@pytest.mark.parametrize("m", [1, 16, 40, 100, 1200])
def test_nt_w4_special_values(g, m):
    """Infinities and NaN reach the results that the definition gives them, and
    no other; a group of zeros is zero; the largest weights do not overflow."""
    rng = np.random.default_rng(m)
    n, k = 40, 320
    codes = rng.integers(1, 8, (n, k)).astype(np.int8)     # no zero: inf times 0 is NaN
    scales = np.full((n, 5), 2.0 ** -6, np.float16)
    a = rng.integers(1, 4, (m, k)).astype(np.float16)
    scales[3, 2] = np.nan
    codes[7, 64:128] = 0
    scales[9, :], codes[9, :] = 8160.0, 0
    codes[9, 5] = -8
    a[0, :] = 0
    a[0, 5] = 1.0
    if m > 4:
        a[4, 300] = np.inf
    q = g.pack_w4(dev(codes), dev(scales), 64)
    full = codes.astype(np.int64)
    w = ref.values(full, ref.round8(scales), 64, k)
    with np.errstate(all="ignore"):
        want = (a.astype(np.float64)[:, None, :] * w[None]).sum(-1).astype(np.float16)
    got = host(g.gemm_nt_w4(dev(a), q))
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    assert (got[ok] == want[ok]).all()
    assert got[0, 9] == -65280.0


@pytest.mark.parametrize("m", [4, 40, 300])
def test_tn_q8_special_values(g, m):
    rng = np.random.default_rng(m)
    n, k = 100, 200
    codes = rng.integers(1, 5, (k, 128)).astype(np.int8)
    codes[:, n:] = 0
    scales = np.full((k, 4), 0.5, np.float16)
    scales[50, 1] = np.nan
    a = rng.integers(1, 3, (k, m)).astype(np.float16)
    a[120, 2] = np.inf
    a[121, 3] = np.nan
    x = ref.values(codes, scales, 32, n)
    with np.errstate(all="ignore"):
        want = (a.astype(np.float64)[:, :, None] * x[:, None, :]).sum(0).astype(np.float16)
    got = host(g.gemm_tn_q8(dev(a), g.Q8Matrix(dev(codes), dev(scales), n)))
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    assert (got[ok] == want[ok]).all()


def test_empty(g):
    import torch

    f16 = dict(dtype=torch.float16, device="cuda")
    for n, k in ((0, 64), (64, 0), (0, 0)):
        q = g.quantize_w4(torch.zeros(n, k, **f16), 32)
        assert tuple(g.dequantize_w4(q).shape) == (n, k)
        got = g.gemm_nt_w4(torch.zeros(3, k, **f16), q, out=torch.full((3, n), 5.0, **f16))
        assert tuple(got.shape) == (3, n) and (host(got) == 0).all()
        c = g.quantize_q8(torch.zeros(n, k, **f16))
        assert tuple(g.dequantize_q8(c).shape) == (n, k)
        got = g.gemm_tn_q8(torch.zeros(n, 3, **f16), c, out=torch.full((3, k), 5.0, **f16))
        assert tuple(got.shape) == (3, k) and (host(got) == 0).all()
    q = g.quantize_w4(torch.ones(32, 64, **f16), 32)
    assert tuple(g.gemm_nt_w4(torch.zeros(0, 64, **f16), q).shape) == (0, 32)
    c = g.quantize_q8(torch.ones(32, 64, **f16))
    assert tuple(g.gemm_tn_q8(torch.zeros(32, 0, **f16), c).shape) == (0, 64)


@pytest.mark.parametrize("k", [333, 336])
@pytest.mark.parametrize("m", [1, 5, 17, 64, 100, 600])
def test_nt_w4_unaligned_and_in_bounds(g, m, k):
    """Operands at 2-byte offsets; nothing around C is written, and what lies
    around A (NaN here) does not enter."""
    import torch

    rng = np.random.default_rng(m)
    n = 71
    codes, scales, w = w4_case(rng, n, k, 64, False)
    a = rng.standard_normal((m, k)).astype(np.float16)
    q = g.pack_w4(dev(codes), dev(scales), 64)
    ab = torch.full((m * k + 600,), float("nan"), dtype=torch.float16, device="cuda")
    av = ab[301:301 + m * k].view(m, k)
    av.copy_(dev(a))
    cb = torch.full((m * n + 64,), 7.0, dtype=torch.float16, device="cuda")
    g.gemm_nt_w4(av, q, out=cb[33:33 + m * n].view(m, n))
    check_product(host(cb[33:33 + m * n].view(m, n)), a.astype(np.float64), w.T, k, False)
    assert (host(cb[:33]) == 7).all() and (host(cb[33 + m * n:]) == 7).all()


@pytest.mark.parametrize("m", [1, 5, 17, 64, 100])
def test_tn_q8_unaligned_and_in_bounds(g, m):
    import torch

    rng = np.random.default_rng(m)
    n, k = 71, 333
    codes, scales, x = q8_case(rng, k, n, False)
    a = rng.standard_normal((k, m)).astype(np.float16)
    ab = torch.full((m * k + 600,), float("nan"), dtype=torch.float16, device="cuda")
    av = ab[301:301 + m * k].view(k, m)
    av.copy_(dev(a))
    sb = torch.full((scales.size + 64,), float("nan"), dtype=torch.float16, device="cuda")
    sv = sb[33:33 + scales.size].view(*scales.shape)
    sv.copy_(dev(scales))
    cb = torch.full((m * n + 64,), 7.0, dtype=torch.float16, device="cuda")
    g.gemm_tn_q8(av, g.Q8Matrix(dev(codes), sv, n), out=cb[33:33 + m * n].view(m, n))
    check_product(host(cb[33:33 + m * n].view(m, n)), a.astype(np.float64).T, x, k, False)
    assert (host(cb[:33]) == 7).all() and (host(cb[33 + m * n:]) == 7).all()


def test_rows_of_a_checkpoint(g):
    """A range of rows is a Q8Matrix too, and gradients over ranges add up."""
    rng = np.random.default_rng(11)
    codes, scales, x = q8_case(rng, 300, 200, True)
    a = rng.integers(-3, 4, (300, 24)).astype(np.float16)
    c, s, ad = dev(codes), dev(scales), dev(a)
    total = np.zeros((24, 200))
    for lo, hi in ((0, 1), (1, 130), (130, 300)):
        part = host(g.gemm_tn_q8(ad[lo:hi], g.Q8Matrix(c[lo:hi], s[lo:hi], 200)))
        check_product(part, a[lo:hi].astype(np.float64).T, x[lo:hi], hi - lo, True)
        total += part
    assert (total == a.astype(np.float64).T @ x).all()


# ---- how they are called --------------------------------------------------------
W4_CALLS = [(1, 512, 1024), (24, 512, 1024), (80, 512, 1024), (1200, 512, 256)]
Q8_CALLS = [(16, 512, 2000), (50, 512, 2000), (512, 1024, 2000), (1200, 1024, 2000)]


def products(g, rng):
    """(call(out, workspace, stream), workspace bytes, shape of C) for each path."""
    import torch

    cus = torch.cuda.get_device_properties(0).multi_processor_count
    for m, n, k in W4_CALLS:
        codes, scales, _ = w4_case(rng, n, k, 64, False)
        q, a = g.pack_w4(dev(codes), dev(scales), 64), dev(rng.standard_normal((m, k)).astype(np.float16))
        need = g.gemm_f16_nt_w4_plan(m, n, k, 64, cus).workspace_bytes
        yield (lambda q=q, a=a, **kw: g.gemm_nt_w4(a, q, **kw)), need, (m, n)
    for m, n, k in Q8_CALLS:
        codes, scales, _ = q8_case(rng, k, n, False)
        c, a = g.Q8Matrix(dev(codes), dev(scales), n), dev(rng.standard_normal((k, m)).astype(np.float16))
        need = g.gemm_f16_tn_q8_plan(m, n, k, cus).workspace_bytes
        yield (lambda c=c, a=a, **kw: g.gemm_tn_q8(a, c, **kw)), need, (m, n)


def test_graph_replays(g):
    """Captured calls give the eager result on every replay, with eager work on
    the same operands in between, whatever the workspace held."""
    import torch

    for call, need, shape in products(g, np.random.default_rng(21)):
        eager = host(call())
        out = torch.empty(shape, dtype=torch.float16, device="cuda")
        ws = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            call(out=out, workspace=ws)
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=s):
                call(out=out, workspace=ws)
        for _ in range(4):
            out.fill_(float("nan"))
            ws.fill_(0xFF)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert (host(out) == eager).all()
            assert (host(call()) == eager).all()


def test_quantisers_in_a_graph(g):
    import torch

    rng = np.random.default_rng(22)
    x = dev(rng.standard_normal((100, 300)).astype(np.float16))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        g.dequantize_w4(g.quantize_w4(x)), g.dequantize_q8(g.quantize_q8(x))
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=s):
            a, b = g.dequantize_w4(g.quantize_w4(x)), g.dequantize_q8(g.quantize_q8(x))
    for _ in range(3):
        x.copy_(dev(rng.standard_normal((100, 300)).astype(np.float16)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert (host(a) == host(g.dequantize_w4(g.quantize_w4(x)))).all()
        assert (host(b) == host(g.dequantize_q8(g.quantize_q8(x)))).all()


def test_same_bits_on_another_stream(g):
    """A stream passed in, its outputs and workspace allocated by the call, with
    the default stream busy and the operands dropped at once."""
    import torch

    s = torch.cuda.Stream()
    for call, _, _ in products(g, np.random.default_rng(23)):
        want = host(call())
        s.wait_stream(torch.cuda.current_stream())
        outs = [call(stream=s) for _ in range(3)]
        s.synchronize()
        for out in outs:
            assert (host(out) == want).all()
    x = dev(np.random.default_rng(2).standard_normal((64, 4096)).astype(np.float16))
    want4, want8 = host(g.dequantize_w4(g.quantize_w4(x))), host(g.dequantize_q8(g.quantize_q8(x)))
    s.wait_stream(torch.cuda.current_stream())
    got4 = g.dequantize_w4(g.quantize_w4(x, stream=s), stream=s)
    got8 = g.dequantize_q8(g.quantize_q8(x, stream=s), stream=s)
    s.synchronize()
    assert (host(got4) == want4).all() and (host(got8) == want8).all()


def test_repeated_calls_same_bits(g):
    for call, _, _ in products(g, np.random.default_rng(24)):
        first = host(call())
        for _ in range(3):
            assert (host(call()) == first).all()


def test_refusals(g):
    import torch

    f16 = dict(dtype=torch.float16, device="cuda")
    q = g.quantize_w4(torch.ones(32, 64, **f16), 32)
    c = g.quantize_q8(torch.ones(32, 64, **f16))
    a = torch.ones(4, 64, **f16)
    for bad in (a.float(), a.cpu().float()):
        with pytest.raises(TypeError):
            g.gemm_nt_w4(bad, q)
    for bad in (a[0], a[:, :63], a.t(), a.cpu(), torch.ones(64, 4, **f16).t()):
        with pytest.raises(ValueError):
            g.gemm_nt_w4(bad, q)
    with pytest.raises(TypeError):
        g.gemm_nt_w4(a, torch.ones(32, 64, **f16))
    for out in (torch.empty(4, 33, **f16), torch.empty(4, 32, device="cuda"),
                torch.empty(32, 4, **f16).t(), torch.empty(4, 32).half()):
        with pytest.raises(ValueError):
            g.gemm_nt_w4(a, q, out=out)
    with pytest.raises(g.GemmError):            # C on top of A
        g.gemm_nt_w4(a, q, out=a.view(-1)[:128].view(4, 32))
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    big, qb = torch.ones(64, 4096, **f16), g.quantize_w4(torch.ones(32, 4096, **f16), 32)
    need = g.gemm_f16_nt_w4_plan(64, 32, 4096, 32, cus).workspace_bytes
    assert need > 0
    for ws in (torch.empty(need - 1, dtype=torch.uint8, device="cuda"),
               torch.empty(need + 64, dtype=torch.uint8, device="cuda")[64:]):
        with pytest.raises(g.GemmError):        # too small, and not 256-byte aligned
            g.gemm_nt_w4(big, qb, workspace=ws)
    with pytest.raises(ValueError):             # not on the GPU
        g.gemm_nt_w4(big, qb, workspace=torch.empty(need, dtype=torch.uint8))
    with pytest.raises(ValueError):
        g.gemm_tn_q8(torch.ones(31, 4, **f16), c)
    with pytest.raises(ValueError):
        g.gemm_tn_q8(torch.ones(4, 32, **f16).t(), c)
    with pytest.raises(ValueError):
        g.quantize_w4(torch.ones(64, 32, **f16).t())
    with pytest.raises(ValueError):
        g.quantize_w4(torch.ones(64, 32, **f16), 48)
    with pytest.raises(ValueError):
        g.pack_w4(torch.ones(4, 64, dtype=torch.int8, device="cuda"), torch.ones(4, 3, **f16), 32)
    with pytest.raises(ValueError):
        g.quantize_q8(torch.ones(64, 32, **f16).t())


# ---- together, as they are used ----------------------------------------------------
def checkpointed_linear(g):
    """x @ w.T whose input is kept in 8 bits for the weight's gradient."""
    import torch

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w):
            kept = g.quantize_q8(x)
            ctx.n = kept.n
            ctx.save_for_backward(kept.codes, kept.scales, w)
            return g.gemm_nt(x, w)

        @staticmethod
        def backward(ctx, dy):
            codes, scales, w = ctx.saved_tensors
            dy = dy.contiguous()
            return g.gemm_nn(dy, w), g.gemm_tn_q8(dy, g.Q8Matrix(codes, scales, ctx.n))

    return Linear.apply


def test_training_step_then_serving(g):
    """Two linear layers with a ReLU between them, trained for a step with
    8-bit checkpoints, then quantised to 4 bits and run for single tokens and a
    prompt.  Gradients against the formula in 64 bits on the stored inputs, and
    against the gradients of exact inputs within what 8 bits allow."""
    import torch

    rng = np.random.default_rng(31)
    t, d, f = 130, 96, 200
    x = rng.standard_normal((t, d)).astype(np.float16)
    w1 = (rng.standard_normal((f, d)) / np.sqrt(d)).astype(np.float16)
    w2 = (rng.standard_normal((d, f)) / np.sqrt(f)).astype(np.float16)
    dy = (rng.standard_normal((t, d)) / 8).astype(np.float16)
    linear = checkpointed_linear(g)
    w1t, w2t, xt = (dev(v).requires_grad_() for v in (w1, w2, x))
    h = torch.relu(linear(xt, w1t))
    linear(h, w2t).backward(dev(dy))
    hh = host(h.detach())
    f64 = lambda v: v.astype(np.float64)  # noqa: E731

    def rounded(v):
        codes, scales = ref.encode(v, 32, **ref.Q8)
        return ref.values(codes, scales, 32, v.shape[1])

    check_product(host(w2t.grad), f64(dy).T, rounded(hh), t, False)
    # each stored value is off by at most half a step, 2^-8 (1 + 1/8) of its
    # group's largest magnitude: the step is s, and 127 s passes the largest by
    # less than one part in eight
    groups = np.repeat(np.abs(f64(np.pad(hh, ((0, 0), (0, -f % 32))))).reshape(t, -1, 32).max(-1), 32,
                       axis=1)[:, :f]
    off = np.abs(f64(dy)).T @ (groups * 1.125 / 127 / 2 + 2.0 ** -25)
    exact = f64(dy).T @ f64(hh)
    assert (np.abs(host(w2t.grad) - exact)
            <= off + ref.product_bound(np.abs(f64(dy)).T @ np.abs(f64(hh)), exact, t) + off * 2.0 ** -11).all()
    dh = host(g.gemm_nn(dev(dy), w2t.detach()))
    check_product(dh, f64(dy), f64(w2), d, False)
    dz = np.where(hh > 0, dh, 0).astype(np.float16)
    check_product(host(w1t.grad), f64(dz).T, rounded(x), t, False)
    check_product(host(xt.grad), f64(dz), f64(w1), f, False)

    q1 = g.quantize_w4(w1t.detach(), 32)
    v1 = f64(host(g.dequantize_w4(q1)))
    for rows in (1, t):
        check_product(host(g.gemm_nt_w4(xt.detach()[:rows], q1)), f64(x[:rows]), v1.T, d, False)


def test_gradient_against_differences(g):
    """dW from an 8-bit checkpoint is the derivative of sum(dy * (X W^T)) at
    the stored X: central differences along random directions, in 64 bits."""
    rng = np.random.default_rng(41)
    t, n, m = 90, 70, 33
    x = rng.standard_normal((t, n)).astype(np.float16)
    dy = rng.integers(-4, 5, (t, m)).astype(np.float16)
    kept = g.quantize_q8(dev(x))
    grad = host(g.gemm_tn_q8(dev(dy), kept)).astype(np.float64)
    xv = host(g.dequantize_q8(kept)).astype(np.float64)
    w = rng.standard_normal((m, n))
    loss = lambda w: (dy.astype(np.float64) * (xv @ w.T)).sum()  # noqa: E731
    bound = ref.product_bound(np.abs(dy.astype(np.float64)).T @ np.abs(xv), grad, t)
    for _ in range(5):
        d = rng.standard_normal((m, n))
        # the loss is linear in w: differences are exact but for float64's rounding
        diff = (loss(w + d) - loss(w - d)) / 2
        assert abs(diff - (grad * d).sum()) <= (bound * np.abs(d)).sum() + 1e-9 * abs(loss(w))


# ---- beyond 32 bits -------------------------------------------------------------
def test_w4_beyond_32_bits(g):
    """Words past 2^32 bytes, the fp16 matrix past 2^34: the last rows of every
    kernel's result, which are those of the last rows alone, and the first."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(31)
    n, k, group = 2 ** 20 + 37, 8320, 128
    nb, kt = -(-n // 16), -(-k // 128)
    words = torch.randint(-2 ** 31, 2 ** 31, (nb, kt, 64, 4), dtype=torch.int32, device="cuda",
                          generator=gen)
    assert words.numel() * 4 > 2 ** 32
    scales = torch.randint(1, 256, (nb, kt, 16), device="cuda", generator=gen).half() / 2 ** 14
    w = g.W4Matrix(words, scales, n, k, group)
    # the first and the last rows, as matrices of their own
    head, rest = 32, n - 16 * (nb - 2)
    lo = g.W4Matrix(words[:2], scales[:2], head, k, group)
    hi = g.W4Matrix(words[-2:], scales[-2:], rest, k, group)
    lo64, hi64 = (host(g.dequantize_w4(x)).astype(np.float64) for x in (lo, hi))
    for m in (1, 3, 16, 48, 1500):
        a = torch.randn((m, k), device="cuda", generator=gen).half()
        c = g.gemm_nt_w4(a, w)
        a64 = host(a).astype(np.float64)
        check_product(host(c[:, :head]), a64, lo64.T, k, False)
        check_product(host(c[:, -rest:]), a64, hi64.T, k, False)
        del c
    full = g.dequantize_w4(w)
    assert (host(full[:head]).astype(np.float64) == lo64).all()
    assert (host(full[-rest:]).astype(np.float64) == hi64).all()
    again = g.quantize_w4(full, group)
    tail = g.quantize_w4(full[-rest:].contiguous(), group)
    assert torch.equal(again.words[-2:], tail.words)
    assert torch.equal(again.scales[-2:], tail.scales)


def test_q8_beyond_32_bits(g):
    """Codes past 2^32 bytes.  Rows of A are zeros but for the first and the last
    1000, so the product is that of those rows of X."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(32)
    r, n, rows = 2 ** 20 + 40037, 4160, 1000
    x = torch.empty((r, n), dtype=torch.float16, device="cuda")
    for i in range(0, r, 2 ** 17):
        x[i:i + 2 ** 17] = torch.randn(x[i:i + 2 ** 17].shape, device="cuda", generator=gen)
    q = g.quantize_q8(x)
    assert q.codes.numel() > 2 ** 32
    ends = []
    for part in (slice(0, rows), slice(r - rows, r)):
        alone = g.quantize_q8(x[part])
        assert torch.equal(q.codes[part], alone.codes) and torch.equal(q.scales[part], alone.scales)
        ends.append(host(g.dequantize_q8(alone)))
    back = g.dequantize_q8(q, out=x)
    assert (host(back[:rows]) == ends[0]).all() and (host(back[-rows:]) == ends[1]).all()
    del back, x
    x64 = np.concatenate(ends).astype(np.float64)
    for m in (16, 40, 512):
        a = torch.zeros((r, m), dtype=torch.float16, device="cuda")
        a[:rows] = torch.randn((rows, m), device="cuda", generator=gen)
        a[-rows:] = torch.randn((rows, m), device="cuda", generator=gen)
        a64 = np.concatenate([host(a[:rows]), host(a[-rows:])]).astype(np.float64)
        # zeros add nothing and round nothing, so the bound is that of 2000 rows
        # with a step more for each range that K may be split into, 256 at most
        c = host(g.gemm_tn_q8(a, q))
        check_product(c, a64.T, x64, 2 * rows, False)


def test_threads_on_their_own_streams(g):
    """Calls of several host threads at once, each with sizes of its own that
    change from call to call: the same bits as alone."""
    import threading

    import torch

    calls = [(call, host(call())) for call, _, _ in products(g, np.random.default_rng(41))]
    torch.cuda.synchronize()
    wrong = []

    def run(first):
        try:
            s = torch.cuda.Stream()
            for i in range(20):
                call, want = calls[(first + i) % len(calls)]
                out = call(stream=s)
                s.synchronize()
                if not (host(out) == want).all():
                    wrong.append((first, i))
        except BaseException as e:
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


# ---- nothing around C and the workspace is written, by any kernel ----------------
def guarded(shape):
    """(tensor of `shape` at a 2-byte offset in a buffer of sentinels, check())."""
    import torch

    count = shape[0] * shape[1]
    buf = torch.full((count + 4096,), 7.0, dtype=torch.float16, device="cuda")
    out = buf[2049:2049 + count].view(shape)

    def check():
        assert (buf[:2049] == 7).all() and (buf[2049 + count:] == 7).all()

    return out, check


def guarded_workspace(need):
    import torch

    buf = torch.full((need + 8192,), 0x5A, dtype=torch.uint8, device="cuda")

    def check():
        assert (buf[:4096] == 0x5A).all() and (buf[4096 + need:] == 0x5A).all()

    return buf[4096:4096 + need], check


@pytest.mark.parametrize("kernel,m,n,k", W4_KERNELS)
def test_nt_w4_every_kernel_in_bounds(g, kernel, m, n, k):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(m * n + k)
    q = g.quantize_w4(torch.randn(n, k, generator=gen, device="cuda").half(), 64)
    a = torch.randn(m, k, generator=gen, device="cuda").half()
    out, out_kept = guarded((m, n))
    ws, ws_kept = guarded_workspace(g.gemm_f16_nt_w4_plan(m, n, k, 64, 256).workspace_bytes)
    g.gemm_nt_w4(a, q, out=out, workspace=ws)
    out_kept(), ws_kept()
    assert torch.equal(out, g.gemm_nt_w4(a, q))


@pytest.mark.parametrize("kernel,splits,m,n,k", Q8_KERNELS)
def test_tn_q8_every_kernel_in_bounds(g, kernel, splits, m, n, k):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(m * n + k)
    x = g.quantize_q8(torch.randn(k, n, generator=gen, device="cuda").half())
    a = torch.randn(k, m, generator=gen, device="cuda").half()
    out, out_kept = guarded((m, n))
    ws, ws_kept = guarded_workspace(g.gemm_f16_tn_q8_plan(m, n, k, 256).workspace_bytes)
    g.gemm_tn_q8(a, x, out=out, workspace=ws)
    out_kept(), ws_kept()
    assert torch.equal(out, g.gemm_tn_q8(a, x))
