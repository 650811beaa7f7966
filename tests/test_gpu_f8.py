"""Operands in 8-bit floating point on the GPU, against plain 64-bit references
(f8_ref.py)."""
import numpy as np
import pytest
import torch

import f8_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_amd as lib

    lib.load()
    return lib


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t if dtype is None else t.to(dtype)).cuda()


def host(x):
    return x.cpu().numpy()


def code_values(codes):
    return ref.code_values()[host(codes.view(torch.uint8))]


def check_storage(q, want_q, want_e, k):
    """An F8Matrix's codes and scales against the reference's, NaN for NaN."""
    kp = -(-k // 128) * 128
    got = code_values(q.codes)
    assert got.shape == (want_q.shape[0], kp)
    np.testing.assert_array_equal(got, want_q)
    scales = ref.stored_scales(want_e)
    have = host(q.scales)
    assert have.shape == scales.shape
    there = ref.stored_scales(np.ones_like(want_e) - 127) == 1
    np.testing.assert_array_equal(have[there], scales[there])


def halves(rng, *shape):
    """Magnitudes over many powers of two, zeros, and rows that are all zero."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-20, 12, shape)
    x[rng.random(shape) < 0.1] = 0
    x[rng.random(shape[0]) < 0.1] = 0
    return np.clip(x, -65504, 65504).astype(np.float16)


SHAPES = [(1, 1), (1, 128), (3, 127), (4, 129), (5, 512), (7, 513), (16, 1000), (127, 130),
          (128, 128), (129, 257), (130, 640), (300, 96), (1, 4096), (1000, 2)]


@pytest.mark.parametrize("r,k", SHAPES)
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize(g, r, k, block, transposed):
    x = halves(np.random.default_rng(r * 10007 + k), r, k)
    q = g.quantize_f8(dev(x), block, transposed)
    y = x.T if transposed else x
    want, e = ref.encode(y, block)
    check_storage(q, want, e, y.shape[1])
    assert q.shape == y.shape and q.block == block
    back = host(g.dequantize_f8(q))
    with np.errstate(over="ignore"):
        np.testing.assert_array_equal(back, ref.values(want, e, block, y.shape[1]).astype(np.float16))


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("transposed", [False, True])
def test_quantize_stack(g, block, transposed):
    x = halves(np.random.default_rng(5), 3, 130, 200)
    q = g.quantize_f8(dev(x), block, transposed)
    for i in range(3):
        one = g.quantize_f8(dev(x[i]), block, transposed)
        assert torch.equal(q.codes[i].view(torch.uint8), one.codes.view(torch.uint8))
        want, e = ref.encode(x[i].T if transposed else x[i], block)
        check_storage(g.F8Matrix(q.codes[i], q.scales[i], q.k, block), want, e, q.k)
    np.testing.assert_array_equal(host(g.dequantize_f8(q)[1]),
                                  host(g.dequantize_f8(g.F8Matrix(q.codes[1], q.scales[1], q.k, block))))


@pytest.mark.parametrize("block,transposed", [(1, False), (1, True), (128, False), (128, True)])
def test_quantize_every_half(g, block, transposed):
    """Every fp16 number, in the order of their bits (groups of like magnitude)
    and mixed (groups of unlike ones); infinities and NaN among them."""
    bits = np.arange(65536, dtype=np.uint16)
    mixed = np.random.default_rng(1).permutation(bits)
    for b in (bits, mixed):
        x = b.view(np.float16).reshape(256, 256)
        q = g.quantize_f8(dev(x), block, transposed)
        y = x.T if transposed else x
        want, e = ref.encode(y, block)
        check_storage(q, want, e, 256)


def test_quantize_not_finite(g):
    """An infinity or NaN becomes NaN alone; its group's scale is the others'."""
    x = np.zeros((4, 256), dtype=np.float16)
    x[0, 3], x[0, 5] = np.inf, 100.0
    x[1, 130], x[1, 131] = np.nan, -0.25
    x[2, 0], x[3, 255] = -np.inf, 65504
    for block, transposed in ((1, False), (1, True), (128, False), (128, True)):
        q = g.quantize_f8(dev(x), block, transposed)
        y = x.T if transposed else x
        want, e = ref.encode(y, block)
        check_storage(q, want, e, y.shape[1])


def test_unaligned_and_guards(g):
    """X at 2-byte alignment; what lies around codes, scales and X stays."""
    rng = np.random.default_rng(2)
    for r, k in ((5, 300), (130, 129)):
        x = halves(rng, r, k)
        buf = torch.zeros(r * k + 16, dtype=torch.float16, device="cuda")
        view = buf[3:3 + r * k].view(r, k)
        view.copy_(dev(x))
        for block, transposed in ((1, False), (1, True), (128, False), (128, True)):
            rr, kk = (k, r) if transposed else (r, k)
            nc, ns = g.gemm_f16_f8_sizes(1, rr, kk, block)
            codes = torch.full((nc + 64,), 7, dtype=torch.uint8, device="cuda")
            scales = torch.full((ns + 64,), 7, dtype=torch.uint8, device="cuda")
            s = torch.cuda.current_stream().cuda_stream
            g.gemm_f16_f8_quantize(1, rr, kk, block, transposed, view.data_ptr(),
                                   codes[32:].data_ptr(), scales[32:].data_ptr(), s)
            same = g.quantize_f8(view.clone(), block, transposed)
            assert torch.equal(codes[32:32 + nc], same.codes.view(torch.uint8).flatten())
            for guard in (codes[:32], codes[32 + nc:], scales[:32], scales[32 + ns:]):
                assert (guard == 7).all()
            out = torch.full((r * k + 16,), 3.0, dtype=torch.float16, device="cuda")
            g.gemm_f16_f8_dequantize(1, rr, kk, block, codes[32:].data_ptr(),
                                     scales[32:].data_ptr(), out[5:].data_ptr(), s)
            assert (out[:5] == 3).all() and (out[5 + r * k:] == 3).all()
            assert torch.equal(out[5:5 + r * k].view(rr, kk), g.dequantize_f8(same))


def test_dequantize_scales(g):
    """Every scale's byte: 0 the smallest, 255 NaN; values round to fp16."""
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))[:, :128]
    scales = np.zeros((1, 256, 4), dtype=np.uint8)
    scales[0, :, 0] = np.arange(256)
    q = g.F8Matrix(dev(codes).view(torch.float8_e4m3fn), dev(scales), 128, 1)
    s = np.ldexp(1.0, np.arange(256) - 127)
    s[255] = np.nan
    with np.errstate(over="ignore"):
        want = (ref.code_values()[:128][None, :] * s[:, None]).astype(np.float16)
    np.testing.assert_array_equal(host(g.dequantize_f8(q)), want)


# ---- products ------------------------------------------------------------------
def whole(rng, r, k, block, spread=3):
    """An F8 matrix of small whole numbers times powers of two, whose products
    and sums are exact in fp32 whatever their order: (codes, scales, values)."""
    q = rng.integers(-2, 3, (r, k)).astype(np.float64)
    e = rng.integers(-spread, spread + 1, (-(-r // block), -(-k // 128)))
    table = {float(v): c for c, v in enumerate(ref.code_values()) if not np.isnan(v) and c != 128}
    codes = np.zeros((r, -(-k // 128) * 128), dtype=np.uint8)
    codes[:, :k] = np.vectorize(table.__getitem__)(q) if k else 0
    return codes, ref.stored_scales(e), ref.values(np.pad(q, ((0, 0), (0, -k % 128))), e, block, k)


def f8(g, codes, scales, k, block):
    return g.F8Matrix(dev(codes).view(torch.float8_e4m3fn), dev(scales), k, block)


PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 300, 1000), (2, 17, 129), (3, 128, 4096), (5, 70, 300),
            (8, 1000, 640), (15, 33, 513), (16, 64, 2048), (17, 130, 384), (31, 257, 1024),
            (33, 100, 640), (48, 512, 128), (49, 96, 700), (64, 128, 1280), (65, 129, 257),
            (100, 257, 513), (128, 256, 512), (129, 130, 1500), (200, 520, 896), (255, 256, 128),
            (257, 300, 2000), (300, 260, 200), (512, 512, 1024), (513, 1025, 130), (1000, 16, 3000)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("block", [1, 128])
def test_product_exact(g, m, n, k, block):
    rng = np.random.default_rng(m * 31 + n * 7 + k)
    ac, as_, a = whole(rng, m, k, 1)
    bc, bs, b = whole(rng, n, k, block)
    c = g.gemm_nt_f8(f8(g, ac, as_, k, 1), f8(g, bc, bs, k, block))
    np.testing.assert_array_equal(host(c), (a @ b.T).astype(np.float16))


@pytest.mark.parametrize("m,n,k", [(1, 100, 300), (7, 129, 640), (16, 256, 1025), (40, 70, 128),
                                   (130, 200, 500), (300, 300, 300)])
@pytest.mark.parametrize("block", [1, 128])
def test_product_of_halves(g, m, n, k, block):
    """A in fp16, quantised in the call: what quantize_f8 gives, bit for bit, and
    the exact sum within the bound."""
    rng = np.random.default_rng(m + n + k)
    x = rng.standard_normal((m, k)).astype(np.float16)
    w = (rng.standard_normal((n, k)) / np.sqrt(k)).astype(np.float16)
    w8 = g.quantize_f8(dev(w), block)
    c = g.gemm_nt_f8(dev(x), w8)
    assert torch.equal(c, g.gemm_nt_f8(g.quantize_f8(dev(x)), w8))
    xq, wq = ref.quantized(x, 1), ref.quantized(w, block)
    exact = xq @ wq.T
    got = host(c).astype(np.float64)
    assert (np.abs(got - exact) <= ref.product_bound(np.abs(xq) @ np.abs(wq).T, exact, k)).all()
    # and on the whole much nearer: roundings to fp16 (2^-11 / sqrt(3) at most)
    # and the cut products (1.4e-5 of the result, measured; four times that)
    rms = np.sqrt(np.mean(exact ** 2))
    assert np.sqrt(np.mean((got - exact) ** 2)) <= rms * (2.0 ** -11 / np.sqrt(3) * 1.5 + 6e-5)


def test_layer_and_gradients(g):
    """A linear layer: Y, dX and dW from the forms that the header names."""
    rng = np.random.default_rng(9)
    t, n, k = 150, 200, 300
    x, w = rng.standard_normal((t, k)).astype(np.float16), rng.standard_normal((n, k)).astype(np.float16)
    dy = rng.standard_normal((t, n)).astype(np.float16)
    y = g.gemm_nt_f8(dev(x), g.quantize_f8(dev(w), 128))
    dx = g.gemm_nt_f8(dev(dy), g.quantize_f8(dev(w), 128, transposed=True))
    dw = g.gemm_nt_f8(g.quantize_f8(dev(dy), transposed=True), g.quantize_f8(dev(x), transposed=True))
    wq = ref.quantized(w, 128)
    for got, a, b in ((y, ref.quantized(x, 1), wq), (dx, ref.quantized(dy, 1), wq.T),
                      (dw, ref.quantized(dy.T.copy(), 1), ref.quantized(x.T.copy(), 1))):
        exact = a @ b.T
        bound = ref.product_bound(np.abs(a) @ np.abs(b).T, exact, a.shape[1])
        assert (np.abs(host(got).astype(np.float64) - exact) <= bound).all()


def test_gradient_by_differences(g):
    """dX against differences of the product itself along directions of powers
    of two, which quantising keeps: the product is linear in them."""
    rng = np.random.default_rng(10)
    m, n, k = 20, 130, 256
    bc, bs, b = whole(rng, n, k, 128, spread=0)
    w = f8(g, bc, bs, k, 128)
    wt = g.quantize_f8(g.dequantize_f8(w), 128, transposed=True)
    x = rng.integers(-2, 3, (m, k)).astype(np.float16)
    x[:, 0] = x[:, 128] = 2
    dy = rng.integers(-2, 3, (m, n)).astype(np.float16)
    dx = host(g.gemm_nt_f8(dev(dy), wt)).astype(np.float64)

    def loss(v):
        return (host(g.gemm_nt_f8(dev(v.astype(np.float16)), w)).astype(np.float64) * dy).sum()

    for i, j in ((0, 1), (3, 77), (19, 255), (7, 129)):
        up, down = x.copy(), x.copy()
        up[i, j], down[i, j] = 1, -1
        assert (loss(up) - loss(down)) / 2 == dx[i, j]


@pytest.mark.parametrize("m,n,k", [(1, 300, 500), (20, 200, 300), (150, 260, 700)])
def test_not_finite(g, m, n, k):
    """A NaN or an infinity reaches the rows and columns that it enters, no others."""
    rng = np.random.default_rng(m)
    x, w = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((n, k)).astype(np.float16)
    x[m // 2, 7] = np.inf
    w[n // 3, k - 1] = np.nan
    c = host(g.gemm_nt_f8(dev(x), g.quantize_f8(dev(w), 128)))
    bad = np.isnan(c)
    assert bad[m // 2].all() and bad[:, n // 3].all()
    bad[m // 2], bad[:, n // 3] = False, False
    assert not bad.any() and np.isfinite(np.delete(np.delete(c, m // 2, 0), n // 3, 1)).all()


def test_scale_of_nan(g):
    """A scale's byte of 255 makes the rows that it scales NaN."""
    rng = np.random.default_rng(3)
    for m in (3, 100):
        ac, as_, a = whole(rng, m, 256, 1)
        bc, bs, b = whole(rng, 140, 256, 128)
        ac[:, 128:] |= 0x08
        as_[0, 1, 1] = 255
        c = host(g.gemm_nt_f8(f8(g, ac, as_, 256, 1), f8(g, bc, bs, 256, 128)))
        assert np.isnan(c[1]).all() and not np.isnan(np.delete(c, 1, 0)).any()


def test_overflow_and_underflow(g):
    """Sums past 65504 become infinities; far scales neither wrap nor vanish early."""
    a = np.full((2, 128), 0x7e, dtype=np.uint8)       # 448
    b = np.full((3, 128), 0x7e, dtype=np.uint8)
    for ea, eb in ((127, 127), (127 + 60, 127 - 60), (127 - 100, 127 + 85), (20, 127), (1, 250)):
        sa = np.full((1, 2, 4), ea, dtype=np.uint8)
        sb = np.full((1, 1, 4), eb, dtype=np.uint8)
        c = host(g.gemm_nt_f8(f8(g, a, sa, 128, 1), f8(g, b, sb, 128, 128)))
        with np.errstate(over="ignore"):
            assert (c == np.float16(448.0 * 448 * 128 * 2.0 ** (ea + eb - 254))).all()


@pytest.mark.parametrize("m,n", [(0, 5), (5, 0), (0, 0), (4, 6), (1, 100)])
def test_empty(g, m, n):
    for k in (0, 128):
        a = torch.empty(m, k, dtype=torch.float16, device="cuda").fill_(1)
        w = g.quantize_f8(torch.ones(n, k, dtype=torch.float16, device="cuda"), 128)
        out = torch.full((m, n), 9.0, dtype=torch.float16, device="cuda")
        for first in (a, g.quantize_f8(a)):
            assert g.gemm_nt_f8(first, w, out=out) is out
            assert out.shape == (m, n) and (out == k).all()
        assert g.dequantize_f8(w).shape == (n, k)


@pytest.mark.parametrize("m,n,k", [(1, 300, 2000), (20, 131, 300), (200, 259, 1000)])
def test_guards_and_workspace(g, m, n, k):
    """What lies around C (at 2-byte alignment) and the workspace stays; the
    workspace's contents do not matter; too small a one is refused."""
    rng = np.random.default_rng(4)
    x = dev(rng.standard_normal((m, k)).astype(np.float16))
    w = g.quantize_f8(dev(rng.standard_normal((n, k)).astype(np.float16)), 128)
    want = g.gemm_nt_f8(x, w)
    cus = g.gemm_f16_device_cus()
    for f16 in (True, False):
        need = g.gemm_f16_nt_f8_plan(m, n, k, 128, f16, cus).workspace_bytes
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device="cuda")
        out = torch.full((m * n + 32,), 3.0, dtype=torch.float16, device="cuda")
        view = out[7:7 + m * n].view(m, n)
        first = x if f16 else g.quantize_f8(x)
        g.gemm_nt_f8(first, w, out=view, workspace=ws[256:256 + need])
        assert torch.equal(view, want)
        assert (out[:7] == 3).all() and (out[7 + m * n:] == 3).all()
        assert (ws[:256] == 255).all() and (ws[256 + need:] == 255).all()
        if need:
            with pytest.raises(g.GemmError):
                g.gemm_nt_f8(first, w, out=view, workspace=ws[256:256 + need - 1])
            with pytest.raises(g.GemmError):
                g.gemm_nt_f8(first, w, out=view, workspace=ws[255:256 + need])


def test_other_stream(g):
    """Calls on a stream other than the current one, operands dropped at once."""
    rng = np.random.default_rng(6)
    x = dev(rng.standard_normal((70, 500)).astype(np.float16))
    w = dev(rng.standard_normal((130, 500)).astype(np.float16))
    want = g.gemm_nt_f8(x, g.quantize_f8(w, 128))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = g.gemm_nt_f8(x.clone(), g.quantize_f8(w.clone(), 128, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_captured(g, m):
    """A captured layer and its gradients, replayed on new inputs."""
    rng = np.random.default_rng(7)
    n, k = 256, 640
    x = dev(rng.standard_normal((m, k)).astype(np.float16))
    w = dev(rng.standard_normal((n, k)).astype(np.float16))

    def step():
        y = g.gemm_nt_f8(x, g.quantize_f8(w, 128))
        dx = g.gemm_nt_f8(y, g.quantize_f8(w, 128, transposed=True))
        dw = g.gemm_nt_f8(g.quantize_f8(y, transposed=True), g.quantize_f8(x, transposed=True))
        return y, dx, dw

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        x.copy_(dev(rng.standard_normal((m, k)).astype(np.float16)))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_refusals(g):
    x = torch.zeros(4, 256, dtype=torch.float16, device="cuda")
    w = g.quantize_f8(x, 128)
    with pytest.raises(TypeError):
        g.quantize_f8(x.float())
    with pytest.raises(ValueError):
        g.quantize_f8(x, 64)
    with pytest.raises(ValueError):
        g.quantize_f8(x.t())
    with pytest.raises(ValueError):
        g.quantize_f8(x[0])
    with pytest.raises(TypeError):
        g.gemm_nt_f8(x, x)
    with pytest.raises(ValueError):
        g.gemm_nt_f8(w, w)                       # blocks of 128 first
    with pytest.raises(ValueError):
        g.gemm_nt_f8(x[:, :128].contiguous(), w)
    with pytest.raises(ValueError):
        g.gemm_nt_f8(x.cpu(), w)
    with pytest.raises(TypeError):
        g.gemm_nt_f8(x.bfloat16(), w)
    with pytest.raises(ValueError):
        g.gemm_nt_f8(x, w, out=torch.empty(4, 5, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        g.F8Matrix(w.codes, w.scales, 300, 128)
    with pytest.raises(ValueError):
        g.F8Matrix(w.codes, w.scales, 256, 1)
    with pytest.raises(TypeError):
        g.F8Matrix(w.codes.view(torch.uint8), w.scales, 256, 128)
    with pytest.raises(ValueError):
        g.F8Matrix(w.codes.cpu(), w.scales, 256, 128)


def test_saved(g, tmp_path):
    x = dev(halves(np.random.default_rng(8), 5, 300))
    q = g.quantize_f8(x)
    torch.save((q.codes.view(torch.uint8), q.scales, q.k, q.block), tmp_path / "q.pt")
    codes, scales, k, block = torch.load(tmp_path / "q.pt", map_location="cuda", weights_only=True)
    again = g.F8Matrix(codes.view(torch.float8_e4m3fn), scales, k, block)
    assert torch.equal(g.dequantize_f8(again), g.dequantize_f8(q))
