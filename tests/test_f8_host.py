"""The 8-bit floating point operands and the experts' layers without a GPU: the C
ABI's checks, sizes and plans, and what the binding refuses."""
import os
import re

import numpy as np
import pytest

import f8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 2


def at(i):
    return (i + 1) << 40


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_amd as lib

    lib.load()
    return lib


def refused(g, status, fn, *args):
    with pytest.raises(g.GemmError) as e:
        fn(*args)
    assert e.value.status == status


@pytest.mark.parametrize("header", ["gemm_f16_f8.h", "gemm_f16_experts.h"])
def test_header_functions_are_bound(g, header):
    text = open(os.path.join(ROOT, "include", header)).read()
    names = set(re.findall(r"^int (gemm_f16_\w+)\(", text, re.M))
    assert names
    for name in names:
        assert getattr(g.load(), name).argtypes is not None
        assert callable(getattr(g, name))


def test_reference_rounding():
    """The oracle's rounding: every code is its own, halfway goes to the even code."""
    v = ref.code_values()[:127]
    np.testing.assert_array_equal(ref.round_codes(v), v)
    mid = (v[:-1] + v[1:]) / 2
    np.testing.assert_array_equal(ref.round_codes(mid), np.where(np.arange(126) % 2 == 0, v[:-1], v[1:]))
    big = np.array([1e-30, 448 * 2.0 ** -32, 448, 448.5, 65504.0])
    np.testing.assert_array_equal(ref.scale_of(big), [-32, -32, 0, 1, 8])


def test_sizes(g):
    assert g.gemm_f16_f8_sizes(1, 3, 129, 1) == (3 * 256, 3 * 4)
    assert g.gemm_f16_f8_sizes(2, 130, 513, 128) == (2 * 130 * 640, 2 * 2 * 2 * 4)
    assert g.gemm_f16_f8_sizes(0, 130, 513, 128) == (0, 0)
    assert g.gemm_f16_f8_sizes(1, 5, 0, 1) == (0, 0)
    for args in ((-1, 1, 1, 1), (1, -1, 1, 1), (1, 1, -1, 1), (1, 1, 1, 64), (1, 1, 1, 0)):
        refused(g, INVALID, g.gemm_f16_f8_sizes, *args)
    for args in ((1, 1, 2 ** 23 + 1, 1), (1, 2 ** 31 - 127, 1, 1), (2, 2 ** 30, 1, 1), (2 ** 31, 1, 1, 1),
                 (1, 2 ** 20, 2 ** 21, 1)):
        refused(g, UNSUPPORTED, g.gemm_f16_f8_sizes, *args)


def test_quantize_refusals(g):
    q = g.gemm_f16_f8_quantize
    refused(g, INVALID, q, 1, 4, 128, 64, False, at(0), at(1), at(2))
    refused(g, INVALID, q, 1, 4, 128, 1, False, 0, at(1), at(2))
    refused(g, INVALID, q, 1, 4, 128, 1, False, at(0), 0, at(2))
    refused(g, INVALID, q, 1, 4, 128, 1, False, at(0), at(0) + 16, at(2))      # codes in X
    refused(g, UNSUPPORTED, q, 1, 4, 128, 1, False, at(0) + 1, at(1), at(2))
    refused(g, UNSUPPORTED, q, 1, 4, 128, 1, False, at(0), at(1) + 8, at(2))
    refused(g, UNSUPPORTED, q, 1, 4, 128, 1, False, at(0), at(1), at(2) + 2)
    refused(g, INVALID, q, 1, 4, 128, 1, 2, at(0), at(1), at(2))
    q(1, 0, 128, 1, False, 0, 0, 0)                                             # nothing to do
    d = g.gemm_f16_f8_dequantize
    refused(g, INVALID, d, 1, 4, 128, 1, at(0), at(1), at(0))
    refused(g, UNSUPPORTED, d, 1, 4, 128, 1, at(0), at(1), at(2) + 1)
    d(3, 0, 128, 128, 0, 0, 0)


def test_product_refusals(g):
    f, x = g.gemm_f16_nt_f8, g.gemm_f16_nt_f8_x
    good = [4, 5, 128, at(0), at(1), 128, at(2), at(3), at(4)]
    for i, v in ((0, -1), (1, -1), (2, -1), (5, 64), (3, 0), (4, 0), (6, 0), (7, 0), (8, 0), (8, at(0)), (8, at(3))):
        refused(g, INVALID, f, *good[:i], v, *good[i + 1:])
    for i, v in ((3, at(0) + 8), (4, at(1) + 1), (6, at(2) + 8), (7, at(3) + 2), (8, at(4) + 1), (2, 2 ** 23 + 1)):
        refused(g, UNSUPPORTED, f, *good[:i], v, *good[i + 1:])
    refused(g, INVALID, f, *good, at(0), 1 << 20)                                # workspace on A
    refused(g, UNSUPPORTED, f, *good, at(5) + 16, 1 << 20)
    refused(g, INVALID, f, *good, at(5), -1)
    goodx = [4, 5, 128, at(0), 128, at(2), at(3), at(4)]
    for i, v in ((3, 0), (5, 0), (7, at(0)), (4, 2)):
        refused(g, INVALID, x, *goodx[:i], v, *goodx[i + 1:])
    refused(g, UNSUPPORTED, x, *goodx[:3], at(0) + 1, *goodx[4:])
    f(0, 5, 128, 0, 0, 128, at(2), at(3), 0)                                     # nothing to compute
    f(4, 0, 128, at(0), at(1), 128, 0, 0, 0)


@pytest.mark.parametrize("f16", [False, True])
def test_plans(g, f16):
    """A plan's grid stays within a launch, its workspace is what its parts take
    and holds A's quantised form where A is fp16."""
    for m in (1, 2, 15, 16, 17, 48, 64, 100, 333, 1000, 4096, 20000):
        for n in (1, 16, 100, 4096, 7001, 65536):
            for k in (1, 128, 1000, 4096, 14336, 2 ** 20):
                for block in (1, 128):
                    p = g.gemm_f16_nt_f8_plan(m, n, k, block, f16, 256)
                    assert p.kernel in (g.LOWBIT_STREAM, g.LOWBIT_TILE)
                    assert p.grid >= 1 and p.grid * 64 * p.waves < 2 ** 32
                    assert p.splits >= 1 and p.workspace_bytes >= 0 and p.workspace_bytes % 256 == 0
                    if p.splits > 1:
                        assert p.workspace_bytes >= 4 * p.splits * m * n
    assert g.gemm_f16_nt_f8_plan(0, 5, 128, 128, f16, 256).workspace_bytes == 0
    refused(g, INVALID, g.gemm_f16_nt_f8_plan, 4, 5, 128, 128, f16, 0)
    refused(g, INVALID, g.gemm_f16_nt_f8_plan, 4, 5, 128, 3, f16, 256)
    refused(g, UNSUPPORTED, g.gemm_f16_nt_f8_plan, 2 ** 30, 2 ** 30, 128, 128, f16, 256)


@pytest.mark.parametrize("f16", [False, True])
@pytest.mark.parametrize("gather", [False, True])
def test_experts_plans(g, f16, gather):
    for t in (1, 2, 33, 333, 4096, 8192):
        for e, top in ((1, 1), (8, 2), (64, 8), (256, 8), (1024, 32)):
            for n, k in ((16, 128), (2048, 4096), (7001, 1000)):
                p = g.gemm_f16_nt_f8_experts_plan(t * top, e, n, k, top if gather else 0, f16, 256)
                assert p.grid >= 1 and p.grid * 64 * p.waves < 2 ** 32 and p.workspace_bytes >= 0
                # a workgroup a tile, or as many as there are compute units for all
                assert p.grid * p.block_m * p.block_n >= t * top * n or p.kernel == g.LOWBIT_STREAM or \
                    p.grid in (256, 512)
    refused(g, UNSUPPORTED, g.gemm_f16_nt_f8_experts_plan, 8, 1025, 16, 128, 0, f16, 256)
    refused(g, INVALID, g.gemm_f16_nt_f8_experts_plan, 8, 0, 16, 128, 0, f16, 256)
    refused(g, INVALID, g.gemm_f16_nt_f8_experts_plan, 9, 8, 16, 128, 2, f16, 256)
    refused(g, UNSUPPORTED, g.gemm_f16_nt_f8_experts_plan, 2 ** 22, 8, 16, 8192, 1, f16, 256)
    assert g.gemm_f16_f8_experts_columns(1000, 8) == 128 * (7 + 8)
    assert g.gemm_f16_f8_experts_columns(3, 8) == 128 * 3
    assert g.gemm_f16_f8_experts_columns(0, 8) == 0


def test_experts_refusals(g):
    f = g.gemm_f16_nt_f8_experts
    good = [8, 4, 16, 128, 2, at(0), at(1), at(2), at(3), at(4), at(5), at(6)]
    for i, v in ((0, -1), (0, 7), (1, 0), (2, -1), (3, -1), (4, -1), (5, 0), (7, 0), (9, 0), (10, 0), (11, 0), (11, at(4)), (11, at(2))):
        refused(g, INVALID, f, *good[:i], v, *good[i + 1:])
    for i, v in ((1, 1025), (5, at(0) + 4), (9, at(4) + 2), (10, at(5) + 1), (11, at(6) + 1)):
        refused(g, UNSUPPORTED, f, *good[:i], v, *good[i + 1:])
    q = g.gemm_f16_f8_quantize_experts
    good = [8, 4, 16, 2, at(0), at(1), at(2), at(3), at(4)]
    for i, v in ((0, 7), (1, 0), (2, -1), (3, -2), (4, 0), (5, 0), (6, 0), (7, 0), (8, at(0))):
        refused(g, INVALID, q, *good[:i], v, *good[i + 1:])
    d = g.gemm_f16_nt_f8_experts_grad
    good = [8, 4, 16, 20, at(0), at(1), at(2), at(3), at(4), at(5)]
    for i, v in ((0, -1), (1, 0), (2, -1), (3, -1), (4, 0), (7, 0), (8, 0), (9, 0), (9, at(2))):
        refused(g, INVALID, d, *good[:i], v, *good[i + 1:])
    refused(g, UNSUPPORTED, d, 8, 1024, 2 ** 20, 2 ** 20, *good[4:])


def test_route_refusals(g):
    good = [4, 8, 2, 0, 1, 1, 0, 1, 1.0, at(0), 1, at(1), at(2), at(3), at(4), at(5), at(6)]
    for i, v in ((0, -1), (1, 0), (1, 1025), (2, 0), (2, 9), (2, 33), (3, 2), (3, -1), (4, 0), (4, 3), (5, 0), (5, 2),
                 (9, 0), (12, 0), (13, 0), (14, 0), (15, 0), (16, 0), (12, at(0)), (14, at(5)), (0, 2 ** 31)):
        refused(g, INVALID, g.gemm_f16_route, *good[:i], v, *good[i + 1:])
    for i, v in ((9, at(0) + 2), (11, at(1) + 1), (12, at(2) + 2)):
        refused(g, UNSUPPORTED, g.gemm_f16_route, *good[:i], v, *good[i + 1:])
    good = [4, 8, 2, 0, 1, 1.0, at(0), 1, at(1), at(2), at(3), at(4)]
    for i, v in ((0, -1), (2, 9), (3, 5), (6, 0), (8, 0), (9, 0), (10, 0), (11, 0), (11, at(0))):
        refused(g, INVALID, g.gemm_f16_route_backward, *good[:i], v, *good[i + 1:])
    g.gemm_f16_route_backward(0, 8, 2, 0, True, 1.0, 0, True, 0, 0, 0, 0)
    assert g.gemm_f16_route_workspace(1, 8, 2) == 0
    refused(g, INVALID, g.gemm_f16_route_workspace, 1, 8, 9)


def test_combine_refusals(g):
    good = [4, 2, 16, at(0), at(1), at(2), at(3)]
    for i, v in ((0, -1), (1, 0), (1, 33), (2, -1), (3, 0), (5, 0), (6, 0), (6, at(0)), (6, at(1))):
        refused(g, INVALID, g.gemm_f16_combine, *good[:i], v, *good[i + 1:])
    refused(g, UNSUPPORTED, g.gemm_f16_combine, *good[:3], at(0) + 1, *good[4:])
    good = [4, 2, 16, at(0), at(1), at(2), at(3), at(4), at(5), at(6)]
    for i, v in ((0, -1), (1, 0), (3, 0), (4, 0), (6, 0), (7, 0), (8, 0), (8, at(1)), (9, at(2))):
        refused(g, INVALID, g.gemm_f16_combine_backward, *good[:i], v, *good[i + 1:])
    g.gemm_f16_combine(0, 2, 16, 0, 0, 0, 0)


def test_binding_refuses_host_tensors(g):
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 128, dtype=torch.float16)
    with pytest.raises(ValueError):
        g.quantize_f8(x)
    with pytest.raises(TypeError):
        g.quantize_f8(x.float())
    with pytest.raises(ValueError):
        g.F8Matrix(torch.zeros(4, 128, dtype=torch.float8_e4m3fn), torch.zeros(1, 4, 4, dtype=torch.uint8), 128, 1)
    with pytest.raises(ValueError):
        g.route(torch.zeros(4, 8), 2)
    with pytest.raises(TypeError):
        g.gemm_nt_f8(x, x)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.Routing(i, torch.zeros(4, 2), torch.zeros(8, dtype=torch.int32), i, torch.zeros(9, dtype=torch.int32))


def test_reference_gradient_by_differences():
    """The oracle's own gradient of the weights, against differences."""
    rng = np.random.default_rng(0)
    x, dw = rng.standard_normal((3, 10)), rng.standard_normal((3, 4))
    experts = np.stack([rng.permutation(10)[:4] for _ in range(3)])
    for kind in ("softmax", "sigmoid"):
        for norm in (True, False):
            got = ref.route_gradient(x, experts, dw, kind, norm, 1.3)
            for i in range(3):
                for j in range(10):
                    h = np.zeros_like(x)
                    h[i, j] = 1e-6
                    d = ((ref.weights_of(x + h, experts, kind, norm, 1.3) -
                          ref.weights_of(x - h, experts, kind, norm, 1.3)) * dw).sum() / 2e-6
                    assert abs(d - got[i, j]) < 1e-8
