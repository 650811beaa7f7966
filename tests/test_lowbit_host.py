"""Host side of the low-bit operands: exports, sizes, plans, refusals (no GPU)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import lowbit_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "gemm_f16_lowbit.h")


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_amd as lib

    lib.load()
    return lib


def test_header_symbols_exported_and_bound(g):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(gemm_f16_\w+)\s*\(", text)))
    assert len(names) == 10
    lib = ctypes.CDLL(g.library_path())
    for name in names:
        assert hasattr(lib, name), f"{name} declared but not exported"
        assert callable(getattr(g, name))


@pytest.mark.parametrize("n,k,group,words,scales", [
    (16, 128, 128, 1024, 32), (17, 129, 64, 4096, 256), (1, 1, 32, 1024, 128),
    (0, 500, 32, 0, 0), (500, 0, 64, 0, 0),
])
def test_w4_sizes(g, n, k, group, words, scales):
    assert g.gemm_f16_w4_sizes(n, k, group) == (words, scales)


@pytest.mark.parametrize("n,k,group,status", [
    (-1, 1, 32, 1), (1, -1, 32, 1), (1, 1, 16, 1), (1, 1, 0, 1), (1, 1, 256, 1),
    (2 ** 31, 1, 32, 2), (1, 2 ** 31, 32, 2), (2 ** 31 - 127, 1, 32, 2), (1, 2 ** 31 - 127, 32, 2), (2 ** 31 - 1, 2 ** 31 - 1, 32, 2),
])
def test_w4_sizes_refused(g, n, k, group, status):
    with pytest.raises(g.GemmError) as e:
        g.gemm_f16_w4_sizes(n, k, group)
    assert e.value.status == status


def test_null_outputs(g):
    lib = g.load()
    assert lib.gemm_f16_w4_sizes(1, 1, 32, None, None) == 1
    assert lib.gemm_f16_nt_w4_plan(1, 1, 1, 32, 256, None) == 1
    assert lib.gemm_f16_tn_q8_plan(1, 1, 1, 256, None) == 1


# fake, well-separated, aligned addresses: every call below is refused before
# anything reaches a device
P = [0x10000000 * (i + 1) for i in range(6)]


@pytest.mark.parametrize("call,status", [
    # NULL, overlap, alignment, sizes: quantising
    (("gemm_f16_w4_quantize", 64, 128, 64, 0, P[1], P[2], 0), 1),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], 0, P[2], 0), 1),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], P[1], 0, 0), 1),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], P[0] + 64, P[2], 0), 1),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], P[1], P[1] + 4095, 0), 1),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0] + 1, P[1], P[2], 0), 2),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], P[1] + 8, P[2], 0), 2),
    (("gemm_f16_w4_quantize", 64, 128, 64, P[0], P[1], P[2] + 4, 0), 2),
    (("gemm_f16_w4_quantize", 64, 128, 48, P[0], P[1], P[2], 0), 1),
    (("gemm_f16_w4_quantize", 0, 128, 64, 0, 0, 0, 0), 0),
    (("gemm_f16_w4_pack", 64, 128, 64, 0, P[1], P[2], P[3], 0), 1),
    (("gemm_f16_w4_pack", 64, 128, 64, P[0], 0, P[2], P[3], 0), 1),
    (("gemm_f16_w4_pack", 64, 128, 64, P[0], P[1] + 1, P[2], P[3], 0), 2),
    (("gemm_f16_w4_pack", 64, 128, 64, P[0], P[2], P[2], P[3], 0), 1),
    (("gemm_f16_w4_pack", 64, 0, 64, 0, 0, 0, 0, 0), 0),
    (("gemm_f16_w4_dequantize", 64, 128, 64, P[0], P[1], P[0], 0), 1),
    (("gemm_f16_w4_dequantize", 64, 128, 64, P[0] + 4, P[1], P[2], 0), 2),
    (("gemm_f16_q8_quantize", -1, 128, P[0], P[1], P[2], 0), 1),
    (("gemm_f16_q8_quantize", 64, 128, P[0], P[0] + 2, P[2], 0), 1),
    (("gemm_f16_q8_quantize", 64, 128, P[0], P[1] + 8, P[2], 0), 2),
    (("gemm_f16_q8_quantize", 64, 128, P[0], P[1], P[2] + 1, 0), 2),
    (("gemm_f16_q8_quantize", 64, 2 ** 31 - 1, P[0], P[1], P[2], 0), 2),
    (("gemm_f16_q8_quantize", 64, 0, 0, 0, 0, 0), 0),
    (("gemm_f16_q8_dequantize", 64, 128, P[0], P[1], P[1] - 2, 0), 1),
    (("gemm_f16_q8_dequantize", 64, 128, P[0], 0, P[2], 0), 1),
    # products
    (("gemm_f16_nt_w4", -1, 64, 128, 64, P[0], P[1], P[2], P[3], P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 96, P[0], P[1], P[2], P[3], P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, 0, P[1], P[2], P[3], P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], 0, P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[0] + 1022, P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[1] + 1024, P[4], 0, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[3], P[3], 1 << 20, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[3], P[4], -1, 0), 1),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[3], P[4] + 128, 1 << 20, 0), 2),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0] + 1, P[1], P[2], P[3], P[4], 1 << 20, 0), 2),
    (("gemm_f16_nt_w4", 4, 64, 128, 64, P[0], P[1], P[2], P[3] + 1, P[4], 1 << 20, 0), 2),
    (("gemm_f16_nt_w4", 2 ** 31, 64, 128, 64, P[0], P[1], P[2], P[3], P[4], 0, 0), 2),
    (("gemm_f16_nt_w4", 0, 64, 128, 64, 0, P[1], P[2], 0, 0, 0, 0), 0),
    (("gemm_f16_nt_w4", 4, 0, 128, 64, P[0], 0, 0, 0, 0, 0, 0), 0),
    (("gemm_f16_tn_q8", 4, -1, 128, P[0], P[1], P[2], P[3], P[4], 0, 0), 1),
    (("gemm_f16_tn_q8", 4, 64, 128, P[0], 0, P[2], P[3], P[4], 0, 0), 1),
    (("gemm_f16_tn_q8", 4, 64, 128, P[0], P[1], P[2], P[2], P[4], 0, 0), 1),
    (("gemm_f16_tn_q8", 4, 64, 128, P[0], P[1], P[2], P[3], P[1], 1 << 20, 0), 1),
    (("gemm_f16_tn_q8", 4, 64, 128, P[0], P[1] + 1, P[2], P[3], P[4], 1 << 20, 0), 2),
    (("gemm_f16_tn_q8", 2 ** 31, 64, 128, P[0], P[1], P[2], P[3], P[4], 1 << 20, 0), 2),
    (("gemm_f16_tn_q8", 0, 64, 128, 0, P[1], P[2], 0, 0, 0, 0), 0),
])
def test_c_refusals(g, call, status):
    assert getattr(g.load(), call[0])(*call[1:]) == status


@pytest.mark.parametrize("m,n,k", [(1, 16, 32), (5, 7001, 4160), (48, 4096, 4096),
                                   (333, 4096, 14336), (5000, 8192, 8192), (2000, 256, 16384)])
def test_w4_plans(g, m, n, k):
    for group in (32, 64, 128):
        p = g.gemm_f16_nt_w4_plan(m, n, k, group, 256)
        assert p.workspace_bytes >= 0 and p.splits >= 1 and p.grid >= 1
        if p.kernel == g.LOWBIT_DECODE:
            assert p.workspace_bytes >= 2 * n * k
    for bad in ((-1, n, k, 64, 256), (m, n, k, 100, 256), (m, n, k, 64, 0)):
        with pytest.raises(g.GemmError):
            g.gemm_f16_nt_w4_plan(*bad)


@pytest.mark.parametrize("m,n,k", [(1, 32, 1), (16, 4096, 8192), (8192, 4160, 4999)])
def test_q8_plans(g, m, n, k):
    p = g.gemm_f16_tn_q8_plan(m, n, k, 256)
    assert p.workspace_bytes >= 0 and p.splits >= 1 and p.grid >= 1
    for bad in ((-1, n, k, 256), (m, -1, k, 256), (m, n, k, 0)):
        with pytest.raises(g.GemmError):
            g.gemm_f16_tn_q8_plan(*bad)


@pytest.mark.parametrize("m", [1, 4, 5, 16, 17, 333, 8192])
@pytest.mark.parametrize("n", [2 ** 26, 2 ** 27 - 16, 2 ** 27, 2 ** 31 - 128])
def test_w4_launches_count_threads_in_32_bits(g, m, n):
    for k in (1, 128):
        try:
            p = g.gemm_f16_nt_w4_plan(m, n, k, 32, 256)
        except g.GemmError as e:   # as the fp16 product of such sizes is
            assert e.status == 2 and 2 * m * n >= 2 ** 40
            continue
        if p.kernel != g.LOWBIT_DECODE:
            assert p.grid * p.waves * 64 < 2 ** 32
        if n > 2 ** 26:
            assert p.kernel == g.LOWBIT_DECODE and p.workspace_bytes >= 2 * n * k


@pytest.mark.parametrize("r,n,status", [
    (2 ** 27, 544, 2), (2 ** 31 - 32, 33, 2), (2 ** 31 - 32, 32, 1), (2 ** 26, 1024, 1),
    (2 ** 26 + 1, 1024, 2), (33, 2 ** 31 - 32, 2), (32, 2 ** 31 - 32, 1),
])
def test_q8_launches_count_threads_in_32_bits(g, r, n, status):
    # what is not refused for its size is refused for its NULL arrays
    lib = g.load()
    assert lib.gemm_f16_q8_quantize(r, n, 0, 0, 0, 0) == status
    assert lib.gemm_f16_q8_dequantize(r, n, 0, 0, 0, 0) == status
    assert lib.gemm_f16_tn_q8(16, n, r, 0, 0, 0, 0, 0, 0, 0) == status
    if status == 1:   # the kernels' rows and columns a workgroup
        chunks = -(-n // 32) * 4
        wide = min(64, 1 << (chunks - 1).bit_length())
        assert -(-chunks // wide) * -(-r // (1024 // wide)) * 256 < 2 ** 32


@pytest.mark.parametrize("m,n,k", [(2 ** 31 - 9, 31, 2 ** 31 - 32), (2 ** 31 - 9, 2 ** 20, 2 ** 16),
                                   (2 ** 31 - 9, 2 ** 31 - 33, 31), (2 ** 30, 2 ** 10, 2 ** 26)])
def test_no_workspace_past_64_bits(g, m, n, k):
    """Refused, or the workspace holds the operand that is decoded."""
    for call in (lambda: g.gemm_f16_tn_q8_plan(m, n, k, 256),
                 lambda: g.gemm_f16_nt_w4_plan(m, n, k, 128, 256)):
        try:
            p = call()
        except g.GemmError as e:
            assert e.status == 2
            continue
        assert p.kernel == g.LOWBIT_DECODE and p.workspace_bytes >= 2 * n * k
    if m * k > 2 ** 60 or m * n > 2 ** 60:
        with pytest.raises(g.GemmError):
            g.gemm_f16_tn_q8_plan(m, n, k, 256)


def test_empty_products_plan_nothing(g):
    for p in (g.gemm_f16_nt_w4_plan(0, 5, 5, 32, 256), g.gemm_f16_nt_w4_plan(5, 5, 0, 32, 256),
              g.gemm_f16_tn_q8_plan(5, 0, 5, 256), g.gemm_f16_tn_q8_plan(5, 5, 0, 256)):
        assert p.workspace_bytes == 0


def test_python_refuses_cpu_and_wrong_types(g):
    h = torch.zeros(16, 128, dtype=torch.float16)
    words, scales = torch.zeros(1, 1, 64, 4, dtype=torch.int32), torch.zeros(1, 1, 16).half()
    for fn in (g.quantize_w4, g.quantize_q8):
        with pytest.raises(ValueError):
            fn(h)                       # not on a GPU
        with pytest.raises(TypeError):
            fn(h.float())
        with pytest.raises(ValueError):
            fn(h[0])
    with pytest.raises(TypeError):
        g.pack_w4(h, scales)
    with pytest.raises(ValueError):
        g.W4Matrix(words, scales, 16, 128, 128)          # right form, not on a GPU
    with pytest.raises(ValueError):
        g.W4Matrix(words, scales, 16, 128, 100)
    with pytest.raises(ValueError):
        g.W4Matrix(words, scales, 17, 128, 128)
    with pytest.raises(ValueError):
        g.W4Matrix(words, scales, -16, 128, 128)
    with pytest.raises(TypeError):
        g.W4Matrix(words.long(), scales, 16, 128, 128)
    with pytest.raises(TypeError):
        g.Q8Matrix(torch.zeros(4, 32), torch.zeros(4, 1).half(), 32)
    with pytest.raises(ValueError):
        g.Q8Matrix(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 2).half(), 32)
    with pytest.raises(ValueError):
        g.Q8Matrix(torch.zeros(4, 32, dtype=torch.int8), torch.zeros(4, 1).half(), 33)
    for fn in (g.dequantize_w4, g.dequantize_q8):
        with pytest.raises(TypeError):
            fn(h)
    for fn in (g.gemm_nt_w4, g.gemm_tn_q8):
        with pytest.raises(TypeError):
            fn(h, h)


def test_scaled_codes_are_exact_in_fp16():
    """What lets every kernel work on the same matrix: scale times code, for
    every admissible scale and code, is an fp16 number."""
    for form in (ref.W4, ref.Q8):
        s = ref.scales_list(form["bits"], form["most"])
        q = np.arange(-form["top"], form["top"] + 1)
        v = s[:, None] * q[None, :]
        v = v[np.abs(v) <= 65504]
        with np.errstate(over="ignore"):
            assert (v.astype(np.float16).astype(np.float64) == v).all()


def test_reference_layout_round_trip():
    """The reference's words hold each code where the header says."""
    rng = np.random.default_rng(3)
    codes = rng.integers(-8, 8, size=(37, 300))
    words = ref.w4_words(codes).view(np.uint32)
    for n, k in [(0, 0), (36, 299), (16, 128), (5, 77), (31, 255), (20, 131)]:
        b, t, i = n // 16, k // 128, k % 8
        lane, j = k % 32 // 8 * 16 + n % 16, k % 128 // 32
        got = (int(words[b, t, lane, j]) >> (16 * (i % 2) + 4 * (i // 2))) & 15
        assert got - 8 == codes[n, k]
