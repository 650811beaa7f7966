"""The low-bit operands at the edges of what gemm_f16_lowbit.h allows."""
import os
import subprocess
import sys

import numpy as np
import pytest

import lowbit_ref as ref
from test_gpu_lowbit import W4_KERNELS, dev, g, host  # noqa: F401  (g: the fixture)

pytestmark = pytest.mark.gpu


# ---- another quantiser's scales ------------------------------------------------
def test_w4_pack_every_scale(g):  # noqa: F811
    """Every fp16 bit pattern as a scale, NaNs of any payload and either sign
    among them: rounded to 8 bits, or its group NaN with codes 0 where it is not
    finite or rounds past 65504; the group beside it as it was."""
    bits = np.arange(1 << 16, dtype=np.uint32).astype(np.uint16)
    scales = np.ones((1 << 16, 2), np.float16)
    scales[:, 0] = bits.view(np.float16)
    codes = np.full((1 << 16, 64), -1, np.int8)
    q = g.pack_w4(dev(codes), dev(scales), 32)
    r = ref.round8(scales)
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(r) <= 65504)
    assert bad[:, 0].sum() > 2 * 1024 and not bad[:, 1].any()
    want = codes.astype(np.int64)
    want[:, :32][bad[:, 0]] = 0
    assert (host(q.words) == ref.w4_words(want)).all()
    stored = host(q.scales).astype(np.float64)
    r[bad] = np.nan
    np.testing.assert_array_equal(stored, ref.w4_scales(r, 1 << 16, 64, 32, 0.0))
    np.testing.assert_array_equal(host(g.dequantize_w4(q)).astype(np.float64),
                                  ref.values(want, r, 32, 64))


# ---- storage that another program laid out ---------------------------------------
def padded(k, group):
    """Whether the last tile of K has groups that lie past K."""
    return -(-k // group) * group < -(-k // 128) * 128


@pytest.mark.parametrize("kernel,m,n,k,group",
                         [(*case, group) for case in W4_KERNELS for group in (32, 64)
                          if padded(case[3], group)])
def test_nt_w4_scales_past_the_matrix(g, kernel, m, n, k, group):  # noqa: F811
    """Scales of groups past K and of rows past N belong to no weight: NaN and
    infinities in them (memory that a program did not fill) reach no result."""
    import torch

    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    q = g.quantize_w4(torch.randn(n, k, generator=gen, device="cuda").half(), group)
    a = torch.randn(m, k, generator=gen, device="cuda").half()
    want = g.gemm_nt_w4(a, q)
    assert want.isfinite().all()
    groups = -(-k // group)
    assert q.scales[:, groups:].numel() > 0
    for value in (float("nan"), float("inf"), -65504.0):
        q.scales[:, groups:] = value
        if n % 16:
            q.scales[-1, :, n % 16:] = value
        assert torch.equal(g.gemm_nt_w4(a, q), want)
        assert g.dequantize_w4(q).isfinite().all()


# ---- saved and read back ----------------------------------------------------------
READ_BACK = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, dense_fp16_gemm_amd as g
safe = sys.argv[3] == "safe"
if safe:
    torch.serialization.add_safe_globals([g.W4Matrix, g.Q8Matrix])
w, x, a, dy, y, dw = torch.load(sys.argv[2], weights_only=safe)
assert torch.equal(g.gemm_nt_w4(a, w), y) and torch.equal(g.gemm_tn_q8(dy, x), dw)
assert (w.shape, w.group, x.shape) == ((50, 200), 64, (30, 70))
print("same")
"""


@pytest.mark.parametrize("how", ["safe", "any"])
def test_saved_matrices_in_a_new_process(g, how, tmp_path):  # noqa: F811
    import torch

    gen = torch.Generator(device="cuda").manual_seed(1)
    w = g.quantize_w4(torch.randn(50, 200, generator=gen, device="cuda").half(), 64)
    x = g.quantize_q8(torch.randn(30, 70, generator=gen, device="cuda").half())
    a = torch.randn(3, 200, generator=gen, device="cuda").half()
    dy = torch.randn(30, 9, generator=gen, device="cuda").half()
    path = str(tmp_path / "matrices.pt")
    torch.save((w, x, a, dy, g.gemm_nt_w4(a, w), g.gemm_tn_q8(dy, x)), path)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", READ_BACK, root, path, how], timeout=100,
                       capture_output=True)
    assert r.returncode == 0 and r.stdout == b"same\n", r.stderr.decode()[-2000:]
