"""Products in 8-bit floating point at the edges of what their header allows."""
import numpy as np
import pytest
import torch

import f8_ref as ref
from test_gpu_f8 import g, host  # noqa: F401  (g: the fixture)
from test_gpu_f8_tiles import generator

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
