"""The low-bit operands at the edges of what gemm_f16_lowbit.h allows."""
import numpy as np
import pytest

import lowbit_ref as ref
from test_gpu_lowbit import dev, g, host  # noqa: F401  (g: the fixture)

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
