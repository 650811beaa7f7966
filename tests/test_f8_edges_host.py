"""The 8-bit floating point operands and the experts' layers at the edges of what
their headers allow, without a GPU."""
import pytest

from test_f8_host import UNSUPPORTED, g  # noqa: F401  (g: the fixture)


def plan_or_refusal(g, fn, *args):
    try:
        return fn(*args)
    except g.GemmError as e:
        assert e.status == UNSUPPORTED
        return None


@pytest.mark.parametrize("big", [2 ** 31 - 128, 2 ** 31 - 255, 2 ** 31 - 256, 2 ** 31 - 300, 2 ** 31 - 1000])
def test_tiles_end_within_32_bits(g, big):
    """What the kernels compute of a tile, its end too, fits 32 bits: a plan has no
    tile that ends past 2^31 - 1."""
    planned = 0
    for small in (1, 16, 17, 64, 128, 200, 256, 300, 1000, 4096):
        for k in (1, 128, 512, 4096):
            for f16 in (False, True):
                for m, n in ((big, small), (small, big)):
                    p = plan_or_refusal(g, g.gemm_f16_nt_f8_plan, m, n, k, 1, f16, 256)
                    if p is None:
                        continue
                    planned += 1
                    assert -(-m // p.block_m) * p.block_m < 2 ** 31
                    assert -(-n // p.block_n) * p.block_n < 2 ** 31
                p = plan_or_refusal(g, g.gemm_f16_nt_f8_experts_plan, small, 1, big, k, 0, f16, 256)
                assert p is None or -(-big // p.block_n) * p.block_n < 2 ** 31
    assert planned
