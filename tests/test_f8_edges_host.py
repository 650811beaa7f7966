"""The 8-bit floating point operands and the experts' layers at the edges of what
their headers allow, without a GPU."""
import pytest

from test_f8_host import INVALID, UNSUPPORTED, g, refused  # noqa: F401  (g: the fixture)


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


def test_gradients_plans(g):
    """The experts' weight gradients: no workspace, one tile of each expert's matrix a
    unit, workgroups that take several units where there are more than fit at once."""
    plan = g.gemm_f16_nt_f8_experts_grad_plan
    for t, e, top in ((1, 1, 1), (33, 8, 2), (4096, 64, 8), (300, 300, 1), (9000, 1024, 4)):
        for m, n in ((16, 128), (1408, 2048), (7001, 33)):
            p = plan(t * top, e, m, n, 256)
            units = -(-e // 8) * 8 * -(-m // p.block_m) * -(-n // p.block_n)
            assert p.kernel == g.LOWBIT_TILE and p.splits == 1 and p.workspace_bytes == 0
            assert p.grid == units or (p.grid in (256, 512) and p.grid < units)
    assert plan(8, 4, 0, 128, 256).grid == 0
    refused(g, INVALID, plan, -1, 4, 16, 128, 256)
    refused(g, INVALID, plan, 8, 0, 16, 128, 256)
    refused(g, INVALID, plan, 8, 4, -1, 128, 256)
    refused(g, INVALID, plan, 8, 4, 16, 128, 0)
    refused(g, UNSUPPORTED, plan, 8, 1025, 16, 128, 256)
    refused(g, UNSUPPORTED, plan, 8, 1024, 2 ** 20, 2 ** 20, 256)
