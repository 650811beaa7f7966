"""Plans of the 8-bit products and workspaces of the routing, without a GPU."""
import random

import pytest

from test_f8_host import INVALID, UNSUPPORTED, at, g, refused  # noqa: F401  (g: the fixture)


def sizes(rng):
    return rng.choice((1, 3, 17, 100, 1000, 4096)), rng.choice((16, 300, 2048, 8190)), rng.choice((1, 130, 2048, 9000))


def test_plans_do_not_depend_on_those_before(g):
    """A plan is the same after many others, in whatever order they come."""
    rng = random.Random(0)
    cases = [sizes(rng) + (rng.random() < 0.5,) for _ in range(40)]
    first = [g.gemm_f16_nt_f8_plan(m, n, k, 128, f16, 256).as_dict() for m, n, k, f16 in cases]
    experts = [g.gemm_f16_nt_f8_experts_plan(8 * m, 16, n, k, 8, f16, 256).as_dict() for m, n, k, f16 in cases]
    for i in rng.sample(range(40), 40):
        m, n, k, f16 = cases[i]
        assert g.gemm_f16_nt_f8_experts_plan(8 * m, 16, n, k, 8, f16, 256).as_dict() == experts[i]
        assert g.gemm_f16_nt_f8_plan(m, n, k, 128, f16, 256).as_dict() == first[i]
        g.gemm_f16_nt_f8_plan(m, n, k, 128, f16, 64)


@pytest.mark.parametrize("cus", [1, 8, 100, 256, 304])
def test_workspaces(g, cus):
    """The ranges' sums, whole tiles of them, and A's quantised form, each at 256
    bytes; ranges end within K; nothing more than fits on the device at once where
    workgroups take several tiles."""
    rng = random.Random(cus)
    for _ in range(300):
        m, n, k = sizes(rng)
        f16 = rng.random() < 0.5
        p = g.gemm_f16_nt_f8_plan(m, n, k, 128, f16, cus)
        need = 0
        if p.splits > 1:
            need += 4 * p.splits * (-(-m // p.block_m) * p.block_m) * (-(-n // p.block_n) * p.block_n)
            assert p.splits <= -(-k // 128)
        if f16 and p.kernel == g.LOWBIT_TILE:
            for size in g.gemm_f16_f8_sizes(1, m, k, 1):
                need += -(-size // 256) * 256
        assert p.workspace_bytes == need
        tiles = -(-m // p.block_m) * -(-n // p.block_n) * p.splits
        assert p.grid == tiles or (p.grid in (cus, 2 * cus) and p.grid < tiles and p.block_m * p.block_n >= 128 * 128)


def test_far_sizes(g):
    """Sizes at the ends of their ranges: a plan within a launch, or a refusal."""
    for m in (1, 2 ** 22, 2 ** 31 - 128):
        for n in (1, 16, 2 ** 22, 2 ** 31 - 128):
            for k in (0, 1, 128, 2 ** 23):
                for f16 in (False, True):
                    try:
                        p = g.gemm_f16_nt_f8_plan(m, n, k, 1, f16, 256)
                    except g.GemmError as e:
                        assert e.status == UNSUPPORTED
                        continue
                    assert 1 <= p.grid and p.grid * 64 * p.waves < 2 ** 32
                    assert 0 <= p.workspace_bytes < 2 ** 45
    for s in (1, 2 ** 20, 2 ** 31 - 1024):
        for e in (1, 1000, 1024):
            for n, k in ((1, 1), (2 ** 20, 128), (128, 2 ** 23)):
                try:
                    p = g.gemm_f16_nt_f8_experts_plan(s, e, n, k, 0, False, 256)
                except g.GemmError as err:
                    assert err.status == UNSUPPORTED
                    continue
                assert 1 <= p.grid and p.grid * 64 * p.waves < 2 ** 32


def test_route_workspaces(g):
    for t, top, e in ((1, 8, 64), (256, 8, 64), (16, 32, 1024)):
        assert g.gemm_f16_route_workspace(t, e, top) == 0
    for t, top, e in ((257, 8, 64), (8192, 8, 256), (100000, 6, 128), ((2 ** 31 - 1024) // 32, 32, 1024)):
        need = g.gemm_f16_route_workspace(t, e, top)
        assert 0 < need <= 256 * e * 4 and need % (4 * e) == 0
        good = [t, e, top, 0, 1, 1, 0, 1, 1.0, at(0), 1, 0, at(1), at(2), at(3), at(4), at(5)]
        refused(g, INVALID, g.gemm_f16_route, *good, 0, 0)
        refused(g, INVALID, g.gemm_f16_route, *good, at(6), need - 1)
        refused(g, INVALID, g.gemm_f16_route, *good, at(0), need)       # over the logits
        refused(g, UNSUPPORTED, g.gemm_f16_route, *good, at(6) + 4, need)
