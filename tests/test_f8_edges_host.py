"""The 8-bit floating point operands and the experts' layers at the edges of what
their headers allow, without a GPU."""
import os
import pickle
import subprocess
import sys

import pytest
import torch

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


# ---- matrices and routings whose tensors left the GPU -------------------------------
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def on_cpu(g):
    g.f8._bind_torch()     # as the first matrix does
    matrix = g.F8Matrix.__new__(g.F8Matrix)._set(torch.zeros(4, 128).to(torch.float8_e4m3fn),
                                                 torch.zeros(1, 4, 4, dtype=torch.uint8), 128, 1)
    i = torch.zeros(4, 2, dtype=torch.int32)
    routing = g.Routing.__new__(g.Routing)._set(i, torch.zeros(4, 2), i.view(-1), i, torch.zeros(9, dtype=torch.int32),
                                                "softmax", True, 1.0)
    return matrix, routing


IN_A_NEW_PROCESS = """
import pickle, sys
sys.path.insert(0, sys.argv[1])
import torch, dense_fp16_gemm_amd as g
try:
    pickle.loads(sys.stdin.buffer.read())
except ValueError as e:
    assert "GPU" in str(e), e
    print("refused")
"""


@pytest.mark.parametrize("which", [0, 1])
def test_read_back_is_checked(g, which):
    """What was stored goes through its constructor again, also where that is the first
    use of the package in a process."""
    stored = pickle.dumps(on_cpu(g)[which])
    with pytest.raises(ValueError, match="GPU"):
        pickle.loads(stored)
    r = subprocess.run([sys.executable, "-c", IN_A_NEW_PROCESS, ROOT], timeout=300, input=stored, capture_output=True)
    assert r.returncode == 0 and r.stdout == b"refused\n", r.stderr.decode()[-2000:]


def test_host_memory_is_refused(g):
    """By every function that takes a matrix or a routing."""
    q, r = on_cpu(g)
    x, dy = torch.zeros(4, 128).half(), torch.zeros(8, 128).half()
    for call in (lambda: g.dequantize_f8(q), lambda: g.gemm_nt_f8(q, q), lambda: g.gemm_nt_f8(x, q),
                 lambda: g.route_backward(torch.zeros(4, 8), r, r.weights), lambda: g.quantize_f8_experts(dy, r),
                 lambda: g.gemm_nt_f8_experts(x, q, r, gather=True), lambda: g.gemm_nt_f8_experts_grad(q, q, r),
                 lambda: g.combine_experts(dy, r), lambda: g.combine_experts_backward(x, dy, r)):
        with pytest.raises(ValueError, match="GPU"):
            call()
