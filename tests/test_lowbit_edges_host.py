"""What the low-bit operands' tests on a GPU cannot show, or need not (no GPU):
matrices read back in a new process, and how a wave's lanes exchange data in LDS."""
import os
import pickle
import re
import subprocess
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def g():
    import dense_fp16_gemm_amd as lib

    lib.load()
    return lib


def on_cpu(g):
    """A matrix of each form whose tensors left the GPU."""
    w = g.W4Matrix.__new__(g.W4Matrix)._set(torch.zeros(1, 1, 64, 4, dtype=torch.int32),
                                            torch.zeros(1, 1, 16).half(), 16, 128, 128)
    x = g.Q8Matrix.__new__(g.Q8Matrix)._set(torch.zeros(4, 32, dtype=torch.int8),
                                            torch.zeros(4, 1).half(), 4, 32)
    return w, x


IN_A_NEW_PROCESS = """
import pickle, sys
sys.path.insert(0, sys.argv[1])
import torch, dense_fp16_gemm_amd as g
data = pickle.load(sys.stdin.buffer)
for name, stored in data.items():
    try:
        m = pickle.loads(stored)
        if name.startswith("gemm"):
            getattr(g, name)(torch.zeros(4, 128).half(), m)
        else:
            getattr(g, name)(m)
    except ValueError as e:
        assert "GPU" in str(e), e
    else:
        raise AssertionError(name)
print("refused")
"""


def test_unpickled_in_a_new_process(g):
    """The first use of this package there is of a matrix that was read back."""
    w, x = (pickle.dumps(m) for m in on_cpu(g))
    for name, m in (("gemm_nt_w4", w), ("gemm_tn_q8", x), ("dequantize_w4", w), ("dequantize_q8", x)):
        r = subprocess.run([sys.executable, "-c", IN_A_NEW_PROCESS, ROOT], timeout=300,
                           input=pickle.dumps({name: m}), capture_output=True)
        assert r.returncode == 0 and r.stdout == b"refused\n", r.stderr.decode()[-2000:]


def test_read_back_matrices_are_checked(g):
    """A stored matrix goes through its constructor again."""
    for m in on_cpu(g):
        with pytest.raises(ValueError, match="GPU"):
            pickle.loads(pickle.dumps(m))


def test_dequantize_refuses_host_memory(g):
    w, x = on_cpu(g)
    for call, m in ((g.dequantize_w4, w), (g.dequantize_q8, x)):
        for out in (None, torch.zeros(m.shape).half()):
            with pytest.raises(ValueError, match="GPU"):
                call(m, out=out)


@pytest.mark.parametrize("kernel,write,read", [
    ("w4_rows_kernel", r"ab\[[^;]*\] = af", r"read_a\(0, mt\)"),
    ("q8_tn_kernel", r"my\.(?:a|s)\[[^;]*(?:av|sv)\[buf\]", r"lds_read_tr16\(src\)|half8_t \*>\(&my\.s"),
], ids=["w4_rows", "q8_tn"])
def test_lanes_of_a_wave_exchange_data_across_a_fence(kernel, write, read):
    """Without one the compiler may move a lane's reads past its own writes, since
    it does not know that other lanes wrote what they read.  One fence stands
    before the writes (of what may still have to be read), one before the reads."""
    source = open(os.path.join(ROOT, "dense_fp16_gemm_amd", "csrc", "lowbit.hip")).read()
    body = source[source.index(f"void {kernel}("):]
    body = body[body.index("auto mma = "):]
    body = body[:body.index("\n    };\n")]
    steps = [m.lastgroup for m in re.finditer(
        rf"(?P<fence>wave_lds_fence\(\);)|(?P<write>{write})|(?P<read>{read})", body)]
    steps = [s for i, s in enumerate(steps) if i == 0 or s != steps[i - 1]]
    assert steps == ["fence", "write", "fence", "read"]
