"""8-bit products and layers of experts as programs use them: at the edges of what
their headers allow, on other streams, saved and read back, all steps together."""
import copy
import os
import pickle
import subprocess
import sys

import pytest
import torch

from test_gpu_f8 import g  # noqa: F401  (g: the fixture)

pytestmark = pytest.mark.gpu


def stream():
    return torch.cuda.current_stream().cuda_stream


# ---- rows of nearly 2^31 columns -------------------------------------------------
WIDEST = 2 ** 31 - 8     # the last of a wave's steps of 2048 columns ends past 2^31


def widest_row():
    """One row of small whole numbers."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    part = torch.randint(-2, 3, (2 ** 28,), device="cuda", generator=gen).half()
    x = torch.empty(1, WIDEST, dtype=torch.float16, device="cuda")
    for at in range(0, WIDEST, 2 ** 28):
        x[0, at:at + 2 ** 28] = part[: WIDEST - at]
    return x


def guarded_row():
    """A row's memory, and what lies around it."""
    memory = torch.full((WIDEST + 8192,), 3.0, dtype=torch.float16, device="cuda")
    return memory[4096:4096 + WIDEST].view(1, WIDEST), (memory[:4096], memory[4096 + WIDEST:])


def test_combine_widest(g):
    """One token, one choice, as many columns as a call takes: both directions."""
    x = widest_row()
    r = g.route(torch.zeros(1, 1, device="cuda"), 1, scale=0.5)
    assert r.places.tolist() == [[0]] and r.weights.tolist() == [[0.5]]
    out, around = guarded_row()
    g.combine_experts(x, r, out=out)
    half = x * 0.5
    assert torch.equal(out, half)
    # the inner product: of the first and the last columns, so that it is a small whole number
    y = torch.zeros_like(x)
    ends = (slice(0, 4096), slice(WIDEST - 4096, WIDEST))
    for part in ends:
        y[0, part] = x[0, part]
    out.fill_(9.0)
    dw = torch.zeros(1, 1, device="cuda")
    g.gemm_f16_combine_backward(1, 1, WIDEST, x.data_ptr(), y.data_ptr(), r.weights.data_ptr(), r.rows.data_ptr(),
                                r.places.data_ptr(), out.data_ptr(), dw.data_ptr(), stream())
    assert torch.equal(out, half)
    assert dw.item() == sum((x[0, part].double() ** 2).sum().item() for part in ends)
    assert all((v == 3).all() for v in around)


def test_combine_widest_of_no_expert(g):
    """The same for a token without an expert: a row of zeros."""
    x = torch.ones(1, WIDEST, dtype=torch.float16, device="cuda")
    r = g.route(torch.full((1, 1), -torch.inf, device="cuda"), 1)
    assert r.places.tolist() == [[-1]] and r.rows.tolist() == [-1]
    out, around = guarded_row()
    g.gemm_f16_combine_backward(1, 1, WIDEST, x.data_ptr(), 0, 0, r.rows.data_ptr(), r.places.data_ptr(),
                                out.data_ptr(), 0, stream())
    assert torch.count_nonzero(out).item() == 0
    out.fill_(9.0)
    g.combine_experts(x, r, out=out)
    assert torch.count_nonzero(out).item() == 0
    assert all((v == 3).all() for v in around)


# ---- streams ----------------------------------------------------------------------
class ElsewhereStream:
    """A stream of another device."""
    device = torch.device("cuda", 1)
    cuda_stream = 0


def test_streams_of_another_device_are_refused(g):
    """By every function, whether it allocates its output or is given it."""
    f16 = dict(dtype=torch.float16, device="cuda")
    t, e, top, n, k = 4, 3, 2, 20, 130
    x, dy, w = torch.ones(t, k, **f16), torch.ones(t * top, n, **f16), torch.ones(e, n, k, **f16)
    logits = torch.zeros(t, e, device="cuda")
    r, w8, one = g.route(logits, top), g.quantize_f8(w, 128), g.quantize_f8(w[0], 128)
    dy8, x8 = g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True)
    s = ElsewhereStream()
    calls = [
        lambda: g.quantize_f8(x, stream=s), lambda: g.quantize_f8(w, 128, stream=s),
        lambda: g.route(logits, top, stream=s), lambda: g.route_backward(logits, r, r.weights, stream=s),
        lambda: g.quantize_f8_experts(x, r, gather=True, stream=s), lambda: g.combine_experts_backward(x, None, r, weighted=False, stream=s),
    ]
    for fn, args, shape in ((g.dequantize_f8, (one,), (n, k)), (g.dequantize_f8, (w8,), (e, n, k)),
                            (g.gemm_nt_f8, (x, one), (t, n)), (g.gemm_nt_f8_experts, (x, w8, r, True), (t * top, n)),
                            (g.gemm_nt_f8_experts_grad, (dy8, x8, r), (e, n, k)), (g.combine_experts, (dy, r), (t, n))):
        fn(*args, out=torch.empty(shape, **f16))      # what is wrong is the stream alone
        for out in (None, torch.empty(shape, **f16)):
            calls.append(lambda fn=fn, args=args, out=out: fn(*args, out=out, stream=s))
    for call in calls:
        with pytest.raises(ValueError, match="stream is on"):
            call()


# ---- saved and read back -----------------------------------------------------------
READ_BACK = """
import sys
sys.path.insert(0, sys.argv[1])
import torch, dense_fp16_gemm_amd as g
safe = sys.argv[3] == "safe"
if safe:
    torch.serialization.add_safe_globals([g.F8Matrix, g.Routing])
stored = torch.load(sys.argv[2], weights_only=safe)
def same(a, b):
    assert torch.equal(a, b)
if "gemm_nt_f8" in stored:
    a, w, stack, y, values = stored["gemm_nt_f8"]
    assert (a.shape, a.block, w.shape, w.block, stack.shape) == ((3, 200), 1, (50, 200), 128, (4, 50, 200))
    same(g.gemm_nt_f8(a, w), y)
    same(g.dequantize_f8(stack), values)
else:
    r, logits, x, w, y, out, dlogits = stored["route"]
    assert (r.tokens, r.top, r.n_experts, r.scores, r.renormalize, r.scale) == (30, 2, 4, "sigmoid", False, 2.5)
    same(g.combine_experts(y, r), out)
    same(g.gemm_nt_f8_experts(x, w, r, gather=True), y)
    same(g.route_backward(logits, r, torch.ones_like(r.weights)), dlogits)
print("same")
"""


@pytest.mark.parametrize("how", ["safe", "any"])
@pytest.mark.parametrize("what", ["gemm_nt_f8", "route"])
def test_saved_in_a_new_process(g, how, what, tmp_path):
    """Matrices and a routing, saved whole: in a process whose first use of the package
    is of what it read back."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def halves(*shape):
        return torch.randn(shape, generator=gen, device="cuda").half()

    stack = g.quantize_f8(halves(4, 50, 200), 128)
    if what == "gemm_nt_f8":
        a, w = g.quantize_f8(halves(3, 200)), g.quantize_f8(halves(50, 200), 128)
        stored = a, w, stack, g.gemm_nt_f8(a, w), g.dequantize_f8(stack)
    else:
        logits, x = torch.randn(30, 4, generator=gen, device="cuda"), halves(30, 200)
        r = g.route(logits, 2, "sigmoid", renormalize=False, scale=2.5)
        y = g.gemm_nt_f8_experts(x, stack, r, gather=True)
        stored = r, logits, x, stack, y, g.combine_experts(y, r), g.route_backward(logits, r, torch.ones_like(r.weights))
    path = str(tmp_path / "stored.pt")
    torch.save({what: stored}, path)
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", READ_BACK, root, path, how], timeout=100, capture_output=True)
    assert done.returncode == 0 and done.stdout == b"same\n", done.stderr.decode()[-2000:]


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))])
def test_copies(g, how):
    """Copies hold the same and are checked as what a program makes itself."""
    x = torch.randn(7, 130, device="cuda").half()
    q = g.quantize_f8(x)
    again = how(q)
    assert (again.shape, again.block) == (q.shape, q.block)
    assert torch.equal(g.dequantize_f8(again), g.dequantize_f8(q))
    r = g.route(torch.randn(7, 5, device="cuda"), 2, scale=0.5)
    s = how(r)
    assert (s.scores, s.renormalize, s.scale, s.n_experts) == (r.scores, r.renormalize, r.scale, r.n_experts)
    assert torch.equal(g.combine_experts(x.repeat(2, 1), s), g.combine_experts(x.repeat(2, 1), r))
    assert (s.weights.data_ptr() == r.weights.data_ptr()) == (how is copy.copy)
