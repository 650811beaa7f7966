"""The low-bit operands at the edges of what gemm_f16_lowbit.h allows."""
import os
import subprocess
import sys

import numpy as np
import pytest

import lowbit_ref as ref
from test_gpu_lowbit import Q8_KERNELS, W4_KERNELS, dev, g, host  # noqa: F401  (g: the fixture)

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


# ---- every quotient --------------------------------------------------------------
@pytest.mark.parametrize("form", ["w4", "q8"])
def test_every_half_over_every_scale(g, form):  # noqa: F811
    """All finite fp16 numbers of both signs in groups of every scale that
    reaches them: the scale is found and each quotient rounded exactly."""
    import torch

    spec = ref.W4 if form == "w4" else ref.Q8
    top = spec["top"]
    all_scales = ref.scales_list(spec["bits"], spec["most"])
    halves = torch.arange(0x7c00, device="cuda", dtype=torch.int16).view(torch.float16)
    halves = torch.nn.functional.pad(halves, (0, -halves.numel() % 31)).view(-1, 31)
    for first in range(0, len(all_scales), 256):
        s = torch.from_numpy(all_scales[first:first + 256]).cuda()
        # the group's largest, exact in fp16 where it is not past its largest
        lead = (s * top).clamp(max=65504.0).half()
        last = s == spec["most"]
        x = halves.repeat(len(s), 1, 1)
        x[(x > lead[:, None, None]) & ~last[:, None, None]] = 0
        x = torch.cat([lead[:, None, None].expand(-1, halves.shape[0], 1), x], 2).view(len(s), -1)
        code = (x.double() / s[:, None]).round().clamp_(-top, top)
        code -= (code * s[:, None] > 65504).double()
        for x, code in ((x, code), (-x, -code)):
            q = g.quantize_w4(x, 32) if form == "w4" else g.quantize_q8(x)
            stored = q.scales.permute(0, 2, 1).reshape(-1, x.shape[1] // 32)[:len(s)] \
                if form == "w4" else q.scales
            assert (stored.double() == s[:, None]).all()
            back = g.dequantize_w4(q) if form == "w4" else g.dequantize_q8(q)
            assert (back.double() == code * s[:, None]).all()


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


# ---- sums of whole numbers -----------------------------------------------------------
# Every sum of the two tests below is a whole number of at most 2048 (times a
# power of two), so it is exact in fp32 in any order and in fp16: one product lost,
# repeated or misplaced changes a result.  With factor 2^-24 the weights are fp16's
# subnormal numbers, and A's 2^10 times larger.
def few(gen, shape, one_in):
    """-1, 0 and 1 in fp16, one in `one_in` not zero."""
    import torch

    r = torch.randint(0, 2 * one_in, shape, generator=gen, device="cuda", dtype=torch.int16)
    return (r == 0).half() - (r == 1).half()


def sign(gen, shape):
    import torch

    return torch.randint(0, 2, shape, generator=gen, device="cuda").half() * 2 - 1


def check_whole(got, a, b, factor):
    """got is a @ b exactly, times factor (a and b whole numbers)."""
    import torch

    want = torch.matmul(a.double(), b.double().contiguous())
    assert want.abs().max() <= 2048
    assert torch.equal(got.double(), want * factor)


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kernel,m,n,k", W4_KERNELS)
def test_nt_w4_whole_sums(g, kernel, m, n, k, small):  # noqa: F811
    import torch

    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    codes = torch.randint(-8, 8, (n, k), generator=gen, device="cuda", dtype=torch.int8)
    signs = sign(gen, (n, -(-k // 32)))
    w = codes.half() * signs.repeat_interleave(32, 1)[:, :k]
    a = few(gen, (m, k), 8)
    scale, up = (2.0 ** -24, 2.0 ** 10) if small else (1.0, 1.0)
    q = g.pack_w4(codes, signs * scale, 32)
    check_whole(g.gemm_nt_w4(a * up, q), a, w.t(), scale * up)


@pytest.mark.parametrize("small", [False, True])
@pytest.mark.parametrize("kernel,splits,m,n,k", Q8_KERNELS)
def test_tn_q8_whole_sums(g, kernel, splits, m, n, k, small):  # noqa: F811
    import torch

    gen = torch.Generator(device="cuda").manual_seed(m + n + k)
    groups = -(-n // 32)
    codes = torch.zeros((k, groups * 32), device="cuda", dtype=torch.int8)
    codes[:, :n] = torch.randint(-20, 21, (k, n), generator=gen, device="cuda", dtype=torch.int8)
    signs = sign(gen, (k, groups))
    x = (codes.half() * signs.repeat_interleave(32, 1))[:, :n]
    a = few(gen, (k, m), 20)
    scale, up = (2.0 ** -24, 2.0 ** 10) if small else (1.0, 1.0)
    got = g.gemm_tn_q8(a * up, g.Q8Matrix(codes, signs * scale, n))
    check_whole(got, a.t().contiguous(), x, scale * up)


# ---- streams --------------------------------------------------------------------
LIVES = ["quantize_w4", "pack_w4", "dequantize_w4", "quantize_q8", "dequantize_q8",
         "w4 streamed", "w4 tiles", "w4 tiles, workspace", "w4 decoded", "q8 streamed", "q8 decoded"]


def operands_and_call(g, what):  # noqa: F811
    """(call(**kw) giving tensors, the tensors that it is given)."""
    import torch

    rng = np.random.default_rng(3)
    x = dev(rng.standard_normal((1024, 2048)).astype(np.float16))
    if what == "quantize_w4":
        def call(**kw):
            q = g.quantize_w4(x, 64, **kw)
            return q.words, q.scales
        return call, [x]
    if what == "quantize_q8":
        def call(**kw):
            q = g.quantize_q8(x, **kw)
            return q.codes, q.scales
        return call, [x]
    if what == "pack_w4":
        codes = dev(rng.integers(-8, 8, (1024, 2048)).astype(np.int8))
        scales = dev(rng.uniform(0.5, 1, (1024, 32)).astype(np.float16))

        def call(**kw):
            q = g.pack_w4(codes, scales, 64, **kw)
            return q.words, q.scales
        return call, [codes, scales]
    if what in ("dequantize_q8", "q8 streamed", "q8 decoded"):
        q = g.quantize_q8(x)
        if what == "dequantize_q8":
            return lambda **kw: (g.dequantize_q8(q, **kw),), [q.codes, q.scales]
        a = dev(rng.standard_normal((1024, 16 if what == "q8 streamed" else 1200)).astype(np.float16))
        return lambda **kw: (g.gemm_tn_q8(a, q, **kw),), [a, q.codes, q.scales]
    q = g.quantize_w4(x, 64)
    if what == "dequantize_w4":
        return lambda **kw: (g.dequantize_w4(q, **kw),), [q.words, q.scales]
    rows = {"w4 streamed": 8, "w4 decoded": 8200}.get(what, 80)
    a = dev(rng.standard_normal((rows, 2048)).astype(np.float16))
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    plan = g.gemm_f16_nt_w4_plan(rows, q.n, q.k, 64, cus)
    assert plan.kernel == {"w4 streamed": g.LOWBIT_STREAM, "w4 decoded": g.LOWBIT_DECODE}.get(
        what, g.LOWBIT_TILE)
    if what != "w4 tiles, workspace":
        return lambda **kw: (g.gemm_nt_w4(a, q, **kw),), [a, q.words, q.scales]
    assert plan.workspace_bytes > 0
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    return lambda **kw: (g.gemm_nt_w4(a, q, workspace=ws, **kw),), [a, q.words, q.scales, ws]


@pytest.mark.parametrize("what", LIVES)
def test_operands_dropped_at_once(g, what):  # noqa: F811
    """Operands (and a workspace) of the default stream, used on a busy stream
    and dropped at once: their memory goes to no other tensor before they are
    read."""
    import torch

    want = [host(t) for t in operands_and_call(g, what)[0]()]
    s, done = torch.cuda.Stream(), torch.cuda.Event()
    filler = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    # torch's memory for what both streams allocate later: new memory from the
    # driver would wait for s
    operands_and_call(g, what)[0](stream=s)
    s.synchronize()
    call, given = operands_and_call(g, what)
    ranges = [(t.data_ptr(), t.numel() * t.element_size()) for t in given]
    spare = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in ranges
             for _ in range(8)]
    del spare
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(200):   # some 40 ms
            filler[:1 << 29].copy_(filler[1 << 29:])
    got = call(stream=s)
    done.record(s)
    del call, given
    later = [torch.empty(size, dtype=torch.uint8, device="cuda") for _, size in ranges
             for _ in range(4)]
    # (asked before the default stream gets work: it may share a hardware queue with s)
    assert not done.query(), "the stream was not busy for long enough to show anything"
    for t in later:
        for at, size in ranges:
            assert t.data_ptr() + t.numel() <= at or at + size <= t.data_ptr()
        t.fill_(0x55)
    s.synchronize()
    for t, w in zip(got, want):
        np.testing.assert_array_equal(host(t), w)


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
