"""The 8-bit products' kernels for many rows, each reached by sizes whose tiles and
ranges end anywhere: whole numbers, whose products and sums are exact in fp32
whatever their order, against 64 bits."""
import numpy as np
import pytest
import torch

import f8_ref as ref
from test_gpu_f8 import g  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu

# e4m3 codes of -2 .. 2
CODES = (0xc0, 0xb8, 0x00, 0x38, 0x40)


def whole(gen, r, k, block, count=None, spread=2):
    """Random codes of small whole numbers and scales from 2^-spread to 2^spread:
    (codes, stored scales, the values in fp64)."""
    lead = () if count is None else (count,)
    kp, groups, blocks = -(-k // 128) * 128, -(-k // 128), -(-r // block)
    i = torch.randint(0, 5, lead + (r, kp), generator=gen, device="cuda")
    i[..., k:] = 2
    codes = torch.tensor(CODES, dtype=torch.uint8, device="cuda")[i]
    e = torch.randint(-spread, spread + 1, lead + (blocks, groups), generator=gen, device="cuda")
    pad = torch.nn.functional.pad(e + 127, (0, -groups % 4), value=127).to(torch.uint8)
    scales = pad.unflatten(-1, (-1, 4)).transpose(-3, -2).contiguous()
    s = torch.exp2(e.double()).repeat_interleave(128, -1).repeat_interleave(block, -2)[..., :r, :]
    return codes.view(torch.float8_e4m3fn), scales, ((i - 2).double() * s)[..., :k].contiguous()


def generator(seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return gen


def product(a, b):
    return torch.matmul(a, b.t().contiguous()).half()


def guarded(shape):
    """A C at 2-byte alignment and what lies around it."""
    size = 1
    for n in shape:
        size *= n
    buf = torch.full((size + 512,), 3.0, dtype=torch.float16, device="cuda")
    return buf[131:131 + size].view(shape), (buf[:131], buf[131 + size:])


# m, n, k, the tile, whether K is in ranges
DENSE = [(5, 100, 2048, 32, 64, True), (70, 300, 200, 32, 64, False),
         (300, 264, 2048, 64, 64, True), (256, 2050, 130, 64, 64, False),
         (333, 1001, 4000, 64, 128, True), (333, 3001, 130, 64, 128, False),
         (333, 2050, 8200, 128, 128, True), (1000, 2050, 300, 128, 128, False),
         (513, 4096, 600, 128, 128, False),
         (5614, 133, 6923, 256, 192, True), (4097, 2050, 130, 256, 192, False),
         (3818, 5761, 700, 256, 192, False),
         (5377, 450, 9558, 256, 256, True), (3001, 4096, 130, 256, 256, False),
         (8191, 4090, 300, 256, 256, False), (1405, 8090, 134, 256, 256, False)]


def test_dense_reaches_every_kernel(g):
    cus = g.gemm_f16_device_cus()
    if cus != 256:
        pytest.skip("the sizes are for 256 compute units")
    reached = set()
    for m, n, k, bm, bn, split in DENSE:
        p = g.gemm_f16_nt_f8_plan(m, n, k, 128, False, cus)
        reached.add((p.block_m, p.block_n, p.splits > 1))
    assert reached == {case[3:] for case in DENSE}


@pytest.mark.parametrize("m,n,k", [case[:3] for case in DENSE])
@pytest.mark.parametrize("block", [1, 128])
def test_dense(g, m, n, k, block):
    gen = generator(m + n + k)
    ac, as_, a = whole(gen, m, k, 1)
    bc, bs, b = whole(gen, n, k, block)
    out, around = guarded((m, n))
    g.gemm_nt_f8(g.F8Matrix(ac, as_, k, 1), g.F8Matrix(bc, bs, k, block), out=out)
    assert torch.equal(out, product(a, b))
    assert all((x == 3).all() for x in around)


def uneven(gen, t, e, top, padded=True):
    """Logits of which some experts get most, some nothing, and some tokens none."""
    x = torch.randn(t, e, generator=gen, device="cuda")
    x += 2 * torch.randn(e, generator=gen, device="cuda")
    x[:, torch.randperm(e, generator=gen, device="cuda")[: e // 4]] -= 100
    if padded:
        x[torch.rand(t, generator=gen, device="cuda") < 0.05] = -torch.inf
        x[t - t // 10:] = -torch.inf
    return x


EXPERTS = [(4100, 32, 2, 1030, 300), (8000, 8, 2, 1025, 130), (16000, 1, 1, 70, 257), (8192, 4, 1, 1024, 600),
           (900, 8, 3, 520, 1000), (4100, 300, 4, 264, 140), (333, 64, 6, 136, 513), (3000, 16, 8, 2050, 140)]


@pytest.mark.parametrize("t,e,top,n,k", EXPERTS)
@pytest.mark.parametrize("gather", [True, False])
def test_experts(g, t, e, top, n, k, gather):
    gen = generator(t + e)
    r = g.route(uneven(gen, t, e, top, padded=e > 1), top)
    bounds = r.offsets.tolist()
    rows = t if gather else t * top
    ac, as_, a = whole(gen, rows, k, 1)
    wc, ws, w = whole(gen, n, k, 128, count=e)
    out, around = guarded((t * top, n))
    g.gemm_nt_f8_experts(g.F8Matrix(ac, as_, k, 1), g.F8Matrix(wc, ws, k, 128), r, gather=gather, out=out)
    if gather:
        a = a[r.rows.long().clamp(min=0) // top]
    for i in range(e):
        lo, hi = bounds[i: i + 2]
        assert torch.equal(out[lo:hi], product(a[lo:hi], w[i])), i
    assert (out[bounds[-1]:] == 0).all()
    assert all((x == 3).all() for x in around)


def whole_halves(gen, *shape):
    return torch.randint(-2, 3, shape, generator=gen, device="cuda").half()


@pytest.mark.parametrize("t,e,top,n,k", [(4099, 32, 4, 1408, 1030), (3000, 5, 2, 1410, 520), (700, 130, 3, 136, 264),
                                         (1500, 40, 2, 1030, 770), (9000, 8, 1, 2048, 1025), (300, 9, 2, 64, 3000),
                                         (16, 8, 2, 500, 700), (128, 1, 1, 260, 516)])
def test_experts_gradient(g, t, e, top, n, k):
    gen = generator(t + n)
    r = g.route(uneven(gen, t, e, top, padded=e > 1), top)
    bounds = r.offsets.tolist()
    dy, x = whole_halves(gen, t * top, n), whole_halves(gen, t, k)
    out, around = guarded((e, n, k))
    g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True), r, out=out)
    xs = x[r.rows.long().clamp(min=0) // top].double()
    for i in range(e):
        lo, hi = bounds[i: i + 2]
        want = product(dy[lo:hi].double().t().contiguous(), xs[lo:hi].t().contiguous())
        assert torch.equal(out[i], want), i
    assert all((v == 3).all() for v in around)


def test_two_streams_and_devices_memory(g):
    """The same products on two streams at once, operands and outputs dropped early."""
    gen = generator(3)
    m, n, k = 3000, 4096, 700
    ac, as_, a = whole(gen, m, k, 1)
    bc, bs, b = whole(gen, n, k, 128)
    want = product(a, b)
    x, w = g.F8Matrix(ac, as_, k, 1), g.F8Matrix(bc, bs, k, 128)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [g.gemm_nt_f8(x, w, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    assert all(torch.equal(c, want) for c in got)


def test_captured(g):
    """A layer of experts and its gradients captured once, replayed on other
    tokens with other experts, every replay against the calls themselves."""
    gen = generator(4)
    t, e, top, n, k = 4100, 16, 2, 1030, 300
    logits, x = uneven(gen, t, e, top), torch.randn(t, k, generator=gen, device="cuda").half()
    w = torch.randn(e, n, k, generator=gen, device="cuda").half() / 16
    w8, wt8 = g.quantize_f8(w, 128), g.quantize_f8(w, 128, transposed=True)
    dout = torch.randn(t, n, generator=gen, device="cuda").half()

    def step():
        r = g.route(logits, top, scale=2.0)
        y = g.gemm_nt_f8_experts(x, w8, r, gather=True)
        out = g.combine_experts(y, r)
        dy, dweights = g.combine_experts_backward(dout, y, r)
        dlogits = g.route_backward(logits, r, dweights)
        dx = g.combine_experts(g.gemm_nt_f8_experts(dy, wt8, r), r, weighted=False)
        dw = g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(dy, r), g.quantize_f8_experts(x, r, gather=True), r)
        return out, dlogits, dx, dw

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for _ in range(4):
        logits.copy_(uneven(gen, t, e, top))
        x.copy_(torch.randn(t, k, generator=gen, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


@pytest.mark.parametrize("t,e,top", [(40000, 8, 8), (20000, 130, 7), (2049, 1024, 1), (300000, 16, 1)])
def test_order_of_many(g, t, e, top):
    """The order of many tokens, by several workgroups and passes."""
    gen = generator(t)
    r = g.route(uneven(gen, t, e, top), top)
    flat = r.experts.reshape(-1).long()
    order = torch.where(flat < 0, e, flat).sort(stable=True)
    here = order.values < e
    assert torch.equal(r.rows, torch.where(here, order.indices, -1).int())
    places = torch.empty_like(r.rows)
    places[order.indices] = torch.where(here, torch.arange(t * top, device="cuda"), -1).int()
    assert torch.equal(r.places.reshape(-1), places)
    assert torch.equal(r.offsets, torch.searchsorted(order.values, torch.arange(e + 1, device="cuda")).int())


@pytest.mark.parametrize("t,e,top,scores", [(16, 512, 4, "softmax"), (16, 1024, 4, "sigmoid"), (2, 300, 32, "softmax"),
                                            (3, 1024, 32, "sigmoid"), (16, 700, 32, "softmax"), (17, 64, 4, "softmax")])
def test_few_as_many(g, t, e, top, scores):
    """A few tokens, which one launch routes, as the same among many."""
    gen = generator(e)
    x = torch.randn(600, e, generator=gen, device="cuda")
    x[1, 5:] = -torch.inf
    x[2, 3] = torch.nan
    few, many = g.route(x[:t].contiguous(), top, scores), g.route(x, top, scores)
    assert torch.equal(few.experts, many.experts[:t])
    assert torch.equal(few.weights.nan_to_num(-1), many.weights[:t].nan_to_num(-1))
    flat = few.experts.reshape(-1).long()
    order = torch.where(flat < 0, e, flat).sort(stable=True)
    assert torch.equal(few.rows, torch.where(order.values < e, order.indices, -1).int())
    assert torch.equal(few.offsets, torch.searchsorted(order.values, torch.arange(e + 1, device="cuda")).int())


def test_threads(g):
    """Products, routing and combination from four host threads at once, each on its
    own stream, with plans that differ from call to call."""
    import threading

    gen = generator(5)
    cases = []
    for m, n, k in ((1, 300, 2000), (70, 300, 200), (333, 1001, 4000), (1000, 2050, 300), (3001, 4096, 130)):
        ac, as_, a = whole(gen, m, k, 1)
        bc, bs, b = whole(gen, n, k, 128)
        cases.append((g.F8Matrix(ac, as_, k, 1), g.F8Matrix(bc, bs, k, 128), product(a, b)))
    logits = uneven(gen, 900, 40, 3)
    want = g.route(logits, 3)
    y = torch.randn(2700, 520, generator=gen, device="cuda").half()
    out = g.combine_experts(y, want)
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            torch.cuda.set_device(0)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for j in range(20):
                    a, b, c = cases[(i + j) % len(cases)]
                    got = g.gemm_nt_f8(a, b)
                    r = g.route(logits, 3)
                    mixed = g.combine_experts(y, r)
                    stream.synchronize()
                    assert torch.equal(got, c)
                    assert torch.equal(r.rows, want.rows) and torch.equal(r.weights.nan_to_num(-1), want.weights.nan_to_num(-1))
                    assert torch.equal(mixed, out)
        except BaseException as e:   # noqa: BLE001  (reported by the test's own thread)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors[0]


def test_graphs_share_a_workspace(g):
    """Two captured products that use one workspace in turn."""
    gen = generator(6)
    graphs, cus = [], g.gemm_f16_device_cus()
    sizes = [(300, 264, 2048), (333, 2050, 4000)]
    need = max(g.gemm_f16_nt_f8_plan(m, n, k, 128, True, cus).workspace_bytes for m, n, k in sizes)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    for m, n, k in sizes:
        x = torch.empty(m, k, dtype=torch.float16, device="cuda")
        bc, bs, b = whole(gen, n, k, 128)
        w, out = g.F8Matrix(bc, bs, k, 128), torch.empty(m, n, dtype=torch.float16, device="cuda")
        x.copy_(whole_halves(gen, m, k))
        g.gemm_nt_f8(x, w, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.gemm_nt_f8(x, w, out=out, workspace=ws)
        graphs.append((graph, x, b, out, w))
    for _ in range(3):
        for graph, x, *_ in graphs:
            x.copy_(whole_halves(gen, *x.shape))
            ws.random_()
            graph.replay()
        torch.cuda.synchronize()
        for _, x, b, out, _ in graphs:
            assert torch.equal(out, product(x.double(), b))


def test_routing_of_other_numbers(g):
    """A routing whose offsets and rows are no routing's: whatever is computed, nothing
    around the outputs changes."""
    gen = generator(7)
    t, e, top, n, k = 2500, 64, 2, 264, 200
    s = t * top
    ac, as_, _ = whole(gen, t, k, 1)
    wc, ws, _ = whole(gen, n, k, 128, count=e)
    y = torch.randn(s, n, generator=gen, device="cuda").half()
    x = torch.randn(t, k, generator=gen, device="cuda").half()
    for kind in range(4):
        offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        if kind == 0:      # every expert has all rows
            offsets[1::2] = s
        elif kind == 1:
            offsets.random_(-2 ** 31, 2 ** 31 - 1, generator=gen)
        elif kind == 2:
            offsets[:] = 2 ** 31 - 1
        else:
            offsets[:] = torch.arange(e, -1, -1, device="cuda") * 100
        any_ = torch.randint(-2 ** 31, 2 ** 31 - 1, (3, s), generator=gen, device="cuda").int()
        r = g.Routing(any_[0].view(t, top), torch.ones(t, top, device="cuda"), any_[1].contiguous(),
                      any_[2].view(t, top), offsets)
        out, around = guarded((s, n))
        g.gemm_nt_f8_experts(g.F8Matrix(ac, as_, k, 1), g.F8Matrix(wc, ws, k, 128), r, gather=True, out=out)
        dw, beyond = guarded((e, n, k))
        g.gemm_nt_f8_experts_grad(g.quantize_f8_experts(y, r), g.quantize_f8_experts(x, r, gather=True), r, out=dw)
        mixed, outside = guarded((t, n))
        g.combine_experts(y, r, out=mixed)
        g.combine_experts_backward(mixed, y, r)
        torch.cuda.synchronize()
        assert all((v == 3).all() for v in around + beyond + outside)


@pytest.mark.parametrize("e", [1, 2, 31, 32, 33, 63, 64, 65, 97, 127, 128, 129])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t", [17, 18, 263])
def test_two_tokens_a_wave(g, t, e, scores):
    """Tokens with ties, masks and without scores side by side in a wave: each has what
    it has by itself, bit for bit, and the plain form's choice."""
    rng = np.random.default_rng(t + e)
    x = np.round(rng.standard_normal((t, e)) * 3).astype(np.float32)     # many ties
    x[3], x[5], x[8, 1:], x[11] = 1.0, -np.inf, -np.inf, 88.0
    x[6, e - 1], x[9, 0] = np.nan, np.inf
    x[12] = 20.0                                                        # told apart by the lower halves
    x[12, e // 2] = np.nextafter(np.float32(20), np.float32(21))
    x[13, e // 3:] = -np.inf
    top = min(e, 32 if t == 18 else 7)
    bias = rng.standard_normal(e).astype(np.float32)
    bias[e // 2] = -np.inf
    dw = rng.standard_normal((t, top)).astype(np.float32)
    for b in (None, bias):
        on = None if b is None else torch.from_numpy(b).cuda()
        r = g.route(torch.from_numpy(x).cuda(), top, scores, on)
        want, weights = ref.route(x, top, scores, b)
        np.testing.assert_array_equal(r.experts.cpu().numpy(), want)
        w = r.weights.cpu().numpy().astype(np.float64)
        assert (np.isnan(w) == np.isnan(weights)).all()
        ok = ~np.isnan(weights)
        # one rounding to fp32, and sums of 64-bit scores in another order
        assert (np.abs(w - weights)[ok] <= np.abs(weights[ok]) * (2.0 ** -24 + 2.0 ** -40) + 2.0 ** -150).all()
        for at in range(0, min(t, 48), 16):
            part = g.route(torch.from_numpy(x[at:at + 16].copy()).cuda(), top, scores, on)
            assert torch.equal(part.experts, r.experts[at:at + 16])
            assert torch.equal(part.weights.nan_to_num(-1), r.weights[at:at + 16].nan_to_num(-1))
        got = g.route_backward(torch.from_numpy(x).cuda(), r, torch.from_numpy(dw).cuda()).cpu().numpy().astype(np.float64)
        for i in range(t):
            if not ok[i].all():
                assert np.isnan(got[i]).all()
                continue
            one = slice(i, i + 1)
            d = ref.route_gradient(x[one].astype(np.float64), want[one], dw[one].astype(np.float64), scores, True, 1.0)
            # one rounding; the 64-bit sums of at most top + E terms, 4 times dw in size
            size = np.abs(dw[i]).max() * 4
            assert (np.abs(got[one] - d) <= np.abs(d) * 2.0 ** -24 + 2.0 ** -150 + size * (top + e + 40) * 2.0 ** -52).all()
