"""How the mixture-of-experts operators are called: graphs, streams and threads, arguments of every form, refusals, and
offsets past 32 bits."""
import os
import subprocess
import sys
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe8_reference as R  # noqa: E402

BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
D = torch.float64


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, typical=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * typical).to(dtype)


def _bits(t):
    """Tensors, and tuples of them, as bytes."""
    if isinstance(t, torch.Tensor):
        return [t.contiguous().view(torch.uint8)]
    return [b for x in t for b in _bits(x)]


def _same(a, b):
    a, b = _bits(a), _bits(b)
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


class Layer:
    """A layer's weights and one batch; run() is its forward and backward pass."""

    def __init__(self, seed, T=40, X=5, k=2, width=160, hidden=288):
        Q, g = _Q(), _gen(seed)
        self.X, self.k, self.T = X, k, T
        self.up = Q.pack_f8(*Q.quantize_weight_f8(_randn(g, (X, 2 * hidden, width), width ** -0.5)))
        self.down = Q.pack_f8(*Q.quantize_weight_f8(_randn(g, (X, width, hidden), hidden ** -0.5)))
        self.x, self.dy = _randn(g, (T, width)), _randn(g, (T, width))
        self.ids = torch.randint(0, X, (T, k), generator=g, device="cuda")
        self.w = torch.rand((T, k), generator=g, device="cuda")

    def fill(self, seed):
        g = _gen(seed)
        for t in (self.x, self.dy):
            t.copy_(_randn(g, t.shape))
        self.ids.copy_(torch.randint(0, self.X, (self.T, self.k), generator=g, device="cuda"))
        self.w.copy_(torch.rand((self.T, self.k), generator=g, device="cuda"))

    def run(self):
        Q = _Q()
        order = Q.expert_order(self.ids, self.X)
        x, s = Q.dispatch_tokens(self.x, order, f8=True)
        raw = Q.grouped_linear_f8(x, s, self.up, order.counts)
        h, hs = Q.quantize_f8(raw, act="swiglu")
        out = Q.grouped_linear_f8(h, hs, self.down, order.counts)
        y = Q.combine_tokens(out, order, self.w)
        dout, dw = Q.combine_tokens_backward(self.dy, out, order, self.w)
        draw = Q.quantize_f8_backward(Q.grouped_linear_f8_backward(dout, self.down, order.counts), raw)
        dx = Q.dispatch_tokens_backward(Q.grouped_linear_f8_backward(draw, self.up, order.counts), order)
        return y, dw, dx, order.counts, order.rows, order.source


def _split(seed, back=False):
    """A product that splits its sum, so that it needs a workspace."""
    Q, g = _Q(), _gen(seed)
    N, K = (4746, 192) if back else (73, 6592)
    w, ws = R.weights(g, (N, K))
    pw = Q.pack_f8(w, ws)
    if back:
        dy = _randn(g, (17, N))
        assert Q.f8_backward_workspace_bytes(17, N, K) > 0
        return lambda: Q.linear_f8_backward(dy, pw)
    x, xs = R.activations(g, 17, K)
    assert Q.f8_workspace_bytes(17, N, K) > 0
    return lambda: Q.linear_f8(x, xs, pw)


# ---- graphs, streams, threads ----------------------------------------------------------

@pytest.mark.parametrize("T", [3, 40, 5000])
def test_a_captured_layer(T):
    """The whole layer in one graph: every replay, on new inputs and with eager work between, equals the eager result."""
    layer = Layer(T, T=T)
    layer.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = layer.run()
    for seed in range(4):
        layer.fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert _same(got, layer.run())
        torch.randn((512, 512), device="cuda").mm(torch.randn((512, 512), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert _same(got, outs)


def test_two_graphs_share_no_workspace():
    calls = [_split(1), _split(2), _split(3, True), _split(4, True)]
    refs = [f() for f in calls]
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for o in outs:
            o.fill_(0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert _same(outs, refs)


def test_streams():
    """Inputs made on one stream, used on another that waits for it."""
    layers = [Layer(i) for i in range(3)]
    refs = [layer.run() for layer in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(4):
        got = []
        for s, layer in zip(streams, layers):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.append(layer.run())
        torch.cuda.synchronize()
        assert all(_same(a, b) for a, b in zip(got, refs))


def test_threads():
    calls = [_split(i, i % 2 == 1) for i in range(4)]
    refs = [f() for f in calls]
    torch.cuda.synchronize()
    bad = []

    def work(f, ref):
        for _ in range(20):
            if not _same(f(), ref):
                bad.append(f)
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, refs)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


_CAPTURE_FIRST = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import bit_weight_only_offline_amd as Q
from test_gpu_moe8_calls import Layer, _same
layer = Layer(1, T=700)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):        # the first calls of this process, inside the capture
    outs = layer.run()
for _ in range(3):
    graph.replay()
    torch.cuda.synchronize()
    assert _same(outs, layer.run())
print("capture-first ok", flush=True)
"""


def test_first_calls_inside_a_capture():
    """The kernels' dynamic-LDS limits are raised inside a graph capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CAPTURE_FIRST, root], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0 and "capture-first ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def test_repeated_calls_give_the_same_bits():
    layer = Layer(7, T=3000, X=60, k=6)
    first = layer.run()
    for _ in range(3):
        assert _same(layer.run(), first)


# ---- arguments -------------------------------------------------------------------------

def test_views_of_any_start_and_stride():
    Q, g = _Q(), _gen(1)
    big = _randn(g, (40, 2, 333))
    x = big[3:23, 1, 5:325]                                   # rows of 320 at odd addresses, strides of 666
    codes, scales = Q.quantize_f8(x)
    assert _same((codes, scales), Q.quantize_f8(x.contiguous().clone()))
    assert torch.equal(Q.dequantize_f8(codes.t().contiguous().t(), scales.t().contiguous().t()), Q.dequantize_f8(codes, scales))
    w, ws = R.weights(g, (200, 320))
    pw = Q.pack_f8(w.t().contiguous().t(), ws.t().contiguous().t())
    assert _same(Q.unpack_f8(pw), (w, ws))
    y = Q.linear_f8(codes, scales, pw)
    wide = torch.empty((20, 640), dtype=F8, device="cuda")
    wide.view(torch.uint8)[:, 7:327] = codes.view(torch.uint8)
    assert torch.equal(Q.linear_f8(wide[:, 7:327], scales[:, None].expand(20, 2, 3)[:, 1], pw), y)
    bias = _randn(g, (400,))
    assert torch.equal(Q.linear_f8(codes, scales, pw, bias=bias[::2]), Q.linear_f8(codes, scales, pw, bias=bias[::2].contiguous()))
    dy = _randn(g, (20, 401))[:, 1:201]
    assert torch.equal(Q.linear_f8_backward(dy, pw), Q.linear_f8_backward(dy.contiguous().clone(), pw))

    ids = torch.randint(0, 6, (20, 6), generator=g, device="cuda")[:, ::2]
    order, plain = Q.expert_order(ids, 6), Q.expert_order(ids.contiguous(), 6)
    assert _same((order.counts, order.rows, order.source), (plain.counts, plain.rows, plain.source))
    assert torch.equal(Q.dispatch_tokens(x, order), x[order.source.long() // 3])
    v = _randn(g, (20 * 60 + 1,))[1:].reshape(60, 20)         # rows at odd addresses
    weights = torch.rand((3, 20), generator=g, device="cuda").t()
    ref = Q.combine_tokens(v.clone(), order, weights.contiguous())
    assert torch.equal(Q.combine_tokens(v, order, weights), ref)
    dout = _randn(g, (20, 23))[:, 3:]
    assert _same(Q.combine_tokens_backward(dout, v, order, weights),
                 Q.combine_tokens_backward(dout.contiguous().clone(), v.clone(), order, weights.contiguous()))


def test_leading_shapes():
    """Tokens of any leading shape, and a single token without one."""
    Q, g = _Q(), _gen(2)
    x = _randn(g, (2, 3, 4, 160))
    codes, scales = Q.quantize_f8(x)
    w, ws = R.weights(g, (48, 160))
    pw = Q.pack_f8(w, ws)
    y = Q.linear_f8(codes, scales, pw)
    assert codes.shape == x.shape and scales.shape == (2, 3, 4, 2) and y.shape == (2, 3, 4, 48)
    assert torch.equal(y.reshape(24, 48), Q.linear_f8(codes.reshape(24, 160), scales.reshape(24, 2), pw))
    assert Q.linear_f8_backward(y, pw).shape == x.shape
    one = Q.linear_f8(*Q.quantize_f8(x[0, 0, 0]), pw)
    assert one.shape == (48,)
    ids = torch.randint(0, 5, (2, 3, 4, 2), generator=g, device="cuda")
    order = Q.expert_order(ids, 5)
    rows = Q.dispatch_tokens(x, order)
    weights = torch.rand(ids.shape, generator=g, device="cuda")
    out = Q.combine_tokens(rows, order, weights)
    assert out.shape == x.shape and rows.shape == (48, 160)
    dy, dw = Q.combine_tokens_backward(out, rows, order, weights)
    assert dy.shape == rows.shape and dw.shape == weights.shape
    single = Q.expert_order(ids[0, 0, 0], 5)
    assert Q.combine_tokens(Q.dispatch_tokens(x[0, 0, 0], single), single).shape == (160,)


def test_no_rows():
    Q, g = _Q(), _gen(3)
    w, ws = R.weights(g, (3, 40, 96))
    pw, experts = Q.pack_f8(w[0], ws[0]), Q.pack_f8(w, ws)
    codes, scales = Q.quantize_f8(torch.empty((0, 96), device="cuda"))
    assert codes.shape == (0, 96) and scales.shape == (0, 1)
    assert Q.dequantize_f8(codes, scales).shape == (0, 96)
    assert Q.linear_f8(codes, scales, pw).shape == (0, 40) and Q.linear_f8_backward(torch.empty((0, 40), dtype=BF, device="cuda"), pw).shape == (0, 96)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert Q.grouped_linear_f8(codes, scales, experts, none).shape == (0, 40)
    assert Q.quantize_f8_backward(torch.empty((0, 32), dtype=BF, device="cuda"), torch.empty((0, 64), dtype=BF, device="cuda")).shape == (0, 64)


def test_buffers_of_the_caller():
    """Outputs and workspaces that the caller gives are used; a workspace is not written past its need."""
    Q, g = _Q(), _gen(4)
    w, ws = R.weights(g, (73, 6592))
    pw = Q.pack_f8(w, ws)
    x, xs = R.activations(g, 17, 6592)
    ref = Q.linear_f8(x, xs, pw)
    need = Q.f8_workspace_bytes(17, 73, 6592)
    space = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.empty((17, 73), dtype=BF, device="cuda")
    assert Q.linear_f8(x, xs, pw, out=out, workspace=space) is out and torch.equal(out, ref)
    assert bool((space[need:] == 0xAB).all())
    ids = torch.randint(0, 60, (3000, 4), generator=g, device="cuda")
    need = Q.expert_order_workspace_bytes(12000, 60)
    space = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    a, b = Q.expert_order(ids, 60, workspace=space), Q.expert_order(ids, 60)
    assert _same((a.counts, a.rows, a.source), (b.counts, b.rows, b.source)) and bool((space[need:] == 0xAB).all())


def test_next_to_the_weight_only_product():
    """The order's counts and rows are what grouped_linear() takes too."""
    Q, g = _Q(), _gen(5)
    X, k, T, N, K = 4, 2, 30, 64, 128
    w = torch.randn((X, N, K), generator=g, device="cuda") * 0.1
    parts = [Q.quantize("int8", w[e], 64) for e in range(X)]
    pe = Q.pack_experts("int8", N, K, 64, parts)
    x = _randn(g, (T, K))
    ids = torch.randint(0, X, (T, k), generator=g, device="cuda")
    weights = torch.rand((T, k), generator=g, device="cuda")
    order = Q.expert_order(ids, X)
    y = Q.combine_tokens(Q.grouped_linear(Q.dispatch_tokens(x, order), pe, order.counts, out_dtype=F32), order, weights)
    dense = torch.stack([c.to(D) * s.to(D).repeat_interleave(64, 1) for c, s, _ in parts])
    ref = (torch.bmm(dense[ids.reshape(-1)], x.to(D).repeat_interleave(k, 0)[:, :, None]).reshape(T, k, N) * weights.to(D)[..., None]).sum(1)
    # float32 sums of K products of bf16 and of eight-bit codes under bf16 scales, and of k rows
    assert float((y.to(D) - ref).abs().max()) <= (K + k + 8) * 2.0 ** -24 * float(ref.abs().max()) * 40


# ---- refusals --------------------------------------------------------------------------

def test_refusals():
    Q, g = _Q(), _gen(6)
    err = Q.QLinearError
    x = _randn(g, (8, 160))
    codes, scales = Q.quantize_f8(x)
    w, ws = R.weights(g, (3, 48, 160))
    pw, experts = Q.pack_f8(w[0], ws[0]), Q.pack_f8(w, ws)
    counts = torch.tensor([3, 3, 2], dtype=torch.int32, device="cuda")
    ids = torch.randint(0, 3, (8, 2), generator=g, device="cuda")
    order = Q.expert_order(ids, 3)
    rows = Q.dispatch_tokens(x, order)
    weights = torch.rand((8, 2), device="cuda")
    dy = _randn(g, (8, 48))
    grad = lambda t: t.float().requires_grad_()  # noqa: E731
    E = torch.empty
    for name, call in {
        "half": lambda: Q.quantize_f8(x.half()), "grad": lambda: Q.quantize_f8(grad(x)), "K": lambda: Q.quantize_f8(x[:, :40]),
        "act": lambda: Q.quantize_f8(x, act="gelu"), "odd pair": lambda: Q.quantize_f8(x[:, :96], act="swiglu"),
        "scalar": lambda: Q.quantize_f8(x[0, 0]), "cpu": lambda: Q.quantize_f8(x.cpu()),
        "raw": lambda: Q.quantize_f8_backward(x, x), "raw type": lambda: Q.quantize_f8_backward(x, torch.cat([x, x], 1).float()),
        "back act": lambda: Q.quantize_f8_backward(x, torch.cat([x, x], 1), act=None),
        "codes": lambda: Q.dequantize_f8(codes.view(torch.uint8), scales), "few scales": lambda: Q.dequantize_f8(codes, scales[:, :1]),
        "out type": lambda: Q.dequantize_f8(codes, scales, torch.float16),
        "weight": lambda: Q.quantize_weight_f8(x[0]), "weight K": lambda: Q.quantize_weight_f8(x[:, :40]),
        "weight scales": lambda: Q.pack_f8(w, ws[:, :, :1]), "plain scales": lambda: Q.pack_f8(w[0], ws), "pack K": lambda: Q.pack_f8(w[0, :, :40], ws[0, :, :1]),
        "scales type": lambda: Q.pack_f8(w, ws.double()), "unpack": lambda: Q.unpack_f8(w),
        "not packed": lambda: Q.linear_f8(codes, scales, w), "experts": lambda: Q.linear_f8(codes, scales, experts),
        "no experts": lambda: Q.grouped_linear_f8(codes, scales, pw, counts), "inputs": lambda: Q.linear_f8(codes[:, :128], scales[:, :1], pw),
        "e5m2": lambda: Q.linear_f8(codes.float().to(torch.float8_e5m2), scales, pw), "scales shape": lambda: Q.linear_f8(codes, scales.t(), pw),
        "bias": lambda: Q.linear_f8(codes, scales, pw, bias=dy[0, :40]), "bias type": lambda: Q.linear_f8(codes, scales, pw, bias=dy[0].float()),
        "product type": lambda: Q.linear_f8(codes, scales, pw, out_dtype=torch.float16),
        "out shape": lambda: Q.linear_f8(codes, scales, pw, out=E((8, 40), dtype=BF, device="cuda")),
        "out strides": lambda: Q.linear_f8(codes, scales, pw, out=E((48, 8), dtype=BF, device="cuda").t()),
        "out grad": lambda: Q.linear_f8(codes, scales, pw, out_dtype=F32, out=E((8, 48), device="cuda", requires_grad=True)),
        "counts type": lambda: Q.grouped_linear_f8(codes, scales, experts, counts.long()),
        "counts shape": lambda: Q.grouped_linear_f8(codes, scales, experts, counts[:2]), "counts cpu": lambda: Q.grouped_linear_f8(codes, scales, experts, counts.cpu()),
        "grouped rows": lambda: Q.grouped_linear_f8(codes[None], scales[None], experts, counts),
        "dy": lambda: Q.linear_f8_backward(x, pw), "dy type": lambda: Q.linear_f8_backward(dy.float(), pw), "dy grad": lambda: Q.linear_f8_backward(dy.clone().requires_grad_(), pw),
        "grouped dy": lambda: Q.grouped_linear_f8_backward(dy[None], experts, counts), "back experts": lambda: Q.linear_f8_backward(dy, experts),
        "ids": lambda: Q.expert_order(ids.float(), 3), "no ids": lambda: Q.expert_order(ids[:, :0], 3), "no experts at all": lambda: Q.expert_order(ids, 0),
        "too many": lambda: Q.expert_order(ids, 1025), "0-dim": lambda: Q.expert_order(ids[0, 0], 3),
        "tokens": lambda: Q.dispatch_tokens(x[:7], order), "token type": lambda: Q.dispatch_tokens(x.half(), order), "order": lambda: Q.dispatch_tokens(x, order.rows),
        "f8 width": lambda: Q.dispatch_tokens(x[:, :40].contiguous(), order, f8=True), "f8 out": lambda: Q.dispatch_tokens(x, order, f8=True, out=rows),
        "rows type": lambda: Q.dispatch_tokens(x, Q.ExpertOrder(order.counts, order.rows.long(), order.source)),
        "rows strides": lambda: Q.dispatch_tokens(x, Q.ExpertOrder(order.counts, order.rows.t().contiguous().t(), order.source)),
        "dispatch out": lambda: Q.dispatch_tokens(x, order, out=rows[:8]),
        "sorted": lambda: Q.combine_tokens(rows[:9], order, weights), "weights": lambda: Q.combine_tokens(rows, order, weights[:, :1]),
        "weights type": lambda: Q.combine_tokens(rows, order, weights.bfloat16()), "sorted grad": lambda: Q.combine_tokens(grad(rows), order, weights),
        "dout": lambda: Q.combine_tokens_backward(x[:7], rows, order, weights), "dout type": lambda: Q.combine_tokens_backward(x.float(), rows, order, weights),
        "no weights": lambda: Q.combine_tokens_backward(x, rows, order, None),
    }.items():
        with pytest.raises(err):
            call()
            print("not refused:", name, flush=True)
    y = Q.linear_f8(codes, scales, pw)
    for space in (E(16, dtype=torch.uint8, device="cuda"), E((1,), dtype=torch.uint8, device="cuda").expand(1 << 24), E(1 << 24, dtype=torch.uint8)):
        bw, bs = R.weights(g, (73, 6592))
        big = Q.pack_f8(bw, bs)
        bx, bxs = R.activations(g, 17, 6592)
        with pytest.raises(err):
            Q.linear_f8(bx, bxs, big, workspace=space)
        with pytest.raises(err):
            Q.expert_order(torch.zeros((9000, 2), dtype=torch.int64, device="cuda"), 3, workspace=space)
    torch.cuda.synchronize()
    assert y.shape == (8, 48)


def test_rows_of_no_order():
    """Rows outside the slots, which expert_order() never gives, are skipped on the device."""
    Q, g = _Q(), _gen(7)
    x = _randn(g, (4, 64))
    rows = torch.tensor([[0, 7], [-1, 8], [2 ** 31 - 1, 3], [-2 ** 31, 1]], dtype=torch.int32, device="cuda")
    order = Q.ExpertOrder(torch.zeros(2, dtype=torch.int32, device="cuda"), rows, rows.reshape(-1))
    out = torch.full((8, 64), 7.0, dtype=BF, device="cuda")
    Q.dispatch_tokens(x, order, out=out)
    for row, t in ((0, 0), (7, 0), (3, 2), (1, 3)):
        assert torch.equal(out[row], x[t])
    assert bool((out[[2, 4, 5, 6]] == 7.0).all())
    assert torch.equal(Q.combine_tokens(out, order), torch.stack([(x[0].float() * 2).bfloat16(), torch.zeros_like(x[0]), x[2], x[3]]))
    dy, dw = Q.combine_tokens_backward(x, out, order, torch.ones((4, 2), device="cuda"), out=torch.full_like(out, 7.0))
    assert bool((dy[[2, 4, 5, 6]] == 7.0).all()) and dw[1].tolist() == [0.0, 0.0]


# ---- offsets past 32 bits --------------------------------------------------------------

def test_weights_past_four_gigabytes():
    """Experts' codes that pass 2^32 bytes: the last expert's products, forward and backward."""
    Q, g = _Q(), _gen(8)
    X, N, K, T = 40, 8192, 14336, 20
    codes = torch.zeros((X, N, K), dtype=F8, device="cuda")
    scales = torch.ones((X, N // 128, K // 128), device="cuda")
    last, s = R.weights(g, (N, K), True)
    codes[X - 1], scales[X - 1] = last, s
    pw = Q.pack_f8(codes, scales)
    del codes
    counts = torch.zeros(X, dtype=torch.int32, device="cuda")
    counts[X - 1] = T
    x, xs = R.activations(g, T, K, True)
    y = Q.grouped_linear_f8(x, xs, pw, counts, out_dtype=F32)
    dense = R.dense_weight(last, s)
    assert torch.equal(y.to(D), (x.to(D) * R.spread_rows(xs, K)) @ dense.t())
    dy = torch.randint(-3, 4, (T, N), generator=g, device="cuda").bfloat16()
    assert torch.equal(Q.grouped_linear_f8_backward(dy, pw, counts), (dy.to(D) @ dense).float().bfloat16())


def test_rows_past_four_gigabytes():
    """Rows in expert order, and outputs, whose element offsets pass 2^32."""
    Q, g = _Q(), _gen(9)
    T, k, X, width = 70000, 8, 16, 8192
    ids = torch.randint(0, X, (T, k), generator=g, device="cuda")
    order = Q.expert_order(ids, X)
    x = _randn(g, (T, width))
    rows = Q.dispatch_tokens(x, order)
    assert rows.numel() > 1 << 32
    some = torch.tensor([0, 1, T * k // 2, T * k - 2, T * k - 1], device="cuda")
    assert torch.equal(rows[some], x[order.source[some].long() // k])
    weights = torch.rand((T, k), generator=g, device="cuda")
    out = Q.combine_tokens(rows, order, weights)
    for t in (0, T // 2, T - 1):
        ref = x[t].to(D) * weights[t].to(D).sum()
        assert float((out[t].to(D) - ref).abs().max()) <= (2.0 ** -8 + 20 * 2.0 ** -24) * float(ref.abs().max())
    dy, dw = Q.combine_tokens_backward(x, rows, order, weights, out=rows)
    slot = order.source[some].long()
    assert torch.equal(dy[some], (weights.reshape(-1)[slot][:, None] * x[slot // k].float()).bfloat16())
    del rows, dy
    M, N, K = 300000, 16384, 32
    w, ws = R.weights(g, (N, K), True)
    a, s = R.activations(g, 64, K, True)
    y = Q.linear_f8(a.repeat(M // 64 + 1, 1)[:M], s.repeat(M // 64 + 1, 1)[:M], Q.pack_f8(w, ws))
    assert y.numel() > 1 << 32
    ref = ((a.to(D) * R.spread_rows(s, K)) @ R.dense_weight(w, ws).t()).float().bfloat16()
    assert torch.equal(y[M - 32:], ref[[(m % 64) for m in range(M - 32, M)]])
