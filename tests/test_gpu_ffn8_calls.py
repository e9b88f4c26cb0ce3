"""How the 8-bit operators are called: workspaces in graphs and threads, and what their
arguments may be."""
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)


def _bf(g, shape):
    return torch.randn(shape, generator=g, device="cuda").bfloat16()


def _scales(g, n, typical=1e-3):
    return torch.exp(torch.randn((n,), generator=g, device="cuda")) * typical


# ---- workspaces --------------------------------------------------------------------------

def _call(kind, seed, M):
    """(function of no arguments, its main input, bytes of its workspace), at sizes that use one."""
    Q, g = _Q(), _gen(seed)
    if kind in ("linear", "linear back"):
        N, K = 1024, 14336
        pw = Q.pack_channel(_codes(g, N, K), _scales(g, N))
        if kind == "linear":
            x, xs = _codes(g, M, K), _scales(g, M)
            return (lambda: (Q.linear_i8(x, xs, pw),)), x, Q.i8_workspace_bytes(M, N, K)
        dy = _bf(g, (M, N))
        return (lambda: (Q.linear_i8_backward(dy, pw),)), dy, Q.i8_backward_workspace_bytes(M, N, K)
    if kind in ("gated", "gated back"):
        N, K = (320, 14144) if kind == "gated" else (1000, 1056)
        pw = Q.pack_gated(_codes(g, N, K), _scales(g, N, 1e-6), _codes(g, N, K), _scales(g, N, 1e-6))
        if kind == "gated":
            x, xs = _codes(g, M, K), _scales(g, M, 1.0)
            return (lambda: Q.gated_i8(x, xs, pw, keep_raw=True)), x, Q.i8_workspace_bytes(M, N, K, True)
        dh, raw = _bf(g, (M, N)), _bf(g, (M, 2 * N))
        return (lambda: Q.gated_i8_backward(dh, raw, pw)), dh, Q.i8_backward_workspace_bytes(M, N, K, True)
    C = 512
    dx, r, y, w = _bf(g, (M, C)), _bf(g, (M, C)), _bf(g, (M, C)), torch.rand((3, C), generator=g, device="cuda")
    return ((lambda: Q.block_norm_backward(dx, None, r, y, post_weight=w[0], pre_weight=w[1], gate=w[2])), dx,
            Q.block_norm_backward_workspace_bytes(M, C, 1))


KINDS = ["linear", "gated", "linear back", "gated back", "norm back"]


@pytest.mark.parametrize("kind", KINDS)
def test_a_graph_keeps_its_workspace(kind):
    """Warmed up and captured on a stream, then a larger call on that stream and new tensors of
    the first workspace's size: replays give the right results and leave those tensors alone."""
    f, x, need = _call(kind, 1, 70)
    big, _, more = _call(kind, 2, 190)
    assert 0 < need < more
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            f()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = f()
    with torch.cuda.stream(side):
        big()
        others = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in (need, need, more, need // 2 + 1) * 3]
    side.synchronize()
    g = _gen(9)
    for i in range(4):
        x.copy_(torch.randint(-100, 100, x.shape, generator=g, device="cuda").to(x.dtype))
        torch.cuda.synchronize()
        print(kind, "replay", i, flush=True)
        graph.replay()
        torch.cuda.synchronize()
        want = f()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert all(bool((t == 0x5A).all()) for t in others), i


@pytest.mark.parametrize("kind", KINDS)
def test_graphs_of_one_stream_replay_on_two(kind):
    """Two graphs captured one after the other and replayed at the same time, next to eager
    calls on a third stream."""
    calls = [_call(kind, s, 70) for s in (3, 4, 5)]
    want = [tuple(t.clone() for t in f()) for f, _, _ in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f, _, _ in calls[:2]:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(f())
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                for _ in range(3):
                    graph.replay()
        with torch.cuda.stream(streams[2]):
            for _ in range(3):
                eager = calls[2][0]()
        torch.cuda.synchronize()
        for got, w in zip((*outs, eager), want):
            assert all(torch.equal(a, b) for a, b in zip(got, w)), i


@pytest.mark.parametrize("kind", KINDS)
def test_threads_on_one_stream(kind):
    """Threads that queue their calls on one stream, each with inputs of its own: the launches of
    one call may fall between those of another."""
    calls = [_call(kind, 10 + s, 70 + 10 * s) for s in range(3)]
    want = [tuple(t.clone() for t in f()) for f, _, _ in calls]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        for i in range(60):
            got = calls[k][0]()
            if i % 6 == 0 and not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                wrong.append((k, i))
    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong, wrong


def _no_workspaces(need):
    """Tensors of at least `need` elements that are no workspace of `need` bytes."""
    room = torch.zeros(2 * need + 64, dtype=torch.uint8, device="cuda")
    return [room[:1].expand(need), room[:2 * need].view(need, 2)[:, 0], room[:2 * need:2], room[:need - 1],
            torch.zeros(need, dtype=torch.uint8), bytearray(need), need]


@pytest.mark.parametrize("kind", KINDS)
def test_workspaces_that_are_none(kind):
    """Expanded and strided views, on the CPU, too small, no tensor: refused before anything is
    queued.  A view of a larger tensor, and of another type, are workspaces."""
    Q, g, M = _Q(), _gen(1), 70
    if kind == "linear":
        pw, x, xs = Q.pack_channel(_codes(g, 1024, 14336), _scales(g, 1024)), _codes(g, M, 14336), _scales(g, M)
        need, f = Q.i8_workspace_bytes(M, 1024, 14336), lambda w: Q.linear_i8(x, xs, pw, workspace=w)
    elif kind == "gated":
        pw = Q.pack_gated(_codes(g, 320, 14144), _scales(g, 320), _codes(g, 320, 14144), _scales(g, 320))
        x, xs = _codes(g, M, 14144), _scales(g, M)
        need, f = Q.i8_workspace_bytes(M, 320, 14144, True), lambda w: Q.gated_i8(x, xs, pw, workspace=w)
    elif kind == "linear back":
        pw, dy = Q.pack_channel(_codes(g, 64, 96), _scales(g, 64)), _bf(g, (M, 64))
        need, f = Q.i8_backward_workspace_bytes(M, 64, 96), lambda w: Q.linear_i8_backward(dy, pw, workspace=w)
    elif kind == "gated back":
        pw = Q.pack_gated(_codes(g, 64, 96), _scales(g, 64), _codes(g, 64, 96), _scales(g, 64))
        dy, raw = _bf(g, (M, 64)), _bf(g, (M, 128))
        need, f = Q.i8_backward_workspace_bytes(M, 64, 96, True), lambda w: Q.gated_i8_backward(dy, raw, pw, workspace=w)[0]
    else:
        r, w0 = _bf(g, (M, 64)), torch.ones(64, device="cuda")
        need = Q.block_norm_backward_workspace_bytes(M, 64, 0)
        f = lambda w: Q.block_norm_backward(r, None, r, pre_weight=w0, workspace=w)[0]  # noqa: E731
    assert need > 0
    for i, bad in enumerate(_no_workspaces(need)):
        with pytest.raises(Q.QLinearError):
            f(bad)
            pytest.fail(f"workspace {i} was taken")
    want = f(None)
    room = torch.full((need + 512,), 7, dtype=torch.uint8, device="cuda")
    assert torch.equal(f(room[256:256 + need]), want)
    assert bool((room[:256] == 7).all()) and bool((room[256 + need:] == 7).all())
    assert torch.equal(f(torch.zeros((need + 7) // 8, dtype=torch.float64, device="cuda")), want)


def test_workspaces_that_are_none_of_the_weight_only_products():
    Q, g = _Q(), _gen(2)
    N, K, G, M = 1024, 2048, 128, 64
    codes, s, _ = Q.quantize("int4", torch.randn((N, K), generator=g, device="cuda"), G)
    pw = Q.pack("int4", N, K, G, codes, s, None)
    x = _bf(g, (M, K))
    calls = [(Q.workspace_bytes("int4", M, N, K, G, None, (12, 4)), lambda w: Q.linear(x, pw, schedule=(12, 4), workspace=w)),
             (Q.a8_workspace_bytes("int4", M, N, K, G), lambda w: Q.linear_a8(x, pw, workspace=w))]
    for need, f in calls:
        assert need > 0
        want = f(None)
        for i, bad in enumerate(_no_workspaces(need)):
            with pytest.raises(Q.QLinearError):
                f(bad)
                pytest.fail(f"workspace {i} was taken")
        assert torch.equal(f(torch.zeros(need, dtype=torch.uint8, device="cuda")), want)


# ---- outputs -----------------------------------------------------------------------------

def test_outputs_that_are_none():
    """Outputs that require grad (a leaf, or what autograd has a history of) and what is no tensor
    are refused by every operator that takes one."""
    Q, g, M, N, K = _Q(), _gen(3), 5, 32, 64
    w, s = _codes(g, N, K), _scales(g, N)
    cw, gw = Q.pack_channel(w, s), Q.pack_gated(w, s, w, s)
    x, xs, dy, raw = _codes(g, M, K), _scales(g, M), _bf(g, (M, N)), _bf(g, (M, 2 * N))
    r, one = _bf(g, (M, K)), torch.ones(K, device="cuda")
    calls = [(N, lambda o: Q.linear_i8(x, xs, cw, out=o)), (N, lambda o: Q.gated_i8(x, xs, gw, out=o)),
             (2 * N, lambda o: Q.gated_i8(x, xs, gw, raw=o)), (K, lambda o: Q.linear_i8_backward(dy, cw, out=o)),
             (K, lambda o: Q.gated_i8_backward(dy, raw, gw, out=o)),
             (2 * N, lambda o: Q.gated_i8_backward(dy, raw, gw, draw=o)),
             (K, lambda o: Q.block_norm(r, pre_weight=one, residual_out=o))]
    for i, (width, f) in enumerate(calls):
        good = torch.zeros((M, width), dtype=torch.bfloat16, device="cuda")
        f(good)
        leaf = torch.zeros((M, width), dtype=torch.bfloat16, device="cuda", requires_grad=True)
        for bad in (leaf, leaf * 2, good.tolist(), 7):
            with pytest.raises(Q.QLinearError):
                f(bad)
                pytest.fail(f"output {i} was taken")
        assert bool((leaf == 0).all())


# ---- scales ------------------------------------------------------------------------------

@pytest.mark.parametrize("gated", [False, True])
def test_scales_have_the_shape_of_the_tokens(gated):
    """Scales of the tokens' shape or in a row, with dimensions of one anywhere; those of another
    shape with as many values belong to other tokens."""
    Q, g, N, K = _Q(), _gen(5), 48, 64
    w, s = _codes(g, N, K), _scales(g, N)
    pw = Q.pack_gated(w, s, w, s) if gated else Q.pack_channel(w, s)
    f = Q.gated_i8 if gated else Q.linear_i8
    x, xs = _codes(g, 6, K), _scales(g, 6, 1.0)
    want = f(x, xs, pw)
    shaped = x.view(2, 3, K)
    for good in (xs.view(2, 3), xs.view(2, 3, 1), xs, xs.view(2, 3).t().contiguous().t(), xs.view(1, 6), xs.view(6, 1),
                 xs.view(2, 1, 3)):
        assert torch.equal(f(shaped, good, pw), want.view(2, 3, N))
    assert torch.equal(f(x, xs[:, None], pw), want)
    assert torch.equal(f(x[0], xs[0], pw), want[0]) and torch.equal(f(x[0], xs[:1], pw), want[0])
    assert torch.equal(f(x[:1], xs[0], pw), want[:1]) and f(x[:0], xs[:0], pw).shape == (0, N)
    assert f(x[:0].view(2, 0, K), xs[:0], pw).shape == (2, 0, N)
    for bad in (xs.view(3, 2), xs.view(3, 2, 1), xs.view(1, 3, 2), xs[:5], xs[:1], xs[0], xs.view(2, 3)[:, :2]):
        with pytest.raises(Q.QLinearError):
            f(shaped, bad, pw)
            pytest.fail(f"scales {tuple(bad.shape)} were taken")


# ---- the chain ---------------------------------------------------------------------------

@pytest.mark.parametrize("lead", [(), (1,), (7,), (2, 3), (2, 1, 4), (0,), (2, 0)])
def test_activations_of_any_shape_through_a_layer(lead):
    """norm -> gated -> quantisation -> linear -> norm for tokens of any leading shape, and from
    views: what the same tokens give in a row."""
    Q, g, C, N = _Q(), _gen(6), 64, 96
    gw = Q.pack_gated(_codes(g, N, C), _scales(g, N), _codes(g, N, C), _scales(g, N))
    dw = Q.pack_channel(_codes(g, C, N), _scales(g, C))
    pre = torch.rand(C, generator=g, device="cuda") + 0.5

    def layer(r):
        r, (q, s) = Q.block_norm(r, pre_weight=pre, int8=True)
        h = Q.gated_i8(q, s, gw)
        codes, scales = Q.quantize_activations(h)
        y = Q.linear_i8(codes, scales, dw)
        return (h, codes, scales, y, *Q.block_norm(r, y, pre_weight=pre))
    r = _bf(g, (*lead, C))
    M = r.numel() // C
    got, want = layer(r), layer(r.reshape(M, C))
    for a, b, width in zip(got, want, ((N,), (N,), (), (C,), (C,), (C,))):
        assert a.shape == (*lead, *width) and torch.equal(a.reshape(M, *width), b)
    h = got[0]
    room = torch.zeros(h.numel() + 3, dtype=torch.bfloat16, device="cuda")
    room[3:] = h.reshape(-1)
    wide = torch.zeros((*lead, N + 5), dtype=torch.bfloat16, device="cuda")
    wide[..., 2:2 + N] = h
    for view in (room[3:].view(h.shape), wide[..., 2:2 + N]):
        codes, scales = Q.quantize_activations(view)
        assert torch.equal(codes, got[1]) and torch.equal(scales, got[2])


# ---- norm parameters ---------------------------------------------------------------------

def test_one_tensor_as_gate_and_weight():
    """One tensor [C] may be several parameters at once; one [B, C] is a gate, and no norm weight
    even where it is given as the gate too.  Scalars are neither."""
    Q, g, R, C = _Q(), _gen(7), 6, 32
    r, y, dx = _bf(g, (R, C)), _bf(g, (R, C)), _bf(g, (R, C))
    w, both, one = torch.rand(C, device="cuda"), torch.rand((2, C), device="cuda"), torch.tensor(1.0, device="cuda")
    kw = {"post_weight": w, "pre_weight": w, "gate": w}
    for a, b in zip(Q.block_norm(r, y, **kw), Q.block_norm(r, y, **{k: v.clone() for k, v in kw.items()})):
        assert torch.equal(a, b)
    grads = Q.block_norm_backward(dx, None, r, y, **kw)
    for a, b in zip(grads, Q.block_norm_backward(dx, None, r, y, **{k: v.clone() for k, v in kw.items()})):
        assert torch.equal(a, b)
    for change in ({"post_weight": both, "gate": both}, {"pre_weight": both, "gate": both}, {"post_weight": both},
                   {"gate": one}, {"post_weight": one}, {"pre_weight": one, "gate": one}, {"gate": both[None]}):
        bad = {**kw, **change}
        for f in (lambda: Q.block_norm(r, y, **bad), lambda: Q.block_norm_backward(dx, None, r, y, **bad)):
            with pytest.raises(Q.QLinearError):
                f()
                pytest.fail(f"{sorted(change)} was taken")
