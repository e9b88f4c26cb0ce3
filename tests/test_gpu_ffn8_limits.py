"""The 8-bit operators where a thread an element would be more than a launch can have."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = torch.float64


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


@pytest.fixture(autouse=True)
def _room():
    """These hold up to 140 GB each: what the allocator keeps from other tests goes first."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def _codes(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)


@pytest.mark.parametrize("gated", [False, True])
def test_backward_operands_past_two_to_the_32(gated):
    """M N past 2^32 with N odd: gradients and scales that are powers of two, so results are
    exact sums, rounded once."""
    Q, g, K = _Q(), _gen(1), 32
    M, N = (300000, 14337) if not gated else (300000, 7201)
    w, s = _codes(g, N, K), 2.0 ** torch.randint(-2, 3, (N,), generator=g, device="cuda").float()
    dy = torch.randint(-1, 2, (M, N), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    rows = torch.tensor([0, 1, M // 2, 286331, 299999], device="cuda")
    print("backward", M, N, K, gated, flush=True)
    if gated:
        raw = torch.full((M, 2 * N), 32.0, dtype=torch.bfloat16, device="cuda")
        dx, draw = Q.gated_i8_backward(dy, raw, Q.pack_gated(w, s, w, s))
        dv = torch.cat([dy[rows], dy[rows]], 1).to(D) * 32             # act(32) = 32, act'(32) = 1
        assert torch.equal(draw[rows].to(D), dv)
        both = torch.cat([w.to(D) * s.to(D)[:, None]] * 2)
    else:
        dx, dv, both = Q.linear_i8_backward(dy, Q.pack_channel(w, s)), dy[rows].to(D), w.to(D) * s.to(D)[:, None]
    assert torch.equal(dx[rows], torch.mm(dv, both).float().bfloat16())


def test_forward_rows_past_every_small_tile():
    Q, g = _Q(), _gen(2)
    M, N, K = (1 << 29) + 37, 3, 32
    w, s = _codes(g, N, K), torch.ones(N, device="cuda")
    x, xs = _codes(g, M, K), torch.ones(M, device="cuda")
    print("linear_i8", M, N, K, flush=True)
    y = Q.linear_i8(x, xs, Q.pack_channel(w, s))
    rows = torch.tensor([0, 1, M // 2, (1 << 29) - 1, 1 << 29, M - 1], device="cuda")
    assert torch.equal(y[rows], torch.mm(x[rows].to(D), w.to(D).t().contiguous()).float().bfloat16())


def test_pack_weights_past_64_gib():
    Q, N, K = _Q(), 1 << 20, 65568
    w = torch.empty((N, K), dtype=torch.int8, device="cuda")
    g = _gen(3)
    for i in range(0, N, 1 << 16):
        w[i:i + (1 << 16)] = _codes(g, 1 << 16, K)
    s = torch.exp(torch.randn((N,), generator=g, device="cuda")) * 1e-3
    rows = torch.tensor([0, 1, 65535, 65536, N // 2, N - 17, N - 1], device="cuda")
    kept = w[rows].clone()
    print("pack", N, K, flush=True)
    pw = Q.pack_channel(w, s)
    del w
    torch.cuda.empty_cache()
    x, xs = _codes(g, 3, K), torch.ones(3, device="cuda")
    y = Q.linear_i8(x, xs, pw, out_dtype=torch.float32)[:, rows].to(D)
    ref = torch.mm(x.to(D), kept.to(D).t().contiguous()) * s[rows].to(D)
    assert bool(((y - ref).abs() <= 4 * 2.0 ** -24 * ref.abs()).all())
    codes, scales = Q.unpack_channel(pw)
    assert torch.equal(codes[rows], kept) and torch.equal(scales, s)


def test_no_rows_and_many_gates():
    Q, C, B = _Q(), 8, 70000
    r, y, gate = torch.zeros((0, C), device="cuda"), torch.zeros((0, C), device="cuda").bfloat16(), torch.ones((B, C), device="cuda")
    w = torch.ones(C, device="cuda")
    got = Q.block_norm_backward(y, None, r, y, post_weight=w, pre_weight=w, gate=gate)
    assert got[4].shape == (B, C) and all(bool((t == 0).all()) for t in got[2:])
