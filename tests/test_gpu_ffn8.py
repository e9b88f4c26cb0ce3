"""The 8-bit feed-forward operators against plain 64-bit implementations.

Tolerances come from the arithmetic: `E` is the rounding unit of float32 and `H` that of
bf16 (eight significant bits: half an ulp is at most 2^-8 of the value).  A product's
integer sum is exact, so a float32 result differs by the roundings of the sum, the two
scales and the bias; sums in float32 by their length or depth times E; every bf16 result by
H of itself.  Cases whose values are exact in every
format are compared bit for bit.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E, H = 2.0 ** -24, 2.0 ** -8
D = torch.float64


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(g, rows, cols):
    return torch.randint(-128, 128, (rows, cols), generator=g, device="cuda", dtype=torch.int8)


def _scales(g, n, typical):
    return torch.exp(torch.randn((n,), generator=g, device="cuda")) * typical


def _bf(g, shape, typical=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * typical).bfloat16()


def _mm(a, b):
    return torch.mm(a.to(D), b.to(D).t().contiguous())


def _close(got, ref, tol, what):
    got = got.to(D)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs() - tol
    assert bool(torch.isfinite(got).all()) and float(off.max()) <= 0.0, (what, float(off.max()), int(off.argmax()))


# ---- packing ---------------------------------------------------------------------------

@pytest.mark.parametrize("N,K", [(1, 32), (17, 96), (16, 64), (333, 1056)])
def test_pack_round_trip(N, K):
    Q, g = _Q(), _gen(N + K)
    parts = [_codes(g, N, K), _scales(g, N, 0.1), _codes(g, N, K), _scales(g, N, 0.1)]
    for got, want in zip(Q.unpack_channel(Q.pack_channel(*parts[:2])), parts[:2]):
        assert torch.equal(got, want)
    for got, want in zip(Q.unpack_gated(Q.pack_gated(*parts)), parts):
        assert torch.equal(got, want)


# ---- linear ----------------------------------------------------------------------------

def _linear_case(M, N, K, seed, bias=True):
    g = _gen(seed)
    x, xs, w, ws = _codes(g, M, K), _scales(g, M, 0.02), _codes(g, N, K), _scales(g, N, 0.002)
    return x, xs, w, ws, (_bf(g, (N,)) if bias else None)


def _linear_ref(x, xs, w, ws, b):
    p = _mm(x, w) * xs.to(D)[:, None] * ws.to(D)
    ref = p if b is None else p + b.to(D)
    return ref, 4 * E * (p.abs() + ref.abs())


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 129, 300, 513])
@pytest.mark.parametrize("N,K", [(1, 32), (19, 64), (200, 736), (516, 2080)])
def test_linear_matches(M, N, K):
    Q = _Q()
    for bias in (False, True):
        x, xs, w, ws, b = _linear_case(M, N, K, M * 7 + N + K, bias)
        pw = Q.pack_channel(w, ws)
        print("linear_i8", M, N, K, bias, flush=True)
        y32 = Q.linear_i8(x, xs, pw, bias=b, out_dtype=torch.float32)
        y16 = Q.linear_i8(x, xs, pw, bias=b)
        ref, tol = _linear_ref(x, xs, w, ws, b)
        _close(y32, ref, tol, "float32")
        assert torch.equal(y16, y32.bfloat16())


@pytest.mark.parametrize("M,N,K", [(3000, 1000, 544), (1100, 4100, 96), (520, 8200, 64), (4200, 4300, 160),
                                   (5000, 4200, 32), (1030, 5001, 4128), (600, 520, 20000)])
def test_linear_large_tiles(M, N, K):
    Q = _Q()
    x, xs, w, ws, b = _linear_case(M, N, K, 11)
    y = Q.linear_i8(x, xs, Q.pack_channel(w, ws), bias=b, out_dtype=torch.float32)
    ref, tol = _linear_ref(x, xs, w, ws, b)
    _close(y, ref, tol, (M, N, K))


# tiles of every size, with the input dimension whole and split
@pytest.mark.parametrize("M,N,K", [(20, 200, 14336), (1900, 8035, 352), (1578, 3949, 640), (67, 5792, 21184), (1024, 4090, 8224),
                                   (8580, 71, 13376), (270, 3658, 288), (67, 2146, 12544), (200, 4099, 4128),
                                   (298, 582, 14400), (251, 31, 2816), (33, 334, 12736), (17, 16, 11712)])
def test_linear_schedules(M, N, K):
    Q = _Q()
    x, xs, w, ws, b = _linear_case(M, N, K, 13)
    print("linear_i8", M, N, K, flush=True)
    pw = Q.pack_channel(w, ws)
    y = Q.linear_i8(x, xs, pw, bias=b, out_dtype=torch.float32)
    ref, tol = _linear_ref(x, xs, w, ws, b)
    _close(y, ref, tol, (M, N, K))
    assert torch.equal(Q.linear_i8(x, xs, pw, bias=b), y.bfloat16())


# outputs that start at any element, through each way they are stored
@pytest.mark.parametrize("start", range(8))
@pytest.mark.parametrize("M,N,K", [(5, 37, 64), (40, 100, 96), (70, 61, 8224), (300, 4100, 160), (2100, 2901, 544),
                                   (2400, 2104, 1056)])
def test_outputs_at_any_element(M, N, K, start):
    Q = _Q()
    x, xs, w, ws, b = _linear_case(M, N, K, 5)
    pw = Q.pack_channel(w, ws)
    print("linear_i8 at", start, M, N, K, flush=True)
    for dtype in (torch.bfloat16, torch.float32):
        room = torch.full((start + M * N + 8,), 7.0, dtype=dtype, device="cuda")
        out = room[start:start + M * N].view(M, N)
        Q.linear_i8(x, xs, pw, bias=b, out_dtype=dtype, out=out)
        assert torch.equal(out, Q.linear_i8(x, xs, pw, bias=b, out_dtype=dtype))
        assert bool((room[:start] == 7).all()) and bool((room[start + M * N:] == 7).all())
    if N > 3000:
        return
    gx, gxs, up, us, gt, gs, gb = _gated_case(M, N, K, 6, True)
    pg = Q.pack_gated(up, us, gt, gs)
    want, want_raw = Q.gated_i8(gx, gxs, pg, bias=gb, keep_raw=True)
    room = torch.full((start + M * N + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    rooms = torch.full((start + 2 * M * N + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
    out, raw = room[start:start + M * N].view(M, N), rooms[start:start + 2 * M * N].view(M, 2 * N)
    Q.gated_i8(gx, gxs, pg, bias=gb, out=out, raw=raw)
    assert torch.equal(out, want) and torch.equal(raw, want_raw)
    for t, n in ((room, M * N), (rooms, 2 * M * N)):
        assert bool((t[:start] == 7).all()) and bool((t[start + n:] == 7).all())


@pytest.mark.parametrize("M", [1, 20, 64, 70, 260])
def test_linear_longest_rows_do_not_wrap(M):
    """The largest input dimension with all codes -128: sums of 2146959360, just below 2^31."""
    Q, K, N = _Q(), 131040, 40
    x = torch.full((M, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((N, K), -128, dtype=torch.int8, device="cuda")
    w[1::2] = 127
    one = torch.ones(max(M, N), device="cuda")
    y = Q.linear_i8(x, one[:M], Q.pack_channel(w, one[:N]), out_dtype=torch.float32)
    want = torch.where(torch.arange(N, device="cuda") % 2 == 0, 128.0 * 128 * K, -128.0 * 127 * K).float()
    assert torch.equal(y, want.expand(M, N))


def test_linear_scales_that_are_not_numbers_stay_in_their_rows_and_columns():
    Q, M, N, K = _Q(), 70, 50, 128
    x, xs, w, ws, _ = _linear_case(M, N, K, 5, False)
    good = Q.linear_i8(x, xs, Q.pack_channel(w, ws), out_dtype=torch.float32)
    xs2, ws2 = xs.clone(), ws.clone()
    xs2[3], xs2[40], ws2[7] = float("nan"), 0.0, float("inf")
    y = Q.linear_i8(x, xs2, Q.pack_channel(w, ws2), out_dtype=torch.float32)
    rows = [m for m in range(M) if m not in (3, 40)]
    cols = [n for n in range(N) if n != 7]
    assert torch.equal(y[rows][:, cols], good[rows][:, cols])
    assert bool(torch.isnan(y[3]).all()) and bool((y[40][cols] == 0).all()) and not bool(torch.isfinite(y[rows][:, 7]).any())


def test_linear_views_shapes_and_outputs():
    Q, N, K = _Q(), 40, 96
    x, xs, w, ws, b = _linear_case(30, N, K, 9)
    pw = Q.pack_channel(w, ws)
    want = Q.linear_i8(x, xs, pw, bias=b)
    assert torch.equal(Q.linear_i8(x.view(5, 6, K), xs.view(5, 6), pw, bias=b), want.view(5, 6, N))
    wide = torch.zeros((30, 2 * K), dtype=torch.int8, device="cuda")
    wide[:, 7:7 + K] = x                                       # strided and misaligned
    assert torch.equal(Q.linear_i8(wide[:, 7:7 + K], xs, pw, bias=b), want)
    flat = torch.empty(30 * K + 3, dtype=torch.int8, device="cuda")
    flat[3:] = x.reshape(-1)
    assert torch.equal(Q.linear_i8(flat[3:].view(30, K), xs, pw, bias=b), want)
    spaced = torch.empty((30, 2), device="cuda")
    spaced[:, 0] = xs
    assert torch.equal(Q.linear_i8(x, spaced[:, 0], pw, bias=b), want)
    back = torch.full((30 * N + 1,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = back[1:].view(30, N)                                 # rows off every vector boundary
    assert Q.linear_i8(x, xs, pw, bias=b, out=out) is out and torch.equal(out, want) and float(back[0]) == 7.0
    e = Q.linear_i8(x[:0], xs[:0], pw)
    assert e.shape == (0, N)


def test_outputs_past_two_to_the_31_elements():
    Q, M, N, K = _Q(), 70000, 32768, 32
    x, xs, w, ws, _ = _linear_case(M, N, K, 3, False)
    y = Q.linear_i8(x, xs, Q.pack_channel(w, ws))
    rows = torch.tensor([0, 1, 65535, 65536, M - 1], device="cuda")
    ref, tol = _linear_ref(x[rows], xs[rows], w, ws, None)
    _close(y[rows], ref, tol + H * ref.abs(), "rows")


def test_weights_past_four_gib():
    Q, N, K = _Q(), 1 << 20, 4224
    g = _gen(8)
    w = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = _scales(g, N, 0.002)
    pw = Q.pack_channel(w, ws)
    cols = torch.tensor([0, 1, 508000, 508401, N - 17, N - 1], device="cuda")
    for M in (3, 70):
        x, xs = _codes(g, M, K), _scales(g, M, 0.02)
        y = Q.linear_i8(x, xs, pw, out_dtype=torch.float32)
        ref, tol = _linear_ref(x, xs, w[cols], ws[cols], None)
        _close(y[:, cols], ref, tol, M)
    dy = torch.zeros((2, N), dtype=torch.bfloat16, device="cuda")
    dy[0, N - 1] = 1.0
    dy[1, 508401] = -2.0
    ref = torch.stack([w[N - 1].to(D) * ws[N - 1].to(D), -2.0 * w[508401].to(D) * ws[508401].to(D)])
    _close(Q.linear_i8_backward(dy, pw), ref, 2 * H * ref.abs(), "backward")


# ---- linear, backward --------------------------------------------------------------------

def _back_tol(dy, ws, w, ref):
    size = torch.mm(dy.to(D).abs() * ws.to(D), w.to(D).abs())
    return (H + 2 * dy.shape[1] * E) * size + H * ref.abs()


BACK = [(1, 8, 32), (1, 37, 64), (5, 64, 96), (16, 200, 736), (33, 129, 160), (64, 516, 288), (130, 1000, 416),
        (300, 264, 2080), (520, 77, 544)]


@pytest.mark.parametrize("M,N,K", BACK)
def test_linear_backward_matches(M, N, K):
    Q, g = _Q(), _gen(M + N + K)
    w, ws, dy = _codes(g, N, K), _scales(g, N, 0.002), _bf(g, (M, N))
    print("linear_i8_backward", M, N, K, flush=True)
    dx = Q.linear_i8_backward(dy, Q.pack_channel(w, ws))
    ref = torch.mm(dy.to(D) * ws.to(D), w.to(D))
    _close(dx, ref, _back_tol(dy, ws, w, ref), "dx")


@pytest.mark.parametrize("M,N,K", BACK + [(700, 2056, 1056), (2100, 520, 4128)])
def test_linear_backward_exact_values(M, N, K):
    """Scales that are powers of two and few small integers in dy: every product and sum is
    exact in float32, so the result is the rounding of the exact one, bit for bit."""
    Q, g = _Q(), _gen(M + N)
    w = _codes(g, N, K)
    ws = 2.0 ** torch.randint(-3, 4, (N,), generator=g, device="cuda").float()
    dy = torch.randint(-4, 5, (M, N), generator=g, device="cuda").bfloat16()
    dx = Q.linear_i8_backward(dy, Q.pack_channel(w, ws))
    want = torch.mm(dy.to(D) * ws.to(D), w.to(D)).float().bfloat16()
    assert torch.equal(dx, want)


def test_linear_backward_against_differences():
    """<dx, d> against differences of the forward pass in 64 bits (which is linear, so the
    step does not matter) along random directions."""
    Q, g, M, N, K = _Q(), _gen(2), 9, 72, 128
    w, ws, dy = _codes(g, N, K), _scales(g, N, 0.01), _bf(g, (M, N))
    dx = Q.linear_i8_backward(dy, Q.pack_channel(w, ws)).to(D)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=D)

    def loss(v):
        return float((torch.mm(v, (w.to(D) * ws.to(D)[:, None]).t().contiguous()) * dy.to(D)).sum())
    for _ in range(3):
        d = torch.randn((M, K), generator=g, device="cuda", dtype=D)
        diff = (loss(x + 1e-3 * d) - loss(x - 1e-3 * d)) / 2e-3
        size = torch.mm(dy.to(D).abs() * ws.to(D), w.to(D).abs())
        assert abs(float((dx * d).sum()) - diff) <= float(((2.5 * H * size) * d.abs()).sum())


def test_backward_rows_of_other_tokens_do_not_mix():
    """A token whose gradient is infinite leaves the others as they are, also in the rows'
    padding past the last channel."""
    Q, g = _Q(), _gen(4)
    for N in (40, 37):
        w, ws, dy = _codes(g, N, 96), _scales(g, N, 0.01), _bf(g, (70, N))
        pw = Q.pack_channel(w, ws)
        good = Q.linear_i8_backward(dy, pw)
        dy2 = dy.clone()
        dy2[20] = float("inf")
        bad = Q.linear_i8_backward(dy2, pw)
        keep = [m for m in range(70) if m != 20]
        assert torch.equal(bad[keep], good[keep]) and not bool(torch.isfinite(bad[20]).any())


# ---- gated -------------------------------------------------------------------------------

def _act(z, act):
    """act(g), act'(g) in 64 bits."""
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * torch.special.expit(-z)
    c = (2.0 / torch.pi) ** 0.5
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z ** 2)


def _gated_case(M, N, K, seed, bias):
    g = _gen(seed)
    t = 1.0 / (74.0 * 74.0 * K ** 0.5)                       # pre-activations of about one
    return (_codes(g, M, K), _scales(g, M, 1.0), _codes(g, N, K), _scales(g, N, t), _codes(g, N, K), _scales(g, N, t),
            _bf(g, (2 * N,)) if bias else None)


def _gated_ref(x, xs, up, us, gt, gs, b, act):
    N = up.shape[0]
    u, eu = _linear_ref(x, xs, up, us, None if b is None else b[:N])
    z, ez = _linear_ref(x, xs, gt, gs, None if b is None else b[N:])
    a, _ = _act(z, act)
    h = a * u
    # |act'| <= 1.13; the exponential's relative error grows with its argument, which for
    # the cubic of GELU is at most 2 (|z| + |z|^3), and is past mattering beyond 100
    arg = (z.abs() if act == "silu" else 2 * (z.abs() + z.abs() ** 3)).clamp(max=100)
    tol = 1.13 * ez * u.abs() + a.abs() * eu + (arg + 10) * 4 * E * (h.abs() + E)
    return u, eu, z, ez, h, tol


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M", [1, 16, 31, 64, 66, 140, 400])
@pytest.mark.parametrize("N,K", [(1, 32), (24, 96), (333, 544)])
def test_gated_matches(M, N, K, act):
    Q = _Q()
    for bias in (False, True):
        case = _gated_case(M, N, K, M + N, bias)
        x, xs, up, us, gt, gs, b = case
        pw = Q.pack_gated(up, us, gt, gs)
        print("gated_i8", M, N, K, act, bias, flush=True)
        h32, raw = Q.gated_i8(x, xs, pw, bias=b, act=act, keep_raw=True, out_dtype=torch.float32)
        h16 = Q.gated_i8(x, xs, pw, bias=b, act=act)
        u, eu, z, ez, h, tol = _gated_ref(*case, act)
        _close(h32, h, tol, "h")
        _close(raw[:, :N], u, eu + H * u.abs(), "up")
        _close(raw[:, N:], z, ez + H * z.abs(), "gate")
        assert torch.equal(h16, h32.bfloat16())


@pytest.mark.parametrize("M,N,K", [(1500, 1000, 96), (600, 4104, 160), (2100, 4200, 224), (4400, 2101, 64), (520, 264, 20000)])
def test_gated_large_tiles(M, N, K):
    Q = _Q()
    case = _gated_case(M, N, K, 3, True)
    pw = Q.pack_gated(*case[2:6])
    h = Q.gated_i8(case[0], case[1], pw, bias=case[6], out_dtype=torch.float32)
    _, _, _, _, ref, tol = _gated_ref(*case, "silu")
    _close(h, ref, tol, (M, N, K))


@pytest.mark.parametrize("M,N,K", [(1913, 3977, 544), (325, 8329, 640), (65, 4470, 14464), (1060, 1186, 4000), (8241, 40, 15104),
                                   (77, 5730, 288), (190, 900, 19136), (33, 4098, 32), (325, 320, 12384), (35, 16, 32),
                                   (80, 1300, 14144), (25, 779, 128)])
def test_gated_schedules(M, N, K):
    Q = _Q()
    case = _gated_case(M, N, K, 17, True)
    print("gated_i8", M, N, K, flush=True)
    pw = Q.pack_gated(*case[2:6])
    h, raw = Q.gated_i8(case[0], case[1], pw, bias=case[6], keep_raw=True, out_dtype=torch.float32)
    u, eu, z, ez, ref, tol = _gated_ref(*case, "silu")
    _close(h, ref, tol, (M, N, K))
    _close(raw[:, :N], u, eu + H * u.abs(), "up")
    _close(raw[:, N:], z, ez + H * z.abs(), "gate")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_extreme_pre_activations(act):
    """Huge pre-activations: the activation is 0 or the identity there, and no cube or
    exponential in between overflows into NaN, forward or backward."""
    Q, N, K = _Q(), 16, 32
    x = torch.zeros((4, K), dtype=torch.int8, device="cuda")
    x[:, 0] = torch.tensor([1, -1, 127, -127], dtype=torch.int8)
    w = torch.zeros((N, K), dtype=torch.int8, device="cuda")
    w[:, 0] = 1
    one = torch.ones(N, device="cuda")
    gs = (10.0 ** torch.linspace(0, 30, N)).cuda()
    pw = Q.pack_gated(w, one, w, gs)
    xs = torch.ones(4, device="cuda")
    h, raw = Q.gated_i8(x, xs, pw, act=act, keep_raw=True, out_dtype=torch.float32)
    u, z = x[:, :1].to(D), x[:, :1].to(D) * gs.to(D)
    a, da = _act(z, act)
    _close(h, a * u, 500 * E * ((a * u).abs() + 1.0), "h")
    dh = torch.ones((4, N), dtype=torch.bfloat16, device="cuda")
    dx, draw = Q.gated_i8_backward(dh, raw, pw, act=act)
    a, da = _act(raw[:, N:].to(D), act)
    da = torch.nan_to_num(da, nan=1.0)                        # inf * 0 of the 64-bit cube
    # next to a saturated exponential the slope is held to its argument's relative error
    _close(draw[:, :N], a, H * a.abs() + 500 * E * (a.abs() + 1.0), "dup")
    want = raw[:, :N].to(D) * da
    _close(draw[:, N:], want, H * want.abs() + 127 * 500 * E, "dgate")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,N,K", [(1, 8, 32), (3, 37, 96), (16, 200, 544), (70, 136, 160), (300, 329, 288), (520, 520, 1056)])
def test_gated_backward_matches(M, N, K, act):
    Q, g = _Q(), _gen(M + N)
    _, _, up, us, gt, gs, _ = _gated_case(1, N, K, N, False)
    pw = Q.pack_gated(up, us, gt, gs)
    dh, raw = _bf(g, (M, N)), _bf(g, (M, 2 * N), 1.5)
    print("gated_i8_backward", M, N, K, act, flush=True)
    dx, draw = Q.gated_i8_backward(dh, raw, pw, act=act)
    d, u, z = dh.to(D), raw[:, :N].to(D), raw[:, N:].to(D)
    a, da = _act(z, act)
    arg = (z.abs() if act == "silu" else 2 * (z.abs() + z.abs() ** 3)).clamp(max=100)
    loss = (arg + 10) * 8 * E                                 # of the logistic factors
    _close(draw[:, :N], d * a, (H + loss) * (d * a).abs() + E, "dup")
    _close(draw[:, N:], d * u * da, H * (d * u * da).abs() + 4 * loss * (d * u).abs() * (1 + z.abs()) ** 2 + E, "dgate")
    # the product's operand is the scaled gradient, rounded once
    w = torch.cat([up.to(D) * us.to(D)[:, None], gt.to(D) * gs.to(D)[:, None]])
    exact = torch.cat([d * a, d * u * da], 1)
    slip = torch.cat([loss * (d * a).abs(), 4 * loss * (d * u).abs() * (1 + z.abs()) ** 2], 1)
    ref = torch.mm(exact, w)
    size = torch.mm(exact.abs(), w.abs())
    _close(dx, ref, (H + 4 * N * E) * size + torch.mm(slip, w.abs()) + H * ref.abs(), "dx")


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward_against_differences(act):
    Q, g, M, N, K = _Q(), _gen(6), 7, 48, 96
    x, xs, up, us, gt, gs, _ = _gated_case(M, N, K, 5, False)
    pw = Q.pack_gated(up, us, gt, gs)
    dh = _bf(g, (M, N))
    h, raw = Q.gated_i8(x, xs, pw, act=act, keep_raw=True)
    dx, _ = Q.gated_i8_backward(dh, raw, pw, act=act)
    wu, wg = up.to(D) * us.to(D)[:, None], gt.to(D) * gs.to(D)[:, None]
    v = x.to(D) * xs.to(D)[:, None]

    def forward(t):
        return _act(torch.mm(t, wg.t().contiguous()), act)[0] * torch.mm(t, wu.t().contiguous())
    u, z = torch.mm(v, wu.t().contiguous()), torch.mm(v, wg.t().contiguous())
    # roundings to bf16 of raw (up, gate: slopes at most 1.13 and |act''| <= 1.13), of draw
    # and of the weights, each H of its term
    size = torch.mm(dh.to(D).abs() * (z.abs() + 1) * 4, wu.abs()) + torch.mm(
        dh.to(D).abs() * (u.abs() + 1) * 4 * (1 + z.abs()), wg.abs())
    for _ in range(3):
        d = torch.randn((M, K), generator=g, device="cuda", dtype=D)
        e = 1e-6
        diff = float(((forward(v + e * d) - forward(v - e * d)) / (2 * e) * dh.to(D)).sum())
        assert abs(float((dx.to(D) * d).sum()) - diff) <= float((4 * H * size * d.abs()).sum()) + 1e-6 * abs(diff)


# ---- block norm --------------------------------------------------------------------------

# depth of the float32 sums: values of one thread (at most 32), a wavefront's tree (6) and 16
# wavefronts, so a sum of squares is off by at most 54 E of itself and its inverse root by
# half of that and its own few roundings
DEPTH = 64 * E


def _norm_case(R, C, B, seed, f32, params=torch.float32, has_y=True, post=True, pre=True):
    g = _gen(seed)
    c = {"r": torch.randn((R, C), generator=g, device="cuda") * 2}
    c["r"] = c["r"] if f32 else c["r"].bfloat16()
    c["y"] = _bf(g, (R, C), 0.7) if has_y else None
    c["post"] = (1 + 0.2 * torch.randn((C,), generator=g, device="cuda")).to(params) if post and has_y else None
    c["pre"] = (1 + 0.2 * torch.randn((C,), generator=g, device="cuda")).to(params) if pre else None
    shape = {0: None, 1: (C,)}.get(B, (B, C))
    c["gate"] = None if shape is None or not has_y else torch.randn(shape, generator=g, device="cuda").to(params)
    return c


def _gate_rows(gate, R):
    return gate.to(D) if gate.dim() == 1 else gate.to(D).repeat_interleave(R // gate.shape[0], 0)


def _norm_ref(c, alpha, eps):
    r = alpha * c["r"].to(D)
    size = r.abs()
    if c["y"] is not None:
        t = c["y"].to(D)
        if c["post"] is not None:
            t = t / (t.square().mean(1, keepdim=True) + eps).sqrt() * c["post"].to(D)
        if c["gate"] is not None:
            t = t * _gate_rows(c["gate"], t.shape[0])
        r, size = r + t, size + t.abs()
    e_r = DEPTH * size
    if c["pre"] is None:
        return r, e_r, None, None
    root = (r.square().mean(1, keepdim=True) + eps).sqrt()
    x = r / root * c["pre"].to(D)
    # r' itself may be off by e_r, which also moves the root
    moved = (e_r.square().mean(1, keepdim=True)).sqrt() / root
    return r, e_r, x, (2 * DEPTH + 2 * moved) * x.abs() + 2 * e_r / root * c["pre"].to(D).abs()


NORMS = [(1, 32, 1), (5, 8, 0), (7, 1, 1), (3, 255, 1), (4, 4096, 4), (40, 1000, 2), (33, 96, 0), (1500, 264, 3),
         (6, 4104, 1), (5, 9001, 1), (8, 14336, 2), (3, 32768, 1), (2, 32767, 1)]


@pytest.mark.parametrize("R,C,B", NORMS)
@pytest.mark.parametrize("f32", [False, True])
def test_block_norm_matches(R, C, B, f32):
    Q, alpha, eps = _Q(), 0.9, 1e-6
    for params in (torch.float32, torch.bfloat16):
        c = _norm_case(R, C, B, R + C, f32, params)
        print("block_norm", R, C, B, f32, params, flush=True)
        r, x = Q.block_norm(c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"],
                            residual_scale=alpha, eps=eps)
        rr, e_r, xr, e_x = _norm_ref(c, alpha, eps)
        _close(r, rr, e_r + (0 if f32 else H) * rr.abs(), "r")
        _close(x, xr, e_x + H * xr.abs(), "x")
        r2, (q, s) = Q.block_norm(c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"],
                                  residual_scale=alpha, eps=eps, int8=True)
        assert torch.equal(r2, r)
        want = xr.abs().amax(1) / 127
        _close(s, want, 4 * E * want + e_x.amax(1) / 127, "scales")
        assert int(q.abs().max()) <= 127
        _close(q.to(D) * s.to(D)[:, None], xr, 0.501 * s.to(D)[:, None] + e_x, "codes")
        assert bool((q.abs().amax(1) == 127).all())


@pytest.mark.parametrize("has_y,post,pre,B", [(False, False, True, 0), (True, False, True, 1), (True, True, False, 0),
                                              (True, False, False, 5), (False, False, False, 0), (True, True, True, 10)])
@pytest.mark.parametrize("C", [64, 61])
def test_block_norm_parts(has_y, post, pre, B, C):
    """Without a block, a post norm, a gate, a pre norm; a gate for each row."""
    Q, R = _Q(), 10
    c = _norm_case(R, C, B, 7, True, has_y=has_y, post=post, pre=pre)
    r, x = Q.block_norm(c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"], residual_scale=0.5)
    rr, e_r, xr, e_x = _norm_ref(c, 0.5, 1e-6)
    _close(r, rr, e_r, "r")
    assert (x is None) == (not pre)
    if pre:
        _close(x, xr, e_x + H * xr.abs(), "x")
    _check_back(Q, c, R, C, 0.5, 1e-6, 3)


def test_block_norm_rows_of_zeros_and_bad_rows():
    Q, R, C = _Q(), 9, 128
    c = _norm_case(R, C, 1, 3, True)
    kw = {k + "_weight": c[k] for k in ("post", "pre")}
    good = Q.block_norm(c["r"], c["y"], gate=c["gate"], int8=True, **kw)
    r, y = c["r"].clone(), c["y"].clone()
    r[2] = 0
    y[2] = 0
    y[4, 5] = float("nan")
    r[6, 7] = float("inf")
    out, (q, s) = Q.block_norm(r, y, gate=c["gate"], int8=True, **kw)
    keep = [0, 1, 3, 5, 7, 8]
    assert torch.equal(out[keep], good[0][keep]) and torch.equal(q[keep], good[1][0][keep]) and torch.equal(s[keep], good[1][1][keep])
    assert bool((out[2] == 0).all()) and bool((q[2] == 0).all()) and float(s[2]) == 0.0
    assert bool(torch.isnan(s[[4, 6]]).all()) and bool((q[[4, 6]] == 0).all())
    x = Q.block_norm(r, y, gate=c["gate"], **kw)[1]
    assert bool((x[2] == 0).all()) and bool(torch.isnan(x[4]).all())


def test_block_norm_views_in_place_and_empty():
    Q, R, C = _Q(), 12, 64
    c = _norm_case(R, C, 3, 5, True)
    kw = dict(post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"])
    r, x = Q.block_norm(c["r"], c["y"], **kw)
    wide = torch.zeros((R, C + 5), device="cuda")
    wide[:, 3:3 + C] = c["r"]
    flat = torch.zeros(R * C + 1, dtype=torch.bfloat16, device="cuda")
    flat[1:] = c["y"].reshape(-1)
    r2, x2 = Q.block_norm(wide[:, 3:3 + C], flat[1:].view(R, C), **kw)      # strided; off 16 bytes
    # the path for rows off 16-byte boundaries adds in another order
    _close(r2, r.to(D), 2 * DEPTH * (r.to(D).abs() + 4), "r")
    _close(x2, x.to(D), 2 * H * (x.to(D).abs() + E * 64), "x")
    r3, x3 = Q.block_norm(c["r"].view(3, 4, C), c["y"].view(3, 4, C), **kw)
    assert torch.equal(r3.view(R, C), r) and torch.equal(x3.view(R, C), x)
    stream = c["r"].clone()
    r4, x4 = Q.block_norm(stream, c["y"], residual_out=stream, **kw)
    assert r4 is stream and torch.equal(r4, r) and torch.equal(x4, x)
    e, (q, s) = Q.block_norm(c["r"][:0], c["y"][:0], int8=True, **kw)
    assert e.shape == (0, C) and q.shape == (0, C) and s.shape == (0,)
    got = Q.block_norm_backward(x[:0], None, r[:0], c["y"][:0], **kw)
    assert got[0].shape == (0, C) and all(bool((t == 0).all()) for t in got[2:]) and got[4].shape == (3, C)


def test_block_norm_past_two_to_the_31_elements():
    Q, R, C = _Q(), 70000, 32768
    g = _gen(2)
    r = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((R, C), dtype=torch.bfloat16, device="cuda")
    rows = [0, 65535, 65536, R - 1]
    for i in rows:
        r[i], y[i] = _bf(g, (C,)), _bf(g, (C,))
    w = torch.ones(C, device="cuda")
    out, (q, s) = Q.block_norm(r, y, post_weight=w, pre_weight=w, int8=True)
    c = {"r": r[rows], "y": y[rows], "post": w, "pre": w, "gate": None}
    rr, e_r, xr, e_x = _norm_ref(c, 1.0, 1e-6)
    _close(out[rows], rr, e_r + H * rr.abs(), "r")
    _close(q[rows].to(D) * s[rows].to(D)[:, None], xr, 0.501 * s[rows].to(D)[:, None] + e_x, "x")
    assert float(s.sum()) == float(s[rows].sum())


def _back_ref(c, dx, dr, alpha, eps):
    """Gradients in 64 bits, and their sizes (the sums of the terms' magnitudes)."""
    R = c["r"].shape[0]
    Dd = torch.zeros_like(c["r"], dtype=D) if dr is None else dr.to(D)
    size = Dd.abs()
    dpre = s_pre = dpost = s_post = dgate = s_gate = dy = s_dy = None
    if c["pre"] is not None:
        r = c["r"].to(D)
        iq = 1 / (r.square().mean(1, keepdim=True) + eps).sqrt()
        u, n = r * iq, dx.to(D) * c["pre"].to(D)
        Dd = Dd + iq * (n - u * (n * u).mean(1, keepdim=True))
        size = size + iq * (n.abs() + u.abs() * (n * u).abs().mean(1, keepdim=True))
        dpre, s_pre = (dx.to(D) * u).sum(0), (dx.to(D) * u).abs().sum(0)
    if c["y"] is not None:
        y = c["y"].to(D)
        gate = torch.ones_like(y) if c["gate"] is None else _gate_rows(c["gate"], R) * torch.ones_like(y)
        if c["post"] is None:
            t, dy, s_dy = y, Dd * gate, size * gate.abs()
        else:
            ip = 1 / (y.square().mean(1, keepdim=True) + eps).sqrt()
            v, post = y * ip, c["post"].to(D)
            t = v * post
            dv, s_v = Dd * gate * post, size * (gate * post).abs()
            dy = ip * (dv - v * (dv * v).mean(1, keepdim=True))
            s_dy = ip * (s_v + v.abs() * (s_v * v.abs()).mean(1, keepdim=True))
            dpost, s_post = (Dd * gate * v).sum(0), (size * (gate * v).abs()).sum(0)
        if c["gate"] is not None:
            shape = c["gate"].shape
            B = 1 if len(shape) == 1 else shape[0]
            dgate = (Dd * t).reshape(B, -1, t.shape[1]).sum(1).reshape(shape)
            s_gate = (size * t.abs()).reshape(B, -1, t.shape[1]).sum(1).reshape(shape)
    return (alpha * Dd, dy, dpost, dpre, dgate), (alpha * size, s_dy, s_post, s_pre, s_gate)


def _check_back(Q, c, R, C, alpha, eps, seed, with_dr=True):
    g = _gen(seed)
    dx = _bf(g, (R, C)) if c["pre"] is not None else None
    dr = torch.randn((R, C), generator=g, device="cuda").to(c["r"].dtype) if with_dr else None
    print("block_norm_backward", R, C, c["r"].dtype, flush=True)
    got = Q.block_norm_backward(dx, dr, c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"],
                                residual_scale=alpha, eps=eps)
    ref, size = _back_ref(c, dx, dr, alpha, eps)
    names = ("dresidual", "dy", "dpost", "dpre", "dgate")
    for name, a, b, s in zip(names, got, ref, size):
        assert (a is None) == (b is None), name
        if a is None:
            continue
        # inverse roots, means and products: a few DEPTH of the terms; column sums besides
        # one E of the terms for each row that is added
        tol = 4 * DEPTH * s + (R * E * s if name.startswith("dp") or name == "dgate" else 0)
        if a.dtype == torch.bfloat16:
            tol = tol + H * b.abs()
        _close(a, b, tol, name)
    again = Q.block_norm_backward(dx, dr, c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"],
                                  residual_scale=alpha, eps=eps)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("R,C,B", NORMS + [(2000, 40, 1000), (1200, 24, 1200), (1024, 48, 512), (600, 72, 2)])
@pytest.mark.parametrize("f32", [False, True])
def test_block_norm_backward_matches(R, C, B, f32):
    Q = _Q()
    for params in (torch.float32, torch.bfloat16):
        _check_back(Q, _norm_case(R, C, B, R + C, f32, params), R, C, 0.9, 1e-6, R)
    _check_back(Q, _norm_case(R, C, B, R + C, f32), R, C, 0.9, 1e-6, R, with_dr=False)


def test_block_norm_backward_against_differences():
    Q, R, C, B, alpha, eps = _Q(), 6, 40, 2, 0.8, 1e-5
    c = _norm_case(R, C, B, 1, True)
    g = _gen(9)
    kw = dict(post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"], residual_scale=alpha, eps=eps)
    r_out, _ = Q.block_norm(c["r"], c["y"], **kw)
    dx, dr = _bf(g, (R, C)), torch.randn((R, C), generator=g, device="cuda")
    grads = Q.block_norm_backward(dx, dr, r_out, c["y"], **kw)

    def loss(v):
        r, _, x, _ = _norm_ref(v, alpha, eps)
        return float((r * dr.to(D)).sum() + (x * dx.to(D)).sum())
    for name, grad in zip(("r", "y", "post", "pre", "gate"), grads):
        d = torch.randn(c[name].shape, generator=g, device="cuda", dtype=D)
        e = 1e-5
        plus, minus = ({**c, name: c[name].to(D) + s * e * d} for s in (1, -1))
        diff = (loss(plus) - loss(minus)) / (2 * e)
        terms = float((grad.to(D) * d).abs().sum())
        # central differences: the third derivative's e^2, the loss's own 64-bit rounding / e
        tol = (H if grad.dtype == torch.bfloat16 else 1e-5) * terms + 1e-5 * terms + 1e-6
        assert abs(float((grad.to(D) * d).sum()) - diff) <= tol, name


# ---- together ----------------------------------------------------------------------------

def _sub_layer(Q, c, gw, dw, act="silu"):
    r, (q, s) = Q.block_norm(c["r"], c["y"], post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"], int8=True)
    h = Q.gated_i8(q, s, gw, act=act)
    return r, Q.linear_i8(*Q.quantize_activations(h), dw)


@pytest.mark.parametrize("M", [1, 5, 80])
def test_sub_layer_on_another_stream_and_in_a_graph(M):
    """The operators together: on a side stream with the inputs of another, and captured into
    a graph that is replayed several times with other work in between."""
    Q, C, N = _Q(), 256, 608
    g = _gen(M)
    c = _norm_case(M, C, 1, 3, False)
    gw = Q.pack_gated(_codes(g, N, C), _scales(g, N, 1e-3), _codes(g, N, C), _scales(g, N, 1e-3))
    dw = Q.pack_channel(_codes(g, C, N), _scales(g, C, 1e-3))
    want = _sub_layer(Q, c, gw, dw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _sub_layer(Q, c, gw, dw)
        for _ in range(2):
            _sub_layer(Q, c, gw, dw)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = _sub_layer(Q, c, gw, dw)
    for i in range(4):
        c["y"].copy_(_bf(g, (M, C)))
        graph.replay()
        torch.cuda.synchronize()
        again = _sub_layer(Q, c, gw, dw)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, again)), i


def test_refusals():
    Q, g = _Q(), _gen(1)
    w, s = _codes(g, 32, 64), _scales(g, 32, 0.1)
    cw, gw = Q.pack_channel(w, s), Q.pack_gated(w, s, w, s)
    x, xs = _codes(g, 4, 64), _scales(g, 4, 0.1)
    h = _bf(g, (4, 32))
    c = _norm_case(4, 64, 2, 1, True)
    kw = dict(post_weight=c["post"], pre_weight=c["pre"], gate=c["gate"])
    bad = [
        lambda: Q.pack_channel(w.float(), s), lambda: Q.pack_channel(w, s[:3]), lambda: Q.pack_channel(w[:, :40], s),
        lambda: Q.pack_channel(w.cpu(), s.cpu()), lambda: Q.pack_gated(w, s, w[:16], s[:16]),
        lambda: Q.linear_i8(x, xs, gw), lambda: Q.gated_i8(x, xs, cw), lambda: Q.linear_i8(x[:, :32], xs, cw),
        lambda: Q.linear_i8(x, xs[:2], cw), lambda: Q.linear_i8(x, xs, cw, bias=h[0][:5]),
        lambda: Q.linear_i8(x, xs, cw, out_dtype=torch.float16),
        lambda: Q.linear_i8(x, xs, cw, out=torch.empty((4, 31), dtype=torch.bfloat16, device="cuda")),
        lambda: Q.linear_i8(x, xs.double(), cw), lambda: Q.linear_i8(x.cpu(), xs.cpu(), cw),
        lambda: Q.gated_i8(x, xs, gw, act="relu"), lambda: Q.gated_i8(x, xs, gw, bias=h[0]),
        lambda: Q.linear_i8_backward(h.float(), cw), lambda: Q.linear_i8_backward(h[:, :8], cw),
        lambda: Q.linear_i8_backward(h.clone().requires_grad_(), cw),
        lambda: Q.gated_i8_backward(h, h, gw), lambda: Q.gated_i8_backward(h, torch.cat([h, h], 1), gw, act="tanh"),
        lambda: Q.block_norm(c["r"], None, **kw), lambda: Q.block_norm(c["r"], c["y"].float(), **kw),
        lambda: Q.block_norm(c["r"][:3], c["y"][:3], **kw), lambda: Q.block_norm(c["r"], c["y"], eps=0.0, **kw),
        lambda: Q.block_norm(c["r"], c["y"], int8=True), lambda: Q.block_norm(c["r"].half(), c["y"], **kw),
        lambda: Q.block_norm(c["r"], c["y"], **{**kw, "gate": c["gate"].bfloat16()}),
        lambda: Q.block_norm(c["r"], c["y"], residual_scale=float("nan"), **kw),
        lambda: Q.block_norm_backward(None, None, c["r"], c["y"], **kw),
        lambda: Q.block_norm_backward(c["y"], c["y"], c["r"], c["y"], **kw),
        lambda: Q.block_norm_backward(c["y"], None, c["r"], c["y"], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"), **kw),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(Q.QLinearError):
            call()
            pytest.fail(f"refusal {i} did not raise")


def test_example_stack_learns_its_gates():
    """The example's stack: gates and norms moved off a teacher's come back towards it, and the
    gradient of one gate agrees with the change of the loss along it (int8 activations make the
    loss a step function at the scale of a code, hence the wide step and bound)."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "feed_forward.py")
    spec = importlib.util.spec_from_file_location("feed_forward_example", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    stack = ex.FeedForwardStack(2, 256, 512, seed=3)
    g = _gen(4)
    x = torch.randn((192, 256), generator=g, device="cuda")
    target = stack.forward(x).float()
    for name in ("post", "gate"):
        for p in stack.params[name]:
            p.mul_(1 + 0.3 * torch.randn(p.shape, generator=g, device="cuda"))

    def loss():
        return float(0.5 * (stack.forward(x).float() - target).square().sum() / x.shape[0])
    out, saved = stack.forward(x, keep=True)
    grads, _ = stack.backward(((out.float() - target) / x.shape[0]).bfloat16(), saved)
    gate, d = stack.params["gate"][1], torch.sign(grads["gate"][1])
    kept = gate.clone()
    gate.add_(0.02 * d)
    plus = loss()
    gate.copy_(kept - 0.02 * d)
    minus = loss()
    gate.copy_(kept)
    slope, want = (plus - minus) / 0.04, float((grads["gate"][1] * d).sum())
    assert abs(slope - want) <= 0.1 * abs(want)
    losses = [float(stack.tune(x, target, rate=0.3)) for _ in range(12)]
    assert losses[-1] < losses[0], losses
