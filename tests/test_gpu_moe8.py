"""Mixture-of-experts operators in 8-bit floating point against plain 64-bit implementations.

Tolerances come from the arithmetic: `E` is the rounding unit of float32, `H` that of bf16, `F` that of e4m3, each at
most half a step relative to the value.  Sums in float32 differ by their length times E of the sum of magnitudes;
a bf16 result by H of itself.  Where all sums are exact in float32, results are compared bit for bit.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe8_reference as R  # noqa: E402

E, H, F = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4
D = torch.float64
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, shape, typical=1.0, dtype=BF):
    return (torch.randn(shape, generator=g, device="cuda") * typical).to(dtype)


def _close(got, ref, tol, what):
    got = got.to(D)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    off = (got - ref).abs() - tol
    assert bool(torch.isfinite(got).all()) and (off.numel() == 0 or float(off.max()) <= 0.0), (what, float(off.max()), int(off.argmax()))


def _same(a, b):
    """Equal values, NaN in the same places."""
    return torch.equal(torch.nan_to_num(a.to(D), 1e30), torch.nan_to_num(b.to(D), 1e30))


# ---- quantisation ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 128), (3, 160), (17, 4096), (5, 14336), (1000, 96), (2, 131040)])
def test_quantize_is_exact(rows, K, dtype):
    Q, g = _Q(), _gen(rows * K)
    x = _randn(g, (rows, K), 2.0, dtype)
    codes, scales = Q.quantize_f8(x)
    ref, s = R.quantize(x)
    assert codes.dtype == F8 and codes.shape == x.shape and scales.shape == (rows, R.blocks(K))
    assert torch.equal(scales.to(D), s)
    assert torch.equal(codes.to(D), ref)


def test_quantize_next_to_borders():
    """Values whose quotient, rounded to float32, would lie on the border between two codes."""
    Q, g = _Q(), _gen(5)
    x = (torch.randint(-2048, 2049, (4096, 1024), generator=g, device="cuda").float() / 64).bfloat16()
    x = torch.where(torch.rand((4096, 1024), generator=g, device="cuda") < 0.5, x, (x * 1.0625).bfloat16())
    codes, scales = Q.quantize_f8(x)
    ref, s = R.quantize(x)
    assert torch.equal(scales.to(D), s) and torch.equal(codes.to(D), ref)


@pytest.mark.parametrize("scale", [1e-44, 3e-42, 1e-38, 1e-30, 1e30, 7e37])
def test_quantize_at_the_ends_of_the_range(scale):
    """Blocks whose scale is subnormal, or nearly float32's largest; codes never leave e4m3's values."""
    Q, g = _Q(), _gen(6)
    x = (torch.randn((8, 256), generator=g, device="cuda", dtype=D).clamp(-4, 4) * scale).float()
    codes, scales = Q.quantize_f8(x)
    ref, s = R.quantize(x)
    assert torch.equal(scales.to(D), s)
    assert bool(torch.isfinite(codes.float()).all()) and torch.equal(codes.to(D), ref)


def test_quantize_special_blocks():
    Q = _Q()
    x = torch.ones((4, 384), device="cuda")
    x[0, :128] = 0.0
    x[1, 5] = float("nan")
    x[2, 130] = float("inf")
    x[3, 300] = -float("inf")
    codes, scales = Q.quantize_f8(x)
    assert scales[0, 0] == 0 and bool((codes[0, :128].float() == 0).all())
    for r, b in ((1, 0), (2, 1), (3, 2)):
        assert bool(torch.isnan(scales[r, b])) and bool((codes[r, 128 * b:128 * b + 128].float() == 0).all())
        others = [i for i in range(3) if i != b]
        assert bool((scales[r, others] == torch.tensor(1 / 448, dtype=D).float().item()).all())
    assert int(torch.isnan(scales).sum()) == 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,K", [(1, 32), (16, 14336), (77, 160)])
def test_quantize_swiglu(rows, K, dtype):
    """|code s - h| is at most half a step of e4m3 (F of the value, or half the least step, 2^-10 s), and h in float32
    differs by the roundings of the logistic function, a few and four times the argument each E of it."""
    Q, g = _Q(), _gen(rows + K)
    x = _randn(g, (rows, 2 * K), 2.0, dtype)
    codes, scales = Q.quantize_f8(x, act="swiglu")
    up, gate = x.to(D).chunk(2, 1)
    h = up * gate * torch.special.expit(gate)
    d = (16 + 4 * gate.abs()) * E
    s = R.spread_rows(scales, K)
    _close(codes.to(D) * s, h, F * h.abs() * (1 + 2 * d) + s * 2.0 ** -10 + d * h.abs(), "swiglu")
    _, sref = R.quantize(h)
    worst = float(d.max())
    assert float((scales.to(D) / sref - 1).abs().max()) <= worst + 2 * E


@pytest.mark.parametrize("rows,K", [(1, 32), (16, 14336), (300, 416)])
def test_quantize_backward(rows, K):
    Q, g = _Q(), _gen(rows + K + 1)
    raw, dh = _randn(g, (rows, 2 * K), 2.0), _randn(g, (rows, K))
    got = Q.quantize_f8_backward(dh, raw)
    leaf = raw.to(D).requires_grad_()
    up, gate = leaf.chunk(2, 1)
    (up * gate * torch.special.expit(gate) * dh.to(D)).sum().backward()
    up, gate, p = up.detach(), gate.detach(), torch.special.expit(gate.detach())
    d = (16 + 4 * gate.abs()) * E
    size = torch.cat([dh.to(D) * gate * p, dh.to(D) * up * (p + gate.abs() * p * (1 - p))], 1).abs()
    _close(got, leaf.grad, H * leaf.grad.abs() + torch.cat([d, d], 1) * size, "draw")
    # differences of the function
    eps, dx = 1e-6, _randn(g, (rows, 2 * K), 1.0, D)
    def f(x):
        u, v = x.chunk(2, 1)
        return u * v * torch.special.expit(v)
    slope = ((f(raw.to(D) + eps * dx) - f(raw.to(D) - eps * dx)) / (2 * eps) * dh.to(D)).sum()
    size = float((leaf.grad.abs() * dx.abs()).sum())
    assert abs(float((got.to(D) * dx).sum() - slope)) <= (H + 1e-6) * size


def test_dequantize_and_weights():
    Q, g = _Q(), _gen(9)
    for shape in ((1, 32), (130, 160), (3, 257, 288)):
        for dtype in (BF, F32):
            w = _randn(g, shape, 0.02, dtype)
            codes, scales = Q.quantize_weight_f8(w)
            N, K = shape[-2:]
            full = torch.zeros((*shape[:-2], R.blocks(N) * 128, R.blocks(K) * 128), dtype=D, device="cuda")
            full[..., :N, :K] = w.to(D)
            tiles = full.reshape(*shape[:-2], R.blocks(N), 128, R.blocks(K), 128)
            s = (tiles.abs().amax((-3, -1)) / 448).float()
            assert torch.equal(scales, s)
            ref = R.round_e4m3(w.to(D) / R.spread_weight(s, N, K))
            assert torch.equal(codes.to(D), ref)
    x = _randn(g, (5, 7, 160))
    codes, scales = Q.quantize_f8(x)
    ref = codes.to(D) * R.spread_rows(scales, 160)
    assert torch.equal(Q.dequantize_f8(codes, scales, F32).to(D), ref.float().to(D))
    assert torch.equal(Q.dequantize_f8(codes, scales), ref.float().bfloat16())


@pytest.mark.parametrize("shape", [(1, 32), (17, 96), (3, 130, 288), (16, 128)])
def test_pack_round_trip(shape):
    Q, g = _Q(), _gen(sum(shape))
    codes, scales = R.weights(g, shape)
    pw = Q.pack_f8(codes, scales)
    back, s = Q.unpack_f8(pw)
    assert torch.equal(back.view(torch.uint8), codes.view(torch.uint8)) and torch.equal(s, scales)
    scales.zero_()
    assert not torch.equal(pw.s, scales)                      # a copy


# ---- products --------------------------------------------------------------------------

SHAPES = [(1, 32), (19, 160), (200, 736), (516, 2080)]


def _product_tol(x, xs, w, ws):
    """Sum of magnitudes, and how many roundings a sum in float32 has: those inside a block, of the blocks, of a split
    and of the scales."""
    K = x.shape[-1]
    size = (x.to(D).abs() * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).abs().transpose(-1, -2)
    return size * (128 + R.blocks(K) + 16) * E


def _group_tol(x, xs, w, ws):
    """The 8-bit matrix cores, which products to bf16 go through, drop what lies below 2^-13 of the largest of eight
    products: less than 2^-13 of it for each of the seven others, so 7 2^-13 of the group's sum of magnitudes."""
    return _product_tol(x, xs, w, ws) / ((128 + R.blocks(x.shape[-1]) + 16) * E) * 7 * 2.0 ** -13


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 65, 100, 129, 300, 513])
@pytest.mark.parametrize("N,K", SHAPES)
def test_linear(M, N, K):
    Q, g = _Q(), _gen(M * N + K)
    x, xs = R.activations(g, M, K)
    w, ws = R.weights(g, (N, K))
    b = _randn(g, (N,))
    pw = Q.pack_f8(w, ws)
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t()
    tol = _product_tol(x, xs, w, ws)
    y = Q.linear_f8(x, xs, pw, out_dtype=F32)
    _close(y, ref, tol, "no bias")
    y32 = Q.linear_f8(x, xs, pw, bias=b, out_dtype=F32)
    _close(y32, ref + b.to(D), tol + E * (ref + b.to(D)).abs(), "bias")
    y16 = Q.linear_f8(x, xs, pw, bias=b)
    if M <= 16:
        assert torch.equal(y16, y32.bfloat16())                # the same sums, rounded once
    ref = ref + b.to(D)
    _close(y16, ref, (tol + _group_tol(x, xs, w, ws)) * (1 + H) + H * ref.abs(), "bf16")
    if M * N > 1000:                                           # and on average as its type allows
        assert float((y16.to(D) - ref).norm() / ref.norm()) <= 1.01 * float((ref.bfloat16().to(D) - ref).norm() / ref.norm()) + 1e-4
    assert torch.equal(Q.linear_f8(x, xs, pw, out_dtype=F32), y)


@pytest.mark.parametrize("M", [1, 16, 40, 100, 300])
@pytest.mark.parametrize("N,K", SHAPES)
def test_linear_exact(M, N, K):
    """Small whole numbers and scales that are powers of two: every sum is exact, in any order."""
    Q, g = _Q(), _gen(M + N + K)
    x, xs = R.activations(g, M, K, True)
    w, ws = R.weights(g, (N, K), True)
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t()
    assert torch.equal(Q.linear_f8(x, xs, Q.pack_f8(w, ws), out_dtype=F32).to(D), ref)


SCHEDULED = [(5, 300, 1184), (5, 9000, 288), (2048, 4096, 416), (2048, 4096, 1184), (1000, 4096, 1184), (333, 5001, 544),
             (100, 5000, 4128), (200, 4100, 544), (40, 3000, 416), (35, 8297, 9408), (33, 4281, 9440), (1119, 66, 8160),
             (33, 2301, 10304), (612, 67, 7424), (663, 68, 7776), (17, 73, 6592), (23, 112, 12320), (18, 69, 7520), (36, 4638, 28448),
             (4500, 2080, 160)]


@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_schedule_is_among_these(dtype):
    """All tiles, and all but the few-row kernels and the largest tiles also in splits."""
    Q = _Q()
    seen = {(s.tile, s.splits > 1) for s in (Q.f8_default_schedule(*c, out_dtype=dtype) for c in SCHEDULED)}
    assert seen == {(t, False) for t in range(8)} | {(t, True) for t in range(3, 8)}, sorted(seen)


@pytest.mark.parametrize("M,N,K", SCHEDULED)
def test_schedules_exact(M, N, K):
    Q, g = _Q(), _gen(M + N + K)
    x, xs = R.activations(g, M, K, True)
    w, ws = R.weights(g, (N, K), True)
    b = torch.randint(-4, 5, (N,), generator=g, device="cuda").bfloat16()
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t() + b.to(D)
    pw = Q.pack_f8(w, ws)
    assert torch.equal(Q.linear_f8(x, xs, pw, bias=b, out_dtype=F32).to(D), ref)
    assert torch.equal(Q.linear_f8(x, xs, pw, bias=b), ref.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(2100, 4100, 1184), (2750, 4100, 1184), (4700, 4096, 288 * 4 + 32), (2100, 4097, 2080)])
def test_last_rounds_exact(M, N, K):
    """Tiles of 128 x 256 in rounds whose last is cut in two or in four, row and column ends inside the parts."""
    Q, g = _Q(), _gen(M + N + K)
    tiles = -(-M // 128) * -(-N // 256)
    assert 0 < tiles // 8 % 32 <= 15 and Q.f8_default_schedule(M, N, K, out_dtype=F32).tile == 2
    x, xs = R.activations(g, M, K, True)
    w, ws = R.weights(g, (N, K), True)
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t()
    pw = Q.pack_f8(w, ws)
    assert torch.equal(Q.linear_f8(x, xs, pw, out_dtype=F32).to(D), ref)
    assert torch.equal(Q.linear_f8(x, xs, pw), ref.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [(4096, 4090, 1184), (4500, 4100, 800), (5000, 4100, 1184), (8300, 2052, 1184), (4700, 4096, 1184)])
def test_tall_tiles_exact(M, N, K):
    """Tiles of 256 x 256: whole rounds, a last one cut in two or in four, a last block of at most half the rows."""
    Q, g = _Q(), _gen(M + N + K)
    assert Q.f8_default_schedule(M, N, K).tile == 8
    x, xs = R.activations(g, M, K, True)
    w, ws = R.weights(g, (N, K), True)
    b = torch.randint(-4, 5, (N,), generator=g, device="cuda").bfloat16()
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t() + b.to(D)
    out = torch.full((M + 3, N), 7.0, device="cuda", dtype=BF)
    assert torch.equal(Q.linear_f8(x, xs, Q.pack_f8(w, ws), bias=b, out=out[:M]), ref.float().bfloat16())
    assert bool((out[M:] == 7.0).all())


def test_tall_tiles_against_64_bits():
    Q, M, N, K = _Q(), 4500, 4100, 1184
    g = _gen(8)
    assert Q.f8_default_schedule(M, N, K).tile == 8
    x, xs = R.activations(g, M, K)
    w, ws = R.weights(g, (N, K))
    ref = (x.to(D) * R.spread_rows(xs, K)) @ R.dense_weight(w, ws).t()
    tol = _product_tol(x, xs, w, ws) + _group_tol(x, xs, w, ws)
    _close(Q.linear_f8(x, xs, Q.pack_f8(w, ws)), ref, tol * (1 + H) + H * ref.abs(), "tall")


@pytest.mark.parametrize("counts,tile", [([900, 13, 1200, 87], 2), ([1, 0, 1900, 300], 2), ([550, 550, 550, 550], 2),
                                         ([4000, 100, 300, 130], 8), ([2300, 0, 2300, 1], 8), ([1200, 1100, 1300, 1250], 8)])
def test_grouped_last_rounds_exact(counts, tile):
    Q, N, K, T = _Q(), 4100, 1184, sum(counts)
    g = _gen(T)
    assert Q.f8_default_schedule(T, N, K, 4).tile == tile
    x, xs = R.activations(g, T, K, True)
    w, ws = R.weights(g, (4, N, K), True)
    out = torch.full((T + 5, N), 7.0, device="cuda", dtype=BF)
    y = Q.grouped_linear_f8(x, xs, Q.pack_f8(w, ws), torch.tensor(counts, dtype=torch.int32, device="cuda"), out=out[:T])
    at = 0
    for e, c in enumerate(counts):
        ref = (x[at:at + c].to(D) * R.spread_rows(xs[at:at + c], K)) @ R.dense_weight(w[e], ws[e]).t()
        assert torch.equal(y[at:at + c], ref.float().bfloat16()), e
        at += c
    assert bool((out[T:] == 7.0).all())


def test_nan_stays_in_its_row_and_channel():
    """A NaN code, or scale, reaches its own row or channel alone: also where a row ends inside a block and the next
    row begins with NaN."""
    Q = _Q()
    for M, N, K in ((5, 40, 160), (40, 200, 160), (300, 260, 96)):
        g = _gen(M)
        x, xs = R.activations(g, M, K, True)
        w, ws = R.weights(g, (N, K), True)
        pw = Q.pack_f8(w, ws)
        clean = Q.linear_f8(x, xs, pw, out_dtype=F32)
        bad = x.clone()
        bad.view(torch.uint8)[3, :40] = 0x7F
        y = Q.linear_f8(bad, xs, pw, out_dtype=F32)
        assert bool(torch.isnan(y[3]).all())
        keep = [m for m in range(M) if m != 3]
        assert torch.equal(y[keep], clean[keep])
        s2 = xs.clone()
        s2[2, 0] = float("nan")
        y = Q.linear_f8(x, s2, pw, out_dtype=F32)
        assert bool(torch.isnan(y[2]).all()) and int(torch.isnan(y).sum()) == N
        w2 = w.clone()
        w2.view(torch.uint8)[7, K - 1] = 0xFF
        y = Q.linear_f8(x, xs, Q.pack_f8(w2, ws), out_dtype=F32)
        assert bool(torch.isnan(y[:, 7]).all()) and int(torch.isnan(y).sum()) == M


COUNTS = [[3, 0, 5, 1], [0, 0, 0, 17], [16, 16, 16, 16], [40, 1, 0, 200], [130, 300, 129, 1], [0, 0, 0, 0], [1]]


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(19, 160), (300, 416)])
def test_grouped(counts, N, K):
    Q, X, T = _Q(), len(counts), sum(counts)
    g = _gen(T + N)
    x, xs = R.activations(g, T, K)
    w, ws = R.weights(g, (X, N, K))
    b = _randn(g, (X, N))
    pw = Q.pack_f8(w, ws)
    cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
    y32 = Q.grouped_linear_f8(x, xs, pw, cnt, bias=b, out_dtype=F32)
    y16 = Q.grouped_linear_f8(x, xs, pw, cnt, bias=b)
    assert y32.shape == (T, N)
    plain = Q.grouped_linear_f8(x, xs, pw, cnt, out_dtype=F32)
    at = 0
    for e, c in enumerate(counts):
        r = slice(at, at + c)
        ref = (x[r].to(D) * R.spread_rows(xs[r], K)) @ R.dense_weight(w[e], ws[e]).t()
        tol = _product_tol(x[r], xs[r], w[e], ws[e])
        _close(plain[r], ref, tol, f"expert {e}")
        ref = ref + b[e].to(D)
        _close(y32[r], ref, tol + E * ref.abs(), f"expert {e} with bias")
        _close(y16[r], ref, (tol + _group_tol(x[r], xs[r], w[e], ws[e])) * (1 + H) + H * ref.abs(), f"expert {e} to bf16")
        at += c


def test_grouped_many_experts():
    """More experts than a wavefront has lanes; most without rows."""
    Q, X, N, K = _Q(), 300, 40, 96
    for most in (3, 40):
        g = _gen(most)
        counts = [(i * 7) % most if i % 3 == 0 else 0 for i in range(X)]
        T = sum(counts)
        x, xs = R.activations(g, T, K, True)
        w, ws = R.weights(g, (X, N, K), True)
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        y = Q.grouped_linear_f8(x, xs, Q.pack_f8(w, ws), cnt, out_dtype=F32)
        expert = torch.repeat_interleave(torch.arange(X, device="cuda"), cnt)
        dense = R.dense_weight(w, ws)[expert]
        ref = torch.bmm(dense, (x.to(D) * R.spread_rows(xs, K))[:, :, None])[:, :, 0]
        assert torch.equal(y.to(D), ref)


@pytest.mark.parametrize("T", [20, 400])
def test_grouped_clips_and_leaves_rows(T):
    Q, N, K = _Q(), 48, 160
    g = _gen(T)
    x, xs = R.activations(g, T, K, True)
    w, ws = R.weights(g, (4, N, K), True)
    pw, dw = Q.pack_f8(w, ws), R.dense_weight(w, ws)
    xd = x.to(D) * R.spread_rows(xs, K)
    for counts, owned in (([5, -7, 6, 0], [5, 0, 6, 0]), ([T, 5, 5, 5], [T, 0, 0, 0]), ([T - 3, 2 ** 31 - 1, 9, 9], [T - 3, 3, 0, 0]),
                          ([0, 0, 0, 0], [0, 0, 0, 0])):
        cnt = torch.tensor(counts, dtype=torch.int32, device="cuda")
        out = torch.full((T, N), 7.0, device="cuda")
        assert Q.grouped_linear_f8(x, xs, pw, cnt, out_dtype=F32, out=out) is out
        dx = torch.full((T, K), 7.0, device="cuda", dtype=BF)
        dy = torch.randint(-3, 4, (T, N), generator=g, device="cuda").bfloat16()
        Q.grouped_linear_f8_backward(dy, pw, cnt, out=dx)
        at = 0
        for e, c in enumerate(owned):
            assert torch.equal(out[at:at + c].to(D), xd[at:at + c] @ dw[e].t()), (counts, e)
            ref = dy[at:at + c].to(D) @ dw[e]
            assert torch.equal(dx[at:at + c], ref.float().bfloat16()), (counts, e)
            at += c
        assert bool((out[at:] == 7.0).all()) and bool((dx[at:] == 7.0).all())


# ---- backward products -----------------------------------------------------------------

@pytest.mark.parametrize("M", [1, 15, 16, 17, 64, 100, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 32), (19, 160), (200, 736), (516, 2080), (1031, 320)])
def test_linear_backward(M, N, K):
    """Products are exact, sums of N in float32; between two channel blocks the running sums are multiplied by a
    ratio (a division and a product, two roundings), and at the end by the last scale."""
    Q, g = _Q(), _gen(M + N + K)
    w, ws = R.weights(g, (N, K))
    dy = _randn(g, (M, N))
    dense = R.dense_weight(w, ws)
    ref = dy.to(D) @ dense
    tol = (dy.to(D).abs() @ dense.abs()) * (N + 2 * R.blocks(N) + 16) * E + H * ref.abs()
    got = Q.linear_f8_backward(dy, Q.pack_f8(w, ws))
    _close(got, ref, tol, "dx")
    # against differences: the product is linear in its input
    dx = _randn(g, (M, K), 1.0, D)
    slope = float(((dx @ dense.t()) * dy.to(D)).sum())
    assert abs(float((got.to(D) * dx).sum()) - slope) <= float((tol * dx.abs()).sum())


BACK_SCHEDULED = [(5, 300, 288), (1000, 300, 4160), (3000, 260, 4160), (240, 236, 24608), (1691, 1179, 8512), (6876, 4991, 544),
                  (402, 5013, 3456), (387, 2658, 960), (17, 4746, 192), (9000, 40, 2080)]


def test_every_backward_schedule_is_among_these():
    """All tiles, whole and in splits."""
    Q = _Q()
    seen = {(s.tile, s.splits > 1) for s in (Q.f8_default_schedule(*c, backward=True) for c in BACK_SCHEDULED)}
    assert seen == {(t, split) for t in range(4) for split in (False, True)}, sorted(seen)


@pytest.mark.parametrize("M,N,K", BACK_SCHEDULED)
def test_backward_schedules_exact(M, N, K):
    Q, g = _Q(), _gen(M + N + K)
    w, ws = R.weights(g, (N, K), True)
    dy = torch.randint(-4, 5, (M, N), generator=g, device="cuda").bfloat16()
    ref = dy.to(D) @ R.dense_weight(w, ws)
    got = Q.linear_f8_backward(dy, Q.pack_f8(w, ws))
    assert torch.equal(got, ref.float().bfloat16())


@pytest.mark.parametrize("counts", COUNTS)
@pytest.mark.parametrize("N,K", [(19, 160), (300, 416)])
def test_grouped_backward(counts, N, K):
    Q, X, T = _Q(), len(counts), sum(counts)
    g = _gen(T + N + 1)
    w, ws = R.weights(g, (X, N, K))
    dy = _randn(g, (T, N))
    got = Q.grouped_linear_f8_backward(dy, Q.pack_f8(w, ws), torch.tensor(counts, dtype=torch.int32, device="cuda"))
    at = 0
    for e, c in enumerate(counts):
        d = dy[at:at + c].to(D)
        dense = R.dense_weight(w[e], ws[e])
        ref = d @ dense
        _close(got[at:at + c], ref, (d.abs() @ dense.abs()) * (N + 2 * R.blocks(N) + 16) * E + H * ref.abs(), f"expert {e}")
        at += c


def test_backward_scales_of_every_size():
    """Channel blocks with the scales 0, negative, subnormal, tiny and huge ones beside each other: blocks with the
    scale 0 add nothing, and no ratio of scales overflows."""
    Q, g = _Q(), _gen(3)
    N, K, M = 128 * 8, 160, 40
    w, _ = R.weights(g, (N, K))
    col = torch.tensor([0.0, 1e-30, 3e4, 0.0, -2.5e-3, 1e-36, 1.7, 0.0], device="cuda")
    ws = col[:, None].expand(8, 2).contiguous()
    ws[:, 1] = col.flip(0)
    dy = _randn(g, (M, N))
    dense = R.dense_weight(w, ws)
    ref = dy.to(D) @ dense
    tol = (dy.to(D).abs() @ dense.abs()) * (N + 32) * E + H * ref.abs()
    _close(Q.linear_f8_backward(dy, Q.pack_f8(w, ws)), ref, tol, "scales")
    zero = Q.linear_f8_backward(dy, Q.pack_f8(w, torch.zeros_like(ws)))
    assert bool((zero == 0).all())
    nan = ws.clone()
    nan[3, 1] = float("nan")
    got = Q.linear_f8_backward(dy, Q.pack_f8(w, nan))
    assert bool(torch.isnan(got[:, 128:]).all()) and bool(torch.isfinite(got[:, :128]).all())


def test_backward_nan_rows():
    """A row of dy with NaN or infinity stays a row of dx; also where rows end inside a stage."""
    Q, g = _Q(), _gen(4)
    for M, N in ((20, 40), (200, 72), (50, 45)):
        w, ws = R.weights(g, (N, 96), True)
        dy = torch.randint(-4, 5, (M, N), generator=g, device="cuda").bfloat16()
        pw = Q.pack_f8(w, ws)
        clean = Q.linear_f8_backward(dy, pw)
        bad = dy.clone()
        bad[4, :9] = float("nan")
        bad[11, 0] = float("inf")
        got = Q.linear_f8_backward(bad, pw)
        keep = [m for m in range(M) if m not in (4, 11)]
        assert bool(torch.isnan(got[4]).all()) and not bool(torch.isfinite(got[11]).all()) and torch.equal(got[keep], clean[keep])


# ---- expert order ----------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,k,X", [(1, 1, 1), (1, 8, 8), (16, 2, 8), (7, 3, 5), (100, 6, 60), (1000, 8, 256), (2048, 8, 64),
                                   (5000, 4, 1024), (4099, 6, 60), (30000, 3, 7), (70000, 2, 1000), (16385, 1, 3)])
def test_order(T, k, X, dtype):
    Q, g = _Q(), _gen(T + k + X)
    ids = torch.randint(-1 if T % 2 else 0, X, (T, k), generator=g, device="cuda").to(dtype)
    if T > 100:
        ids[T // 2:T // 2 + 40] = X - 1                       # a run
        ids[5, 0] = X                                         # past the last
    if dtype == torch.int64 and T > 100:
        ids[6, 0] = (1 << 40) + 1                             # past 32 bits
    order = Q.expert_order(ids, X)
    counts, rows, source = R.order(ids.cpu(), X)
    assert torch.equal(order.counts.cpu(), counts) and torch.equal(order.rows.cpu(), rows)
    assert torch.equal(order.source.cpu(), source)


def test_order_of_nothing():
    Q = _Q()
    order = Q.expert_order(torch.empty((0, 4), dtype=torch.int64, device="cuda"), 9)
    assert order.counts.tolist() == [0] * 9 and order.rows.shape == (0, 4)
    x = torch.empty((0, 64), device="cuda")
    assert Q.dispatch_tokens(x, order).shape == (0, 64)
    assert Q.combine_tokens(x, order).shape == (0, 64)


def _routed(g, T, k, X, drop):
    ids = torch.randint(0, X, (T, k), generator=g, device="cuda")
    if drop:
        ids = torch.where(torch.rand((T, k), generator=g, device="cuda") < 0.3, -1, ids)
    return ids


ROWS = [(1, 1, 1, 8), (1, 2, 8, 65), (16, 2, 8, 4096), (33, 8, 12, 1000), (200, 5, 60, 5000), (9, 9, 3, 7), (600, 3, 4, 96),
        (5, 2, 3, 1), (3, 70, 80, 130)]


@pytest.mark.parametrize("drop", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,k,X,width", ROWS)
def test_dispatch_and_combine(T, k, X, width, dtype, drop):
    Q, g = _Q(), _gen(T + k + width)
    ids = _routed(g, T, k, X, drop)
    order = Q.expert_order(ids, X)
    rows, total = order.rows.long(), int(order.counts.sum())
    x = _randn(g, (T, width), 1.0, dtype)
    out = torch.full((T * k, width), 7.0, dtype=dtype, device="cuda")
    assert Q.dispatch_tokens(x, order, out=out) is out
    token = order.source[:total].long() // k
    assert torch.equal(out[:total], x[token]) and bool((out[total:] == 7.0).all())

    y = _randn(g, (T * k, width), 1.0, dtype)
    y[total:] = float("nan")                                  # what no slot names is not read
    w = torch.softmax(torch.randn((T, k), generator=g, device="cuda"), 1)
    real = (rows >= 0)[..., None]
    picked = torch.where(real, y[rows.clamp_min(0)].to(D), 0.0)
    half = H if dtype == BF else E
    ref = (picked * w.to(D)[..., None]).sum(1)
    size = (picked.abs() * w.to(D)[..., None]).sum(1)
    _close(Q.combine_tokens(y, order, w), ref, half * ref.abs() + (k + 1) * E * size, "combine")
    ref = picked.sum(1)
    _close(Q.dispatch_tokens_backward(y, order), ref, half * ref.abs() + (k + 1) * E * picked.abs().sum(1), "dispatch backward")

    dout = _randn(g, (T, width), 1.0, dtype)
    dy = torch.full((T * k, width), 7.0, dtype=dtype, device="cuda")
    got, dw = Q.combine_tokens_backward(dout, y, order, w, out=dy)
    assert got is dy and bool((dy[total:] == 7.0).all())
    flat = order.source[:total].long()
    ref = w.reshape(-1)[flat].to(D)[:, None] * dout.to(D)[token]
    _close(dy[:total], ref, half * ref.abs() + E * ref.abs(), "dy")
    prod = picked * dout.to(D)[:, None]
    _close(dw, prod.sum(2), (width + 1) * E * prod.abs().sum(2), "dw")
    assert bool((dw[rows < 0] == 0).all())


@pytest.mark.parametrize("T,k,X,width", [(16, 2, 8, 4096), (33, 8, 12, 160), (5, 3, 4, 32), (700, 2, 3, 288)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dispatch_quantised(T, k, X, width, dtype):
    """Bit for bit the quantised rows in expert order."""
    Q, g = _Q(), _gen(T + width)
    order = Q.expert_order(_routed(g, T, k, X, True), X)
    total = int(order.counts.sum())
    x = _randn(g, (T, width), 1.0, dtype)
    codes, scales = Q.dispatch_tokens(x, order, f8=True)
    c, s = Q.quantize_f8(x)
    token = order.source[:total].long() // k
    assert torch.equal(codes[:total].view(torch.uint8), c.view(torch.uint8)[token]) and torch.equal(scales[:total], s[token])


def test_combine_gradients_against_differences():
    """combine is linear in its rows and in its weights: differences of float32 outputs over powers of two."""
    Q, g = _Q(), _gen(8)
    T, k, X, width = 20, 3, 5, 64
    order = Q.expert_order(_routed(g, T, k, X, True), X)
    total = int(order.counts.sum())
    y = _randn(g, (T * k, width), 1.0, F32)
    w = torch.rand((T, k), generator=g, device="cuda")
    dout = _randn(g, (T, width), 1.0, F32)
    dy, dw = Q.combine_tokens_backward(dout, y, order, w)
    ey, ew = _randn(g, y.shape, 1.0, F32), _randn(g, w.shape, 1.0, F32)
    def f(y, w):
        return float((Q.combine_tokens(y, order, w).to(D) * dout.to(D)).sum())
    size = float(dout.abs().to(D).sum()) * 40 * E * 8
    assert abs((f(y + ey, w) - f(y - ey, w)) / 2 - float((dy[:total].to(D) * ey[:total].to(D)).sum())) <= size
    assert abs((f(y, w + ew) - f(y, w - ew)) / 2 - float((dw.to(D) * ew.to(D)).sum())) <= size


# ---- a layer ---------------------------------------------------------------------------

@pytest.mark.parametrize("T", [3, 200])
def test_layer_forward_and_backward(T):
    """All of them together, each step against the formula on the previous step's own output."""
    Q, g = _Q(), _gen(T)
    X, k, width, hidden = 6, 2, 160, 288
    wu, su = Q.quantize_weight_f8(_randn(g, (X, 2 * hidden, width), width ** -0.5))
    wd, sd = Q.quantize_weight_f8(_randn(g, (X, width, hidden), hidden ** -0.5))
    up_gate, down = Q.pack_f8(wu, su), Q.pack_f8(wd, sd)
    x = _randn(g, (T, width))
    top, ids = torch.topk(torch.randn((T, X), generator=g, device="cuda"), k, dim=1)
    w = torch.softmax(top, 1)

    order = Q.expert_order(ids, X)
    codes, scales = Q.dispatch_tokens(x, order, f8=True)
    raw = Q.grouped_linear_f8(codes, scales, up_gate, order.counts)
    h, hs = Q.quantize_f8(raw, act="swiglu")
    out = Q.grouped_linear_f8(h, hs, down, order.counts)
    y = Q.combine_tokens(out, order, w)
    dy = _randn(g, (T, width))
    dout, dw = Q.combine_tokens_backward(dy, out, order, w)
    dh = Q.grouped_linear_f8_backward(dout, down, order.counts)
    draw = Q.quantize_f8_backward(dh, raw)
    dsorted = Q.grouped_linear_f8_backward(draw, up_gate, order.counts)
    dx = Q.dispatch_tokens_backward(dsorted, order)

    # the whole in 64 bits, from the same quantised values
    xs = (codes.to(D) * R.spread_rows(scales, width)).requires_grad_()
    expert = torch.repeat_interleave(torch.arange(X, device="cuda"), order.counts)
    U, Dn = R.dense_weight(wu, su)[expert], R.dense_weight(wd, sd)[expert]
    u, v = torch.bmm(U, xs[:, :, None])[:, :, 0].chunk(2, 1)
    act = u * v * torch.special.expit(v)
    quant = h.to(D) * R.spread_rows(hs, hidden)
    act = act + (quant - act).detach()                        # straight through
    o = torch.bmm(Dn, act[:, :, None])[:, :, 0]
    o.retain_grad()
    wl = w.to(D).requires_grad_()
    ref = (o[order.rows.long()] * wl[..., None]).sum(1)
    (ref * dy.to(D)).sum().backward()
    def rel(a, b):
        return float((a.to(D) - b).norm() / b.norm())
    # each bf16 result adds at most H of relative error; the steps in a row add up
    assert rel(y, ref.detach()) <= 3 * H
    assert rel(dw, wl.grad) <= 3 * H
    assert rel(dout, o.grad) <= 2 * H
    dx_ref = xs.grad[order.rows.long()].sum(1)
    assert rel(dx, dx_ref) <= 10 * H
