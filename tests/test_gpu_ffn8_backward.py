"""What the backward products of the 8-bit operators round, against 64 bits.

The scaled gradients (dy times channel scales; du and dg times theirs) are rounded once on
their way to the matrix cores, to eleven significant bits (`U`, fp16) after their row's
largest value is scaled to 2^14 .. 2^15: a value v of a row with largest value t is off by at
most max(U |v|, 2^-39 t).  Codes are exact, sums are float32 (`E` a term), and a result is
rounded to bf16 (`H`).  Values that need no more than eleven bits give exact sums.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E, H, U = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
D = torch.float64


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _codes(g, rows, cols, lo=-128, hi=128):
    return torch.randint(lo, hi, (rows, cols), generator=g, device="cuda", dtype=torch.int8)


def _signs(g, shape):
    return (2 * torch.randint(0, 2, shape, generator=g, device="cuda") - 1).bfloat16()


def _eleven_bits(g, n):
    """Scales 1 + i / 1024: eleven significant bits."""
    return 1.0 + torch.randint(0, 1024, (n,), generator=g, device="cuda").float() / 1024.0


def _weights(g, N, K, gated, scales, lo, hi):
    """(packed weight, its dequantised rows in 64 bits, up rows before gate rows)."""
    Q = _Q()
    w, s = _codes(g, N, K, lo, hi), scales(g, N)
    if not gated:
        return Q.pack_channel(w, s), w.to(D) * s.to(D)[:, None]
    v, t = _codes(g, N, K, lo, hi), scales(g, N)
    return Q.pack_gated(w, s, v, t), torch.cat([w.to(D) * s.to(D)[:, None], v.to(D) * t.to(D)[:, None]])


SHAPES = [(1, 1, 32), (3, 37, 96), (16, 200, 544), (70, 136, 160), (130, 1000, 416), (300, 329, 288), (520, 520, 1056),
          (700, 1000, 1056), (2100, 520, 2080)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_eleven_bits_are_exact(M, N, K, gated):
    """Gradients of one (gated: through an activation that is the identity at 32, so 32 both
    ways) times eleven-bit scales and small codes of both signs: sums stay far below 2^24 units
    of 2^-10 and so are exact in float32, and the result is the exact one, rounded once."""
    Q, g = _Q(), _gen(M + N)
    pw, w = _weights(g, N, K, gated, _eleven_bits, -8, 8)
    dy = _signs(g, (M, N))
    print("backward, exact", M, N, K, gated, flush=True)
    if gated:
        raw = torch.full((M, 2 * N), 32.0, dtype=torch.bfloat16, device="cuda")
        raw[:, :N] *= _signs(g, (M, N))
        dx, draw = Q.gated_i8_backward(dy, raw, pw)
        dv = torch.cat([32 * dy.to(D), dy.to(D) * raw[:, :N].to(D)], 1)
        assert torch.equal(draw.to(D), dv)
    else:
        dx, dv = Q.linear_i8_backward(dy, pw), dy.to(D)
    assert torch.equal(dx, torch.mm(dv, w).float().bfloat16())


def _close(got, ref, tol, what):
    off = (got.to(D) - ref).abs() - tol
    assert bool(torch.isfinite(got).all()) and float(off.max()) <= 0.0, (what, float(off.max()), int(off.argmax()))


def _tol(v, q, ref):
    """v: scaled gradients [M, n] in 64 bits; q: codes [n, K]."""
    size = torch.mm(v.abs(), q.abs())
    floor = 2.0 ** -39 * v.abs().amax(1, keepdim=True) * q.abs().sum(0)
    return (U + 2 * v.shape[1] * E) * size + floor + H * ref.abs() + 2.0 ** -133


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,N,K", [(5, 2, 64), (33, 64, 96), (150, 38, 160), (600, 24, 544)])
def test_differences_of_like_terms(M, N, K, gated):
    """Channels in pairs of equal codes and opposite gradients, with scales that differ in the
    tenth bit: what is left of each pair is a thousandth of its terms."""
    Q, g = _Q(), _gen(M + N + K)

    def paired(t):
        return t.repeat_interleave(2, 0).contiguous()

    def scales():
        s = paired(torch.exp(torch.randn((N // 2,), generator=g, device="cuda")) * 0.01)
        s[1::2] *= 1.0 + 2.0 ** -10
        return s
    flip = torch.ones(N, device="cuda")
    flip[1::2] = -1
    q, s = paired(_codes(g, N // 2, K)), scales()
    dy = (torch.randn((M, N // 2), generator=g, device="cuda").repeat_interleave(2, 1) * flip).bfloat16()
    print("backward, differences", M, N, K, gated, flush=True)
    if not gated:
        v = dy.to(D) * s.to(D)
        ref = torch.mm(v, q.to(D))
        _close(Q.linear_i8_backward(dy, Q.pack_channel(q, s)), ref, _tol(v, q.to(D), ref), "dx")
        return
    p, t = paired(_codes(g, N // 2, K)), scales()
    raw = torch.randn((M, 2, N // 2), generator=g, device="cuda").repeat_interleave(2, 2).reshape(M, 2 * N).bfloat16()
    dx, _ = Q.gated_i8_backward(dy, raw, Q.pack_gated(q, s, p, t))
    d, u, z = dy.to(D), raw[:, :N].to(D), raw[:, N:].to(D)
    sig = torch.special.expit(z)
    a, da = z * sig, sig + z * sig * torch.special.expit(-z)
    v = torch.cat([d * a * s.to(D), d * u * da * t.to(D)], 1)
    both = torch.cat([q, p]).to(D)
    # of the logistic factors: a few roundings, and that of their argument
    slip = 4 * (z.abs() + 10) * 8 * E * (1 + z.abs()) ** 2
    slip = torch.cat([d.abs() * slip * s.to(D), (d * u).abs() * slip * t.to(D)], 1)
    ref = torch.mm(v, both)
    _close(dx, ref, _tol(v, both, ref) + torch.mm(slip, both.abs()), "dx")


@pytest.mark.parametrize("power", [-126, -90, -30, 0, 30, 100])
def test_rows_of_any_size(power):
    """Rows whose largest gradient is 2^power, and in each row gradients over thirty octaves."""
    Q, g, M, N, K = _Q(), _gen(200 + power), 40, 72, 96
    q = _codes(g, N, K)
    s = torch.exp(torch.randn((N,), generator=g, device="cuda"))
    spread = 2.0 ** -torch.randint(0, 31, (M, N), generator=g, device="cuda").double()
    dy = (torch.randn((M, N), generator=g, device="cuda").double().clamp(-1, 1) * spread * 2.0 ** power).bfloat16()
    v = dy.to(D) * s.to(D)
    ref = torch.mm(v, q.to(D))
    # a scaled gradient below 2^-126 is subnormal in float32, and held to 2^-149
    tol = _tol(v, q.to(D), ref) + 2.0 ** -149 * q.to(D).abs().sum(0)
    _close(Q.linear_i8_backward(dy, Q.pack_channel(q, s)), ref, tol, power)


def test_each_row_has_its_own_scale():
    """Rows 2^80 apart, a row of zeros and rows with infinities and NaN next to each other: each
    is what it is alone, and infinite where the formula is."""
    Q, g, M, N, K = _Q(), _gen(7), 37, 40, 64
    q = _codes(g, N, K, 1, 100)                               # positive: no infinity times zero
    pw = Q.pack_channel(q, torch.exp(torch.randn((N,), generator=g, device="cuda")))
    dy = torch.randn((M, N), generator=g, device="cuda").bfloat16()
    dy[1::3] *= 2.0 ** -40
    dy[2::3] *= 2.0 ** 40
    dy[5], dy[9, 3], dy[10, 7], dy[11, 8] = 0.0, float("inf"), float("-inf"), float("nan")
    dx = Q.linear_i8_backward(dy, pw)
    for m in range(M):
        alone = Q.linear_i8_backward(dy[m:m + 1].clone(), pw)[0]
        assert torch.equal(dx[m].view(torch.int16), alone.view(torch.int16)) or m == 11, m
    assert bool((dx[5] == 0).all()) and bool((dx[9] == float("inf")).all())
    assert bool((dx[10] == float("-inf")).all()) and bool(torch.isnan(dx[11]).all())
    assert bool(torch.isfinite(dx[[m for m in range(M) if m not in (9, 10, 11)]]).all())


@pytest.mark.parametrize("gated,M,N,K", [
    (False, 9, 1021, 64), (False, 3, 6165, 32), (False, 3, 24581, 32), (False, 2, 32941, 5408), (False, 2, 49957, 8224),
    (False, 10875, 51845, 64), (True, 9, 1021, 64), (True, 3, 3077, 32), (True, 3, 12305, 32), (True, 2, 16421, 5440),
    (True, 2, 17157, 12448), (True, 10797, 24917, 32), (False, 5, 5, 32), (True, 5, 3, 32)])
def test_rows_of_every_length(gated, M, N, K):
    """The operand pass takes a row (its part of a split) by 64 to 1024 threads, and in two
    readings where it does not fit in registers; here at odd lengths, with the last channels
    alone non-zero too."""
    Q, g = _Q(), _gen(N)
    pw, w = _weights(g, N, K, gated, _eleven_bits, -2, 2)
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, N, (M, 200), generator=g, device="cuda")
    dy.scatter_(1, at, _signs(g, (M, 200)))
    dy[0] = 0
    dy[0, N - 1], dy[1, N - 1], dy[1, 0] = 1, -1, -1
    print("backward, row length", gated, M, N, K, flush=True)
    if gated:
        raw = torch.full((M, 2 * N), 32.0, dtype=torch.bfloat16, device="cuda")
        raw[:, :N] *= _signs(g, (M, N))
        dx, draw = Q.gated_i8_backward(dy, raw, pw)
        dv = torch.cat([32 * dy.to(D), dy.to(D) * raw[:, :N].to(D)], 1)
        assert torch.equal(draw.to(D), dv)
    else:
        dx, dv = Q.linear_i8_backward(dy, pw), dy.to(D)
    assert torch.equal(dx, torch.mm(dv, w).float().bfloat16())


# Each schedule (tile, split or whole), at row counts off every tile and odd channel counts;
# besides the shortest of each, contractions of a hundred steps and more.
SCHEDULES = [
    (False, 533, 617, 13088, 0, False), (False, 2047, 4093, 14336, 0, False), (False, 131, 4023, 10816, 0, True),
    (False, 2741, 601, 1312, 1, False), (False, 333, 4099, 4096, 1, True), (False, 1031, 4091, 4096, 1, False),
    (False, 2699, 1283, 64, 1, True), (False, 2081, 601, 288, 2, False), (False, 1035, 769, 64, 2, True),
    (False, 3, 601, 64, 3, False), (False, 1, 641, 64, 3, True), (False, 13, 4091, 14336, 3, True),
    (True, 661, 603, 10880, 0, False), (True, 2047, 14331, 4096, 0, True), (True, 2711, 4935, 64, 0, True),
    (True, 3301, 603, 1056, 1, False), (True, 2691, 645, 64, 1, True), (True, 205, 603, 4928, 2, False),
    (True, 673, 653, 64, 2, True), (True, 3647, 605, 96, 3, False), (True, 1, 601, 64, 3, True),
    (True, 77, 5003, 2080, 1, True)]


@pytest.mark.parametrize("gated,M,N,K,tile,split", SCHEDULES)
def test_every_schedule(gated, M, N, K, tile, split):
    Q, g = _Q(), _gen(M + N)
    s = Q.i8_default_schedule(M, N, K, gated, backward=True)
    assert (s.tile, s.splits > 1) == (tile, split)
    pw, w = _weights(g, N, K, gated, _eleven_bits, -8, 8)
    dy = _signs(g, (M, N))
    print("backward, schedule", gated, M, N, K, s.tile, s.splits, flush=True)
    if gated:
        raw = torch.full((M, 2 * N), 32.0, dtype=torch.bfloat16, device="cuda")
        raw[:, :N] *= _signs(g, (M, N))
        dx, draw = Q.gated_i8_backward(dy, raw, pw)
        dv = torch.cat([32 * dy.to(D), dy.to(D) * raw[:, :N].to(D)], 1)
        assert torch.equal(draw.to(D), dv)
    else:
        dx, dv = Q.linear_i8_backward(dy, pw), dy.to(D)
    assert torch.equal(dx, torch.mm(dv, w).float().bfloat16())
