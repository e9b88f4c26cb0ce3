"""The forward products of the 8-bit operators on each of their schedules, bit for bit: the sums
are exact integers, and scales and biases that are powers of two leave one rounding."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

D = torch.float64

# gated, M, N, K, tile, split
SCHEDULES = [
    (False, 1, 601, 64, 0, False), (False, 16, 4091, 14336, 0, False), (False, 17, 601, 64, 1, False),
    (False, 3863, 2577, 64, 2, False), (False, 1029, 4101, 4128, 3, False), (False, 1091, 5377, 64, 3, False),
    (False, 327, 5591, 8800, 3, True), (False, 3619, 2073, 64, 4, False), (False, 2047, 4093, 14336, 3, False),
    (False, 8431, 69, 13824, 4, True), (False, 323, 5441, 64, 5, False), (False, 333, 5001, 4128, 5, False),
    (False, 33, 2691, 10880, 5, True), (False, 65, 5483, 64, 6, False), (False, 33, 1357, 7616, 6, True),
    (False, 33, 601, 64, 7, False), (False, 17, 609, 11744, 7, True),
    (True, 1, 601, 64, 1, False), (True, 16, 14331, 4096, 1, False), (True, 841, 5845, 64, 2, False),
    (True, 4095, 14331, 4096, 2, False),
    (True, 581, 4873, 64, 3, False), (True, 65, 4261, 14304, 3, True), (True, 645, 5399, 64, 4, False),
    (True, 8203, 35, 14144, 4, True), (True, 129, 5521, 64, 5, False), (True, 33, 1353, 10272, 5, True),
    (True, 33, 4097, 64, 6, False), (True, 33, 675, 7744, 6, True), (True, 33, 601, 64, 7, False),
    (True, 17, 625, 12192, 7, True), (True, 77, 5003, 2080, 7, False)]


def _powers(g, n, lo, hi):
    return 2.0 ** torch.randint(lo, hi, (n,), generator=g, device="cuda").float()


@pytest.mark.parametrize("gated,M,N,K,tile,split", SCHEDULES)
def test_every_schedule(gated, M, N, K, tile, split):
    import bit_weight_only_offline_amd as Q
    g = torch.Generator(device="cuda")
    g.manual_seed(M + N)
    s = Q.i8_default_schedule(M, N, K, gated)
    assert (s.tile, s.splits > 1) == (tile, split)
    print("forward, schedule", gated, M, N, K, s.tile, s.splits, flush=True)
    # codes of a few units: sums below 2^24 are exact in float32 too
    x = torch.randint(-9, 10, (M, K), generator=g, device="cuda", dtype=torch.int8)
    xs = _powers(g, M, -3, 4)
    parts = []
    for _ in range(2 if gated else 1):
        parts += [torch.randint(-9, 10, (N, K), generator=g, device="cuda", dtype=torch.int8), _powers(g, N, -3, 4)]
    b = _powers(g, 2 * N if gated else N, -2, 3).bfloat16()
    sums = [torch.mm(x.to(D), w.to(D).t().contiguous()) * xs.to(D)[:, None] * ws.to(D) for w, ws in zip(parts[::2], parts[1::2])]
    raw = torch.cat(sums, 1) + b.to(D)
    if not gated:
        pw = Q.pack_channel(*parts)
        assert torch.equal(Q.linear_i8(x, xs, pw, bias=b, out_dtype=torch.float32), raw.float())
        assert torch.equal(Q.linear_i8(x, xs, pw, bias=b), raw.float().bfloat16())
        return
    pw = Q.pack_gated(*parts)
    h, got = Q.gated_i8(x, xs, pw, bias=b, keep_raw=True)
    assert torch.equal(got, raw.float().bfloat16())
    u, z = raw[:, :N], raw[:, N:]
    want = z * torch.special.expit(z) * u
    # the exponential's argument is rounded, and every factor a few times; h once to bf16
    tol = 2.0 ** -8 * want.abs() + (z.abs().clamp(max=100) + 10) * 4 * 2.0 ** -24 * (want.abs() + u.abs() * 2.0 ** -24)
    off = (h.to(D) - want).abs() - tol
    assert float(off.max()) <= 0.0, (float(off.max()), int(off.argmax()))
