"""Backward products through weights whose scales lie anywhere in float32's range.

Gradients are chosen so that every block's contribution is of the size of the others, or is the only one: a block that is
lost, doubled or of the wrong sign is then as large an error as any.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe8_reference as R  # noqa: E402

E, H = 2.0 ** -24, 2.0 ** -8
D = torch.float64
BF = torch.bfloat16

# Exponents of the blocks' scales, both signs: the least subnormal, the ends of the subnormal and the normal range, those
# on either side of where a code times the scale would leave bf16's normal values, and ordinary ones between them.
POWERS = [0, -149, 127, -12, -127, 126, -126, 3, 120, -118, 119, -117, -30, 125, -140, 0, 118, -116, 60, -60, -133, 1]
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _blocks_of(v):
    """A value a block of 128 channels, spread over the channels."""
    return v.repeat_interleave(R.B)


# Every tile, channels in one piece and split where there are sizes that do so.
TILES = [(3, True), (3, False), (2, True), (2, False), (1, True), (1, False), (0, False)]


def _size(tile, split, nb):
    """The least product of nb channel blocks that takes this tile."""
    Q = _Q()
    sizes = sorted(((M, K) for M in (17, 40, 160, 387, 700, 1000, 1400, 2000, 3000, 3500, 5000, 7000)
                    for K in (96, 160, 288, 544, 1184, 2080, 3456, 4160)), key=lambda c: c[0] * c[1])
    for M, K in sizes:
        s = Q.f8_default_schedule(M, R.B * nb, K, backward=True)
        if (s.tile, s.splits > 1) == (tile, split):
            return M, K
    raise AssertionError(f"no size takes tile {tile}")


@pytest.mark.parametrize("tile,split", TILES)
def test_each_block_by_itself(tile, split):
    """Powers of two and whole numbers: the result is exact, whatever scales come before and after the block's own."""
    nb = len(POWERS)
    M, K = _size(tile, split, nb)
    Q, g = _Q(), _gen(M)
    sign = torch.where(torch.arange(nb) % 3 == 1, -1.0, 1.0).double()
    col = (torch.exp2(torch.tensor(POWERS, dtype=D)) * sign).float().cuda()
    assert torch.equal(col.to(D).abs(), torch.exp2(torch.tensor(POWERS, dtype=D, device="cuda")))
    w, _ = R.weights(g, (nb * R.B, K), True)
    ws = torch.stack([col.roll(j) for j in range(R.blocks(K))], 1).contiguous()
    pw, whole = Q.pack_f8(w, ws), w.to(D)
    base = torch.randint(1, 5, (M, R.B), generator=g, device="cuda").to(D) * torch.where(
        torch.rand((M, R.B), generator=g, device="cuda") < 0.5, -1.0, 1.0).to(D)
    for b in range(nb):
        # Gradients for the first column block's scale, held to bf16's range; the others have other scales.  Results are
        # compared where float32 holds every partial sum, whose bound is the sum of magnitudes, in units of every scale
        # of a column, 2^-25 to 2^9, as a normal number: in the others float32 itself over- or underflows (2^112 times 8 times a
        # scale of 2^127, with both signs, sums to NaN whatever the exact sum is).
        p = float(max(-112, min(112, -POWERS[b])))
        dy = torch.zeros((M, nb * R.B), dtype=D, device="cuda")
        dy[:, b * R.B:(b + 1) * R.B] = base * 2.0 ** p
        part = dy[:, b * R.B:(b + 1) * R.B] @ whole[b * R.B:(b + 1) * R.B]
        ref = part * R.spread_rows(ws[b:b + 1], K)
        got = Q.linear_f8_backward(dy.to(BF), pw).to(D)
        size = dy[:, b * R.B:(b + 1) * R.B].abs() @ whole[b * R.B:(b + 1) * R.B].abs() * R.spread_rows(ws[b:b + 1].abs(), K)
        ok = ((ref == 0) | (ref.abs() >= 2.0 ** -110)) & (size < 2.0 ** 102)
        assert bool(ok.any()), b
        want = ref.float().to(BF).to(D)
        bad = (got != want) & ok
        assert not bool(bad.any()), (b, POWERS[b], got[bad][:4].tolist(), want[bad][:4].tolist())


@pytest.mark.parametrize("tile,split", TILES)
def test_all_blocks_together(tile, split):
    """Scales of any mantissa, a block's gradients by the inverse of its scale."""
    powers = [p for p in POWERS if -126 <= p <= 120]
    nb = len(powers)
    M, K = _size(tile, split, nb)
    Q, g = _Q(), _gen(M + 1)
    mant = 1.0 + torch.rand((nb, R.blocks(K)), generator=g, device="cuda", dtype=D) * 0.99
    mant *= torch.where(torch.rand(mant.shape, generator=g, device="cuda") < 0.4, -1.0, 1.0)
    power = torch.exp2(torch.tensor(powers, dtype=D, device="cuda"))
    ws = (mant * power[:, None]).float()
    w, _ = R.weights(g, (nb * R.B, K))
    # at least a quarter of 2^-122: no gradient is subnormal
    dy = (0.25 + torch.rand((M, nb * R.B), generator=g, device="cuda", dtype=D)) * torch.where(
        torch.rand((M, nb * R.B), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    dy = (dy / _blocks_of(power)).to(BF)
    dense = R.dense_weight(w, ws)
    ref = dy.to(D) @ dense
    size = dy.to(D).abs() @ dense.abs()
    N = nb * R.B
    # products are exact; a sum of N in float32, two roundings a block for the ratio of two scales, the last scale
    tol = size * (N + 2 * nb + 16) * E + H * ref.abs()
    got = Q.linear_f8_backward(dy, Q.pack_f8(w, ws)).to(D)
    assert bool(torch.isfinite(got).all())
    off = (got - ref).abs() - tol
    assert float(off.max()) <= 0.0, (float(off.max()), float(size.max()))


@pytest.mark.parametrize("s", [1.0, -1.0])
def test_infinite_and_nan_scales(s):
    """A NaN or infinite scale leaves nothing finite in its columns, whatever scales follow it, and does not reach others."""
    Q, g = _Q(), _gen(5)
    nb, K, M = 6, 288, 40
    w, _ = R.weights(g, (nb * R.B, K), True)
    dy = torch.randint(1, 5, (M, nb * R.B), generator=g, device="cuda").to(BF)
    for bad in (float("nan"), float("inf") * s):
        for at in range(nb):
            for after in (0.0, 1.0, 1e-40, 1e38):
                ws = torch.ones((nb, 3), device="cuda")
                ws[at, 1] = bad
                ws[at + 1:, 1] = after
                got = Q.linear_f8_backward(dy, Q.pack_f8(w, ws))
                assert not bool(torch.isfinite(got[:, 128:256]).any()), (bad, at, after)
                assert bool(torch.isfinite(got[:, :128]).all()) and bool(torch.isfinite(got[:, 256:]).all())


def test_an_infinite_scale_next_to_zeros():
    """One block with an infinite scale, the others 0: the infinities of its own sums, not NaN."""
    Q, g = _Q(), _gen(6)
    nb, K, M = 5, 160, 20
    w, _ = R.weights(g, (nb * R.B, K), True)
    dy = torch.randint(1, 5, (M, nb * R.B), generator=g, device="cuda").to(BF)
    for at in range(nb):
        ws = torch.zeros((nb, 2), device="cuda")
        ws[at] = float("inf")
        part = dy[:, at * R.B:(at + 1) * R.B].to(D) @ w[at * R.B:(at + 1) * R.B].to(D)
        got = Q.linear_f8_backward(dy, Q.pack_f8(w, ws)).to(D)
        some = part != 0
        assert torch.equal(got[some], torch.sign(part[some]) * float("inf")) and bool(torch.isnan(got[~some]).all()), at
