"""Grouped products on every tile, exactly, and NaN through every tile of the 8-bit and of the bf16 matrix cores.

Whole numbers and scales that are powers of two make every sum exact, in any order.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import moe8_reference as R  # noqa: E402
from test_gpu_moe8 import SCHEDULED  # noqa: E402

D = torch.float64
BF, F32 = torch.bfloat16, torch.float32


def _Q():
    import bit_weight_only_offline_amd as Q
    return Q


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# Counts around a tile's rows: none, one, one less and one more, and what is left; `behind` rows belong to no expert.
def _ragged(block, T, behind):
    counts = [0, 1, block - 1, 0, block + 1, block]
    return counts + [T - behind - sum(counts)]


# Rows of each tile: forward, backward.  The schedule that a size takes is looked up, so that every tile is reached.
ROWS = {False: [16, 16, 128, 64, 64, 64, 32, 32, 256], True: [256, 64, 32, 16]}
EXPERTS, BEHIND = 7, 3


def _size(back, dtype, tile, long):
    """The least product over seven experts that takes this tile: rows for the counts above, inputs (channels, backward)
    that end inside a block; long: a sum of more than 32 blocks."""
    Q, block = _Q(), ROWS[back][tile]
    sums = (4128, 4192, 5216) if long else (160, 320, 416, 544, 736, 1184)
    outs = (67, 131, 300, 516, 1031, 1179, 2049, 2301, 3000, 4100) if not back else (64, 160, 288, 544, 1088, 2080, 2976, 4128)
    if back:
        sums = [s + 5 for s in sums]
    sizes = sorted(((T, o, s) for T in [*range(70, 400, 12), *range(400, 1200, 36), *range(1200, 4000, 96)]
                    for o in outs for s in sums if T >= 3 * block + 1 + BEHIND), key=lambda c: c[1] * c[2] * (c[0] + 350))
    for T, o, s in sizes:
        N, K = (s, o) if back else (o, s)
        if Q.f8_default_schedule(T, N, K, EXPERTS, backward=back, out_dtype=dtype).tile == tile:
            return block, T, N, K
    raise AssertionError(f"no size takes tile {tile}")


def _case(block, T, N, K, seed):
    g = _gen(seed)
    counts = _ragged(block, T, BEHIND)
    assert len(counts) == EXPERTS and min(counts) >= 0 and sum(counts) == T - BEHIND
    w, ws = R.weights(g, (EXPERTS, N, K), True)
    return g, counts, w, ws


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("dtype,tile", [(BF, t) for t in range(9)] + [(F32, t) for t in range(8)])
def test_grouped_tiles_exact(dtype, tile, long):
    """Each row by its own expert's weight and bias, bit for bit; NaN in one row and in the rows behind the last."""
    Q = _Q()
    block, T, N, K = _size(False, dtype, tile, long)
    g, counts, w, ws = _case(block, T, N, K, T + N)
    x, xs = R.activations(g, T, K, True)
    b = torch.randint(-4, 5, (len(counts), N), generator=g, device="cuda").to(BF)
    last = sum(counts)
    x.view(torch.uint8)[last:] = 0x7F
    xs[last:] = float("nan")
    lost = counts[1] + counts[2] - 1                          # the last row of an expert
    x.view(torch.uint8)[lost, K - 7] = 0xFF
    pw, cnt = Q.pack_f8(w, ws), torch.tensor(counts, dtype=torch.int32, device="cuda")
    out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")
    Q.grouped_linear_f8(x, xs, pw, cnt, bias=b, out_dtype=dtype, out=out)
    assert bool(torch.isnan(out[lost]).all()) and int(torch.isnan(out).sum()) == N
    at = 0
    for e, c in enumerate(counts):
        ref = (x[at:at + c].to(D) * R.spread_rows(xs[at:at + c], K)) @ R.dense_weight(w[e], ws[e]).t() + b[e].to(D)
        keep = torch.arange(at, at + c, device="cuda") != lost
        assert torch.equal(out[at:at + c][keep], ref.float().to(dtype)[keep]), (e, c)
        at += c
    assert bool((out[last:] == 7.0).all())


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("tile", range(4))
def test_grouped_backward_tiles_exact(tile, long):
    Q = _Q()
    block, T, N, K = _size(True, BF, tile, long)
    g, counts, w, ws = _case(block, T, N, K, T + N + 1)
    dy = torch.randint(-4, 5, (T, N), generator=g, device="cuda").to(BF)
    last = sum(counts)
    dy[last:] = float("nan")
    lost = counts[1] + counts[2] - 1
    dy[lost, N - 1] = float("nan")
    out = torch.full((T, K), 7.0, dtype=BF, device="cuda")
    Q.grouped_linear_f8_backward(dy, Q.pack_f8(w, ws), torch.tensor(counts, dtype=torch.int32, device="cuda"), out=out)
    assert bool(torch.isnan(out[lost]).all()) and int(torch.isnan(out).sum()) == K
    at = 0
    for e, c in enumerate(counts):
        ref = dy[at:at + c].to(D) @ R.dense_weight(w[e], ws[e])
        keep = torch.arange(at, at + c, device="cuda") != lost
        assert torch.equal(out[at:at + c][keep], ref.float().to(BF)[keep]), (e, c)
        at += c
    assert bool((out[last:] == 7.0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,K", SCHEDULED + [(4500, 4100, 800)])
def test_nan_stays_in_its_row_and_channel(M, N, K, dtype):
    """In codes and scales of a row, and in a weight: also in the last inputs of a row, behind which the next begins."""
    Q, g = _Q(), _gen(M + K)
    x, xs = R.activations(g, M, K, True)
    w, ws = R.weights(g, (N, K), True)
    pw = Q.pack_f8(w, ws)
    clean = Q.linear_f8(x, xs, pw, out_dtype=dtype)
    assert bool(torch.isfinite(clean).all())
    bad, s2 = x.clone(), xs.clone()
    bad.view(torch.uint8)[1, :40] = 0x7F
    bad.view(torch.uint8)[M - 2, K - 1] = 0xFF
    s2[2, R.blocks(K) - 1] = float("nan")
    rows = torch.zeros(M, dtype=torch.bool, device="cuda")
    rows[[1, 2, M - 2]] = True
    y = Q.linear_f8(bad, s2, pw, out_dtype=dtype)
    assert bool(torch.isnan(y[rows]).all()) and torch.equal(y[~rows], clean[~rows])
    w2, channels = w.clone(), torch.zeros(N, dtype=torch.bool, device="cuda")
    w2.view(torch.uint8)[7, K - 1] = 0xFF
    w2.view(torch.uint8)[N - 1, 0] = 0x7F
    channels[[7, N - 1]] = True
    y = Q.linear_f8(x, xs, Q.pack_f8(w2, ws), out_dtype=dtype)
    assert bool(torch.isnan(y[:, channels]).all()) and torch.equal(y[:, ~channels], clean[:, ~channels])


def test_nan_cases_take_every_tile():
    Q = _Q()
    for dtype, tiles in ((BF, range(9)), (F32, range(8))):
        seen = {(s.tile, s.splits > 1) for s in (Q.f8_default_schedule(*c, out_dtype=dtype) for c in SCHEDULED + [(4500, 4100, 800)])}
        assert seen == {(t, False) for t in tiles} | {(t, True) for t in range(3, 8)}, sorted(seen)
