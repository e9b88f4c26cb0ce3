"""Plain 64-bit implementations of the mixture-of-experts operators in 8-bit floating point, and their inputs."""
import torch

D = torch.float64
B = 128


def blocks(n):
    return -(-n // B)


def round_e4m3(v):
    """Float64 values to the nearest e4m3 value, ties to even, held to 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def quantize(x):
    """(code values, scales) in float64 of rows [R, K]: the scale is the float32 number nearest to max / 448."""
    R, K = x.shape
    full = torch.zeros((R, blocks(K) * B), dtype=D, device=x.device)
    full[:, :K] = x.to(D)
    full = full.reshape(R, -1, B)
    s = (full.abs().amax(2) / 448).float().to(D)
    v = torch.where(s[..., None] > 0, full / s[..., None], 0.0)
    return round_e4m3(v).reshape(R, -1)[:, :K], s


def spread_rows(s, K):
    """Scales [..., blocks] for each of K inputs."""
    return s.to(D).repeat_interleave(B, -1)[..., :K]


def spread_weight(s, N, K):
    return s.to(D).repeat_interleave(B, -1)[..., :K].repeat_interleave(B, -2)[..., :N, :]


def activations(g, M, K, exact=False):
    """e4m3 codes and scales of M rows.  exact: small whole numbers and powers of two, so that float32 sums are exact."""
    dev = g.device
    if exact:
        codes = torch.randint(-8, 9, (M, K), generator=g, device=dev).float()
        scales = torch.exp2(torch.randint(-2, 3, (M, blocks(K)), generator=g, device=dev).float())
    else:
        codes = (torch.randn((M, K), generator=g, device=dev) * 90).clamp(-448, 448)
        scales = torch.exp(torch.randn((M, blocks(K)), generator=g, device=dev)) * 0.01
    return codes.to(torch.float8_e4m3fn), scales


def weights(g, shape, exact=False):
    *lead, N, K = shape
    codes, scales = activations(g, int(torch.tensor(shape[:-1]).prod()), K, exact)
    dev = g.device
    s = torch.exp2(torch.randint(-2, 3, (*lead, blocks(N), blocks(K)), generator=g, device=dev).float()) if exact else \
        torch.exp(torch.randn((*lead, blocks(N), blocks(K)), generator=g, device=dev)) * 0.003
    return codes.reshape(*shape), s


def dense_weight(codes, s):
    return codes.to(D) * spread_weight(s, *codes.shape[-2:])


def order(ids, E):
    """(counts, rows, source) of ids [..., k] on the CPU."""
    flat = ids.reshape(-1).tolist()
    real = sorted((e, i) for i, e in enumerate(flat) if 0 <= e < E)
    rows, source = [-1] * len(flat), [-1] * len(flat)
    counts = [0] * E
    for place, (e, i) in enumerate(real):
        rows[i], source[place] = place, i
        counts[e] += 1
    t = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return t(counts), t(rows).reshape(ids.shape), t(source)
