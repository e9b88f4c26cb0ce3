"""The operators of a mixture-of-experts layer in 8-bit floating point as they are measured: cases, inputs, plain forms
and exact values.

quantize   rows to e4m3 codes with a float32 scale for each block of 128 inputs, s = max|x| / 448; or of
           up * silu(gate) formed from rows [up | gate]; its backward pass, with the quantisation passed straight through
dispatch   slots (token, choice) sorted by their expert, and the tokens' rows in that order, as they are or quantised;
           its backward pass adds up each token's rows
combine    each token's rows back from expert order, weighted and added; backward: gradients of the rows and weights
linear     y = sum over blocks of (x . w^T) xs[m, block] ws[n / 128, block], e4m3 codes with a scale for each 128 inputs
           of a token and each 128 x 128 block of the weight; its backward pass gives the gradient of the input
grouped    the same with one weight an expert, rows in expert order, counts on the device

Layer sizes are those of the benchmark's workloads: 4096 x 14336 and 28672 x 4096, eight experts; token counts run from
one decoded token to prefill and training batches.
"""
import math
import random

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_B = 128
_MOST_MNK = 8192 * 4096 * 14336          # the largest listed product
_MOST_ENK = 8 * 28672 * 4096             # the largest listed weights
_MOST_ROWS = 4096 * 14336                # elements of the largest listed quantisation
_MOST_SORTED = 4096 * 8 * 4096           # elements of the largest listed rows in expert order


def listed():
    return [
        # between a layer's two products for sixteen decoded tokens: SwiGLU and the second product's input
        {"name": "quantize 16x14336 swiglu", "op": "quantize", "R": 16, "K": 14336, "swiglu": True, "f32": False},
        # its gradient in a training batch
        {"name": "quantize back 4096x14336", "op": "quantize_back", "R": 4096, "K": 14336},
        # sixteen decoded tokens, two of eight experts each, as the first product's quantised input
        {"name": "dispatch 16x4096 e8 k2 f8", "op": "dispatch", "T": 16, "D": 4096, "E": 8, "k": 2, "f8": True, "f32": False},
        # a training batch, many experts, odd sizes
        {"name": "dispatch 4099x5000 e60 k6", "op": "dispatch", "T": 4099, "D": 5000, "E": 60, "k": 6, "f8": False, "f32": False},
        # the experts' outputs of a prefill batch back in token order, eight experts a token
        {"name": "combine 4096x4096 e64 k8", "op": "combine", "T": 4096, "D": 4096, "E": 64, "k": 8, "f32": False},
        # its gradient in a training batch, two experts a token
        {"name": "combine back 8192x4096 e8 k2", "op": "combine_back", "T": 8192, "D": 4096, "E": 8, "k": 2, "f32": False},
        # the second projection for one decoded token: the weight's bytes and the latency count
        {"name": "linear 1x4096x14336", "op": "linear", "M": 1, "N": 4096, "K": 14336, "bias": False, "f32": False},
        # a mixed batch of prompts and decoded tokens, sizes off every tile and block, float32 logits-like output
        {"name": "linear 333x5001x4128 f32", "op": "linear", "M": 333, "N": 5001, "K": 4128, "bias": True, "f32": True},
        # the second projection over a prefill batch
        {"name": "linear 2048x4096x14336", "op": "linear", "M": 2048, "N": 4096, "K": 14336, "bias": False, "f32": False},
        # up and gate projections of eight experts for sixteen decoded tokens, two experts each
        {"name": "grouped 32x28672x4096 e8", "op": "grouped", "T": 32, "E": 8, "N": 28672, "K": 4096, "bias": False, "f32": False},
        # the experts' second projection over a prefill batch, 4096 tokens with two experts each
        {"name": "grouped 8192x4096x14336 e8", "op": "grouped", "T": 8192, "E": 8, "N": 4096, "K": 14336, "bias": False, "f32": False},
        # the gradient of its input in training
        {"name": "grouped back 8192x4096x14336 e8", "op": "grouped_back", "T": 8192, "E": 8, "N": 4096, "K": 14336},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize_back", "dispatch", "dispatch", "dispatch_back", "combine", "combine_back",
                     "linear", "linear", "linear_back", "grouped", "grouped", "grouped_back"])
    if op.startswith("quantize"):
        while True:
            R, K = _log(rng, 1, 16384), 32 * _log(rng, 2, 448)
            if R * K <= _MOST_ROWS // 2:
                break
        case = {"op": op, "R": R, "K": K}
        return case | {"swiglu": rng.random() < 0.5, "f32": rng.random() < 0.3} if op == "quantize" else case
    if op.startswith(("dispatch", "combine")):
        while True:
            T, E, k, f8 = _log(rng, 1, 8192), _log(rng, 2, 256), rng.randint(1, 8), op == "dispatch" and rng.random() < 0.5
            D = _log(rng, 64, 8192)
            D = 32 * max(2, D // 32) if f8 or rng.random() < 0.7 else D
            if k <= E and T * k * D <= _MOST_SORTED // 2:
                break
        case = {"op": op, "T": T, "D": D, "E": E, "k": k, "f32": rng.random() < 0.3}
        return case | {"f8": f8} if op == "dispatch" else case
    if op.startswith("linear"):
        while True:
            M, N, K = _log(rng, 1, 4096), _log(rng, 128, 28672), 32 * _log(rng, 4, 448)
            if M * N * K <= _MOST_MNK // 4:
                break
        case = {"op": op, "M": M, "N": N, "K": K}
        return case | {"bias": rng.random() < 0.5, "f32": rng.random() < 0.25} if op == "linear" else case
    while True:
        T, E, N, K = _log(rng, 1, 8192), _log(rng, 2, 64), _log(rng, 128, 28672), 32 * _log(rng, 4, 448)
        if T * N * K <= _MOST_MNK // 4 and E * N * K <= _MOST_ENK // 2:
            break
    case = {"op": op, "T": T, "E": E, "N": N, "K": K}
    return case | {"bias": rng.random() < 0.5, "f32": rng.random() < 0.25} if op == "grouped" else case


def _blocks(n):
    return -(-n // _B)


def work(case):
    op = case["op"]
    e = 4 if case.get("f32") else 2
    if op == "quantize":
        n, wide = case["R"] * case["K"], 2 if case["swiglu"] else 1
        return {"bytes": n * (wide * e + 1 + 2) + 4 * case["R"] * _blocks(case["K"]), "flops": n * (12 if case["swiglu"] else 3)}
    if op == "quantize_back":
        n = case["R"] * case["K"]
        return {"bytes": n * (2 + 4 + 4), "flops": 14 * n}
    if op.startswith(("dispatch", "combine")):
        T, D, k = case["T"], case["D"], case["k"]
        few, many, slots = T * D, T * k * D, T * k
        if op == "dispatch":
            out = many * (1 + 2) + 4 * slots * _blocks(D) if case["f8"] else many * e
            return {"bytes": few * e + out + slots * (8 + 4 + 4) + 4 * case["E"], "flops": few * (3 if case["f8"] else 1)}
        if op == "combine_back":
            return {"bytes": (few + 2 * many) * e + slots * (4 + 4 + 4), "flops": 3 * many}
        return {"bytes": (few + many) * e + slots * (8 if op == "combine" else 4), "flops": 2 * many}
    E, M, N, K = case.get("E", 1), case.get("M", case.get("T")), case["N"], case["K"]
    used = min(E, M)
    weights = used * (N * K + 4 * _blocks(N) * _blocks(K))
    counts = 4 * E if op.startswith("grouped") else 0
    if op.endswith("back"):
        return {"bytes": 2 * M * N + weights + 2 * M * K + counts, "flops": 2 * M * N * K}
    return {"bytes": M * K + 4 * M * _blocks(K) + weights + (2 * used * N if case["bias"] else 0) + e * M * N + counts,
            "flops": 2 * M * N * K}


def _normal(g, shape, typical, dtype):
    return (torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32) * typical).to(dtype)


def _activations(g, rows, cols):
    """e4m3 codes [rows, cols] of normal values and scales [rows, blocks] that give values of about one."""
    nb = _blocks(cols)
    v = torch.randn((rows, nb, _B), generator=g, device=_DEV)
    v = v * torch.exp(0.3 * torch.randn((rows, nb, 1), generator=g, device=_DEV))
    s = v.abs().amax(2, keepdim=True) / 448.0
    codes = (v / s).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).reshape(rows, nb * _B)[:, :cols]
    return codes.contiguous(), s[..., 0].contiguous()


def _weights(g, E, N, K, typical):
    """e4m3 codes [E, N, K] and scales [E, N / 128, K / 128] that give values of about `typical`."""
    codes = torch.empty((E, N, K), dtype=torch.float8_e4m3fn, device=_DEV)
    scales = torch.exp(0.3 * torch.randn((E, _blocks(N), _blocks(K)), generator=g, device=_DEV)) * (typical * 4.5 / 448.0)
    for e in range(E):
        v = torch.randn((N, K), generator=g, device=_DEV, dtype=torch.bfloat16) * (448.0 / 4.5)
        codes[e] = v.clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
    return codes, scales


def _routing(g, T, E, k):
    """k different experts for each token, some experts chosen far more often, and softmaxed weights."""
    logits = torch.randn((T, E), generator=g, device=_DEV) + 0.7 * torch.randn((E,), generator=g, device=_DEV)
    top, ids = torch.topk(logits, k, dim=1)
    return ids, torch.softmax(top, 1)


def _counts(seed, T, E):
    """Rows of each expert: a skewed routing of T rows, some experts without any."""
    rng = random.Random(seed)
    share = [math.exp(rng.gauss(0.0, 0.5)) * (rng.random() < 0.9) for _ in range(E)]
    share[rng.randrange(E)] += 1.0
    total, left, counts = sum(share), T, []
    for i, w in enumerate(share):
        counts.append(min(left, int(T * w / total)))
        left -= counts[-1]
    for i in range(left):
        counts[rng.choices(range(E), share)[0]] += 1
    return counts


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    s = dict(case)
    op, bf = case["op"], torch.bfloat16
    float_ = torch.float32 if case.get("f32") else bf
    if op == "quantize":
        R, K = case["R"], case["K"]
        s["x"] = _normal(g, (R, 2 * K if case["swiglu"] else K), 1.5, float_)
        return s
    if op == "quantize_back":
        R, K = case["R"], case["K"]
        s["raw"] = _normal(g, (R, 2 * K), 1.5, bf)
        s["dh"] = _normal(g, (R, K), 1e-2, bf)
        return s
    if op.startswith(("dispatch", "combine")):
        T, D, E, k = case["T"], case["D"], case["E"], case["k"]
        s["ids"], s["w"] = _routing(g, T, E, k)
        if op == "dispatch":
            s["x"] = _normal(g, (T, D), 1.0, float_)
            return s
        source = torch.argsort(s["ids"].reshape(-1), stable=True)
        s["rows"] = torch.empty_like(source)
        s["rows"][source] = torch.arange(T * k, device=_DEV)
        s["source"] = source
        s["y"] = _normal(g, (T * k, D), 1.0, float_)
        if op == "combine_back":
            s["dout"] = _normal(g, (T, D), 1e-2, float_)
        if own:
            import bit_weight_only_offline_amd as Q
            s["order"] = Q.expert_order(s["ids"], E)
        return s
    E, N, K = case.get("E", 1), case["N"], case["K"]
    M = case.get("M", case.get("T"))
    s["codes"], s["scales"] = _weights(g, E, N, K, 1.0 / math.sqrt(K))
    if op.startswith("grouped"):
        counts = _counts(seed, M, E)
        s["counts"] = torch.tensor(counts, dtype=torch.int32, device=_DEV)
        s["most"] = max(counts)
    if op.endswith("back"):
        s["dy"] = _normal(g, (M, N), 1e-2, bf)
    else:
        s["x"], s["xs"] = _activations(g, M, K)
        s["b"] = _normal(g, (E, N) if op == "grouped" else (N,), 0.1, bf) if case["bias"] else None
    if own:
        import bit_weight_only_offline_amd as Q
        s["packed"] = Q.pack_f8(s["codes"], s["scales"]) if op.startswith("grouped") else Q.pack_f8(s["codes"][0], s["scales"][0])
    return s


def _silu(g):
    """silu(g) and its derivative."""
    p = 1.0 / (1.0 + torch.exp(-g))
    return g * p, p * (1.0 + g * (1.0 - p))


def _rounded(x):
    """The values that e4m3 codes and float32 block scales of float32 rows stand for."""
    R, K = x.shape
    full = torch.zeros((R, _blocks(K) * _B), dtype=torch.float32, device=x.device)
    full[:, :K] = x
    full = full.reshape(R, -1, _B)
    s = full.abs().amax(2, keepdim=True) / 448.0
    # the quotient in 64 bits: rounded to 32 first, those next to a border between two codes would go to either
    v = torch.where(s > 0, full.double() / s, 0.0)
    steps = torch.frexp(v).exponent.clamp_min(-5) - 4            # 2^steps: what codes near v are apart
    q = torch.ldexp(torch.round(torch.ldexp(v, -steps)), steps).clamp(-448.0, 448.0).float()
    return (q * s).reshape(R, -1)[:, :K]


def _weight(s):
    """The experts' float32 weights [E, N, K]."""
    N, K = s["N"], s["K"]
    wide = s["scales"].repeat_interleave(_B, 1)[:, :N].repeat_interleave(_B, 2)[:, :, :K]
    return s["codes"].float() * wide


def _padded(s, x):
    """Rows in expert order as [E, most, ..], and the index that gives them back."""
    E, counts = s["E"], s["counts"].long()
    first = torch.cumsum(counts, 0) - counts
    expert = torch.repeat_interleave(torch.arange(E, device=x.device), counts, output_size=x.shape[0])
    place = torch.arange(x.shape[0], device=x.device) - first[expert]
    full = torch.zeros((E, s["most"], x.shape[1]), dtype=x.dtype, device=x.device)
    full[expert, place] = x
    return full, expert, place


def _plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "quantize":
        x = s["x"].float()
        if s["swiglu"]:
            x = x[:, :s["K"]] * _silu(x[:, s["K"]:])[0]
        return _rounded(x).to(bf)
    if op == "quantize_back":
        dh, up, gate = s["dh"].float(), s["raw"][:, :s["K"]].float(), s["raw"][:, s["K"]:].float()
        a, da = _silu(gate)
        return torch.cat([dh * a, dh * up * da], 1).to(bf)
    if op == "dispatch":
        flat = s["ids"].reshape(-1)
        source = torch.argsort(flat, stable=True)
        rows = torch.empty_like(source)
        rows[source] = torch.arange(flat.numel(), device=flat.device)
        counts = (flat[:, None] == torch.arange(s["E"], device=flat.device)).sum(0)
        x = s["x"][source // s["k"]]
        x = _rounded(x.float()).to(bf) if s["f8"] else x
        return counts.int(), rows.reshape(s["ids"].shape).int(), source.int(), x
    if op in ("dispatch_back", "combine", "combine_back"):
        T, k, dtype = s["T"], s["k"], s["y"].dtype
        y = s["y"].float()[s["rows"]].reshape(T, k, -1)
        if op == "dispatch_back":
            return y.sum(1).to(dtype)
        if op == "combine":
            return (y * s["w"][:, :, None]).sum(1).to(dtype)
        dout = s["dout"].float()
        dy = (s["w"][:, :, None] * dout[:, None]).reshape(T * k, -1)[s["source"]]
        return dy.to(dtype), (y * dout[:, None]).sum(2)
    if op.endswith("back"):
        dy, w = s["dy"].float(), _weight(s)
        if op == "linear_back":
            return (dy @ w[0]).to(bf)
        full, expert, place = _padded(s, dy)
        return torch.bmm(full, w)[expert, place].to(bf)
    x = s["x"].float() * s["xs"].repeat_interleave(_B, 1)[:, :s["K"]]
    w = _weight(s)
    if op == "linear":
        y = x @ w[0].t()
        y = y if s["b"] is None else y + s["b"].float()
    else:
        full, expert, place = _padded(s, x)
        y = torch.bmm(full, w.transpose(1, 2))[expert, place]
        y = y if s["b"] is None else y + s["b"].float()[expert]
    return y if s["f32"] else y.to(bf)


def run(s):
    if not own:
        return _plain(s)
    import bit_weight_only_offline_amd as Q
    op = s["op"]
    if op == "quantize":
        return Q.dequantize_f8(*Q.quantize_f8(s["x"], act="swiglu" if s["swiglu"] else None))
    if op == "quantize_back":
        return Q.quantize_f8_backward(s["dh"], s["raw"], act="swiglu")
    if op == "dispatch":
        order = Q.expert_order(s["ids"], s["E"])
        x = Q.dequantize_f8(*Q.dispatch_tokens(s["x"], order, f8=True)) if s["f8"] else Q.dispatch_tokens(s["x"], order)
        return order.counts, order.rows, order.source, x
    if op == "dispatch_back":
        return Q.dispatch_tokens_backward(s["y"], s["order"])
    if op == "combine":
        return Q.combine_tokens(s["y"], s["order"], s["w"])
    if op == "combine_back":
        return Q.combine_tokens_backward(s["dout"], s["y"], s["order"], s["w"])
    if op == "linear_back":
        return Q.linear_f8_backward(s["dy"], s["packed"])
    if op == "grouped_back":
        return Q.grouped_linear_f8_backward(s["dy"], s["packed"], s["counts"])
    out_dtype = torch.float32 if s["f32"] else torch.bfloat16
    if op == "linear":
        return Q.linear_f8(s["x"], s["xs"], s["packed"], bias=s["b"], out_dtype=out_dtype)
    return Q.grouped_linear_f8(s["x"], s["xs"], s["packed"], s["counts"], bias=s["b"], out_dtype=out_dtype)


def _exact_codes(x):
    """Block by block: the scale as the float32 number that it is, each value to the nearest e4m3 value."""
    R, K = x.shape
    out = torch.empty_like(x)
    for k in range(0, K, _B):
        part = x[:, k:k + _B]
        s = (part.abs().amax(1, keepdim=True) / 448).float().double()
        v = torch.where(s > 0, part / s, 0.0)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        out[:, k:k + _B] = (torch.round(v / step) * step).clamp(-448, 448) * s
    return out


def exact(case, seed):
    s, d = prepare(case, seed), torch.float64
    op = case["op"]
    if op == "quantize":
        x = s["x"].to(d)
        if case["swiglu"]:
            up, gate = x.chunk(2, 1)
            x = up * gate * torch.special.expit(gate)
        return _exact_codes(x)
    if op == "quantize_back":
        up, gate = s["raw"].to(d).chunk(2, 1)
        dh, p = s["dh"].to(d), torch.special.expit(gate)
        return torch.cat([dh * gate * p, dh * up * p * (1 + gate * torch.special.expit(-gate))], 1)
    if op.startswith(("dispatch", "combine")):
        k = case["k"]
        key = s["ids"].reshape(-1) * s["ids"].numel() + torch.arange(s["ids"].numel(), device=_DEV)
        source = torch.sort(key).values % s["ids"].numel()
        if op == "dispatch":
            x = s["x"].to(d)
            return None, None, None, (_exact_codes(x) if case["f8"] else x)[source // k]
        y = torch.zeros_like(s["y"], dtype=d)
        y[source] = s["y"].to(d)                             # in the order of the slots
        y = y.reshape(case["T"], k, -1)
        if op == "dispatch_back":
            return torch.einsum("tkd->td", y)
        w = s["w"].to(d)
        if op == "combine":
            return torch.einsum("tk,tkd->td", w, y)
        dout = s["dout"].to(d)
        dy = dout[source // k] * w.reshape(-1)[source][:, None]
        return dy, torch.einsum("td,tkd->tk", dout, y)
    E, N, K = case.get("E", 1), case["N"], case["K"]
    ends = s["counts"].tolist() if op.startswith("grouped") else [case["M"]]
    back = op.endswith("back")
    out = torch.empty((sum(ends), K if back else N), dtype=d, device=_DEV)
    n_of, k_of = torch.arange(N, device=_DEV) // _B, torch.arange(K, device=_DEV) // _B
    at = 0
    for e, count in enumerate(ends):
        w = s["codes"][e].to(d) * s["scales"][e].to(d)[n_of][:, k_of]
        if back:
            out[at:at + count] = s["dy"][at:at + count].to(d) @ w
        else:
            out[at:at + count] = (s["x"][at:at + count].to(d) * s["xs"][at:at + count].to(d)[:, k_of]) @ w.t().contiguous()
            if s["b"] is not None:
                out[at:at + count] += s["b"].reshape(E, N)[e].to(d)
        at += count
    return out
