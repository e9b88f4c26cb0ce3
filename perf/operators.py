"""The 8-bit feed-forward operators as they are measured: cases, inputs, plain forms and exact values.

linear_i8    y = (xq . wq^T) * xs[m] * ws[n] + b, int8 codes with a scale for each token and channel; its backward
             pass gives the gradient of the activations for frozen weights
gated_i8     h = act(gate) * up, both int8 projections of one input; backward: gradients of the input and of [up|gate]
block_norm   r' = a r + gate * norm(y) w_post, x = norm(r') w_pre, as bf16 or as int8 codes and token scales; backward:
             gradients of r, y, both norm weights and the gate

Layer sizes are those of the benchmark's workloads: 4096 x 4096, 28672 x 4096 (14336 gate and 14336 up channels) and
4096 x 14336; token counts run from one decoded token to prefill and training batches.
"""
import math

import torch

own = False

_DEV = "cuda" if torch.cuda.is_available() else "cpu"
_MOST_MNK = 4096 * 28672 * 4096          # the largest listed product
_MOST_RC = 8192 * 4096                   # the largest listed norm
_C1 = math.sqrt(2.0 / math.pi)
_C2 = 0.044715


def listed():
    return [
        # the second projection of a feed-forward layer for one decoded token: the weight's bytes and the latency count
        {"name": "linear 1x4096x14336", "op": "linear", "M": 1, "N": 4096, "K": 14336, "bias": False, "f32": False},
        # a square projection for a batch of sixteen decoded tokens
        {"name": "linear 16x4096x4096", "op": "linear", "M": 16, "N": 4096, "K": 4096, "bias": True, "f32": False},
        # the second projection over a prefill batch
        {"name": "linear 2048x4096x14336", "op": "linear", "M": 2048, "N": 4096, "K": 14336, "bias": False, "f32": False},
        # a mixed batch of prompts and decoded tokens, sizes off every tile, float32 logits-like output
        {"name": "linear 333x5001x4128 f32", "op": "linear", "M": 333, "N": 5001, "K": 4128, "bias": True, "f32": True},
        # gradient of the activations through the frozen second projection, a training batch
        {"name": "linear back 2048x4096x14336", "op": "linear_back", "M": 2048, "N": 4096, "K": 14336},
        # gate and up projections for four decoded tokens
        {"name": "gated 4x14336x4096", "op": "gated", "M": 4, "N": 14336, "K": 4096, "bias": False, "act": "silu", "keep": False},
        # a small mixed batch, odd sizes, the other activation, with biases
        {"name": "gated 77x5003x2080 gelu", "op": "gated", "M": 77, "N": 5003, "K": 2080, "bias": True, "act": "gelu", "keep": False},
        # gate and up projections of a training batch, which keeps [up|gate] for the backward pass
        {"name": "gated 4096x14336x4096", "op": "gated", "M": 4096, "N": 14336, "K": 4096, "bias": False, "act": "silu", "keep": True},
        # backward through activation, product and both frozen projections
        {"name": "gated back 2048x14336x4096", "op": "gated_back", "M": 2048, "N": 14336, "K": 4096, "act": "silu"},
        # between two blocks, eight decoded tokens, the next block's int8 input
        {"name": "norm 8x4096 int8", "op": "norm", "R": 8, "C": 4096, "B": 0, "f32": False, "int8": True},
        # the same over a prefill batch of two sequences with a gate each, float32 residual stream, bf16 output
        {"name": "norm 8192x4096", "op": "norm", "R": 8192, "C": 4096, "B": 2, "f32": True, "int8": False},
        # its backward pass in training: a learned gate for each channel, bf16 residual stream
        {"name": "norm back 8192x4096", "op": "norm_back", "R": 8192, "C": 4096, "B": 1, "f32": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_back", "gated", "gated", "gated_back", "norm", "norm_back"])
    if op.startswith("norm"):
        while True:
            C = _log(rng, 256, 14336)
            C = C if rng.random() < 0.25 else 32 * max(8, C // 32)
            B = rng.choice([0, 1, 1, 2, 4])
            R = max(1, B) * _log(rng, 1, 4096)
            if R * C <= _MOST_RC:
                break
        case = {"op": op, "R": R, "C": C, "B": B, "f32": rng.random() < 0.4}
        if op == "norm":
            case["int8"] = rng.random() < 0.5 and C % 32 == 0
        return case
    while True:
        M, N, K = _log(rng, 1, 4096), _log(rng, 128, 28672), 32 * _log(rng, 4, 448)
        if op.startswith("gated"):
            N = max(64, N // 2)
        if M * N * K * (2 if op.startswith("gated") else 1) <= _MOST_MNK // (2 if op.endswith("back") else 1):
            break
    case = {"op": op, "M": M, "N": N, "K": K}
    if op == "linear":
        case |= {"bias": rng.random() < 0.5, "f32": rng.random() < 0.25}
    elif op == "gated":
        case |= {"bias": rng.random() < 0.5, "act": rng.choice(["silu", "gelu"]), "keep": rng.random() < 0.5}
    elif op == "gated_back":
        case |= {"act": rng.choice(["silu", "gelu"])}
    return case


def work(case):
    if case["op"].startswith("norm"):
        R, C = case["R"], case["C"]
        e = 4 if case["f32"] else 2
        vectors = 2 * 4 * C + 4 * C * case["B"]
        if case["op"] == "norm":
            return {"bytes": R * C * (2 + 2 * e + (1 if case["int8"] else 2)) + vectors + (4 * R if case["int8"] else 0),
                    "flops": 12 * R * C}
        return {"bytes": R * C * (2 + e + 2 + e + e + 2) + 2 * vectors, "flops": 24 * R * C}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "linear":
        return {"bytes": M * K + 4 * M + N * K + 4 * N + (2 * N if case["bias"] else 0) + M * N * (4 if case["f32"] else 2),
                "flops": 2 * M * N * K}
    if case["op"] == "linear_back":
        return {"bytes": 2 * M * N + N * K + 4 * N + 2 * M * K, "flops": 2 * M * N * K}
    if case["op"] == "gated":
        return {"bytes": M * K + 4 * M + 2 * N * K + 8 * N + (4 * N if case["bias"] else 0) + 2 * M * N + (4 * M * N if case["keep"] else 0),
                "flops": 4 * M * N * K}
    return {"bytes": 2 * M * N + 4 * M * N + 2 * N * K + 8 * N + 4 * M * N + 2 * M * K, "flops": 4 * M * N * K}


def _codes(g, rows, cols, typical):
    """Rows of a normal distribution as symmetric int8 codes, and scales that give values of about `typical`."""
    v = torch.randn((rows, cols), generator=g, device=_DEV, dtype=torch.bfloat16)
    s = v.abs().amax(1, keepdim=True).float() / 127.0
    codes = torch.round(v.float() / s).to(torch.int8)
    spread = torch.exp(0.5 * torch.randn((rows,), generator=g, device=_DEV))
    return codes, s[:, 0] * spread * typical


def _normal(g, shape, typical, dtype):
    return (torch.randn(shape, generator=g, device=_DEV, dtype=torch.float32) * typical).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device=_DEV)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"].startswith("norm"):
        R, C, B = case["R"], case["C"], case["B"]
        stream = torch.float32 if case["f32"] else torch.bfloat16
        s["y"] = _normal(g, (R, C), 0.7, torch.bfloat16)
        s["r"] = _normal(g, (R, C), 2.0, stream)
        s["post"] = 1.0 + _normal(g, (C,), 0.2, torch.float32)
        s["pre"] = 1.0 + _normal(g, (C,), 0.2, torch.float32)
        s["gate"] = None if B == 0 else _normal(g, (C,) if B == 1 else (B, C), 0.5, torch.float32)
        s["scale"], s["eps"] = 0.9, 1e-6
        if case["op"] == "norm_back":
            s["dx"] = _normal(g, (R, C), 1e-2, torch.bfloat16)
            s["dr"] = _normal(g, (R, C), 1e-2, stream)
        return s
    M, N, K = case["M"], case["N"], case["K"]
    typical = 1.0 / math.sqrt(K)
    if case["op"].startswith("gated"):
        s["up"], s["us"] = _codes(g, N, K, typical)
        s["gate"], s["gs"] = _codes(g, N, K, typical)
        width = 2 * N
    else:
        s["w"], s["ws"] = _codes(g, N, K, typical)
        width = N
    if case["op"].endswith("back"):
        s["dy"] = _normal(g, (M, N), 1e-2, torch.bfloat16)
        if case["op"] == "gated_back":
            s["raw"] = _normal(g, (M, 2 * N), 1.0, torch.bfloat16)
    else:
        s["x"], s["xs"] = _codes(g, M, K, 1.0)
        s["b"] = _normal(g, (width,), 0.1, torch.bfloat16) if case["bias"] else None
    if own:
        import bit_weight_only_offline_amd as Q
        if case["op"].startswith("gated"):
            s["packed"] = Q.pack_gated(s["up"], s["us"], s["gate"], s["gs"])
        else:
            s["packed"] = Q.pack_channel(s["w"], s["ws"])
    return s


def _act(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    t = torch.tanh(_C1 * (g + _C2 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * (_C1 * (1.0 + 3.0 * _C2 * g * g))


def _rows(t, R):
    """A gate [C] or [B, C] for each of R rows."""
    return t if t.dim() == 1 else t.repeat_interleave(R // t.shape[0], 0)


def _plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "linear":
        y = (s["x"].float() @ s["w"].float().t()) * s["xs"][:, None] * s["ws"]
        y = y if s["b"] is None else y + s["b"].float()
        return y if s["f32"] else y.to(bf)
    if op == "linear_back":
        return ((s["dy"].float() * s["ws"]) @ s["w"].float()).to(bf)
    if op == "gated":
        x, N = s["x"].float(), s["N"]
        up = (x @ s["up"].float().t()) * s["xs"][:, None] * s["us"]
        gate = (x @ s["gate"].float().t()) * s["xs"][:, None] * s["gs"]
        if s["b"] is not None:
            up, gate = up + s["b"][:N].float(), gate + s["b"][N:].float()
        h = (_act(gate, s["act"])[0] * up).to(bf)
        return (h, torch.cat([up, gate], 1).to(bf)) if s["keep"] else h
    if op == "gated_back":
        dh, N = s["dy"].float(), s["N"]
        up, gate = s["raw"][:, :N].float(), s["raw"][:, N:].float()
        a, da = _act(gate, s["act"])
        du, dg = dh * a, dh * up * da
        dx = (du * s["us"]) @ s["up"].float() + (dg * s["gs"]) @ s["gate"].float()
        return dx.to(bf), torch.cat([du, dg], 1).to(bf)
    y, r, eps = s["y"].float(), s["r"].float(), s["eps"]
    if op == "norm":
        t = y * torch.rsqrt((y * y).mean(1, keepdim=True) + eps) * s["post"]
        t = t if s["gate"] is None else t * _rows(s["gate"], s["R"])
        r = s["scale"] * r + t
        x = r * torch.rsqrt((r * r).mean(1, keepdim=True) + eps) * s["pre"]
        if s["int8"]:
            step = x.abs().amax(1, keepdim=True) / 127.0
            x = torch.round(x / step).clamp(-127, 127).to(torch.int8).float() * step
        return r.to(s["r"].dtype), x.to(bf)
    u = r * (iq := torch.rsqrt((r * r).mean(1, keepdim=True) + eps))
    v = y * (ip := torch.rsqrt((y * y).mean(1, keepdim=True) + eps))
    dx, n = s["dx"].float(), s["dx"].float() * s["pre"]
    dr = s["dr"].float() + iq * (n - u * (n * u).mean(1, keepdim=True))
    dt = dr if s["gate"] is None else dr * _rows(s["gate"], s["R"])
    dv = dt * s["post"]
    dy = ip * (dv - v * (dv * v).mean(1, keepdim=True))
    dgate = None
    if s["gate"] is not None:
        dgate = (dr * v * s["post"]).reshape(s["B"], -1, s["C"]).sum(1).reshape(s["gate"].shape)
    return (s["scale"] * dr).to(s["r"].dtype), dy.to(bf), (dt * v).sum(0), (dx * u).sum(0), dgate


def run(s):
    if not own:
        return _plain(s)
    import bit_weight_only_offline_amd as Q
    op = s["op"]
    if op == "linear":
        return Q.linear_i8(s["x"], s["xs"], s["packed"], bias=s["b"], out_dtype=torch.float32 if s["f32"] else torch.bfloat16)
    if op == "linear_back":
        return Q.linear_i8_backward(s["dy"], s["packed"])
    if op == "gated":
        return Q.gated_i8(s["x"], s["xs"], s["packed"], bias=s["b"], act=s["act"], keep_raw=s["keep"])
    if op == "gated_back":
        return Q.gated_i8_backward(s["dy"], s["raw"], s["packed"], act=s["act"])
    if op == "norm":
        r, x = Q.block_norm(s["r"], s["y"], post_weight=s["post"], pre_weight=s["pre"], gate=s["gate"],
                            residual_scale=s["scale"], eps=s["eps"], int8=s["int8"])
        if s["int8"]:
            x = torch.mul(x[0], x[1][:, None], out=torch.empty_like(s["y"]))
        return r, x
    return Q.block_norm_backward(s["dx"], s["dr"], s["r"], s["y"], post_weight=s["post"], pre_weight=s["pre"],
                                 gate=s["gate"], residual_scale=s["scale"], eps=s["eps"])


def _sigma(g):
    return torch.special.expit(g)


def exact(case, seed):
    s, d = prepare(case, seed), torch.float64
    op = case["op"]
    if op in ("linear", "linear_back"):
        w = s["w"].to(d) * s["ws"].to(d).reshape(-1, 1)
        if op == "linear_back":
            return torch.mm(s["dy"].to(d), w)
        y = torch.mm(s["x"].to(d) * s["xs"].to(d).reshape(-1, 1), w.t().contiguous())
        return y if s["b"] is None else y.add_(s["b"].to(d))
    if op in ("gated", "gated_back"):
        both = torch.cat([s["up"].to(d) * s["us"].to(d).reshape(-1, 1), s["gate"].to(d) * s["gs"].to(d).reshape(-1, 1)])
        if op == "gated":
            raw = torch.mm(s["x"].to(d) * s["xs"].to(d).reshape(-1, 1), both.t().contiguous())
            raw = raw if s["b"] is None else raw.add_(s["b"].to(d))
        else:
            raw = s["raw"].to(d)
        u, g = raw.chunk(2, 1)
        if case["act"] == "silu":
            a = g * _sigma(g)
            slope = _sigma(g) + a * _sigma(-g)
        else:
            z = 2.0 * _C1 * (g + _C2 * g ** 3)          # (1 + tanh(z / 2)) / 2 is the logistic function of z
            a = g * _sigma(z)
            slope = _sigma(z) + g * _sigma(z) * _sigma(-z) * 2.0 * _C1 * (1.0 + 3.0 * _C2 * g ** 2)
        if op == "gated":
            return (a * u, raw) if s["keep"] else a * u
        draw_ = torch.cat([s["dy"].to(d) * a, s["dy"].to(d) * u * slope], 1)
        return torch.mm(draw_, both), draw_
    B, R, C = max(1, s["B"]), s["R"], s["C"]
    gate = torch.ones((1, 1, C), dtype=d, device=_DEV) if s["gate"] is None else s["gate"].to(d).reshape(B, 1, C)
    y, r = s["y"].to(d).reshape(B, -1, C), s["r"].to(d).reshape(B, -1, C)
    post, pre = s["post"].to(d), s["pre"].to(d)
    ly = (y.square().sum(2, keepdim=True) / C + s["eps"]).sqrt()
    if op == "norm":
        new = s["scale"] * r + gate * post * y / ly
        x = pre * new / (new.square().sum(2, keepdim=True) / C + s["eps"]).sqrt()
        if s["int8"]:
            step = x.abs().amax(2, keepdim=True) / 127
            x = step * torch.round(x / step)
        return new.reshape(R, C), x.reshape(R, C)
    lr = (r.square().sum(2, keepdim=True) / C + s["eps"]).sqrt()
    dx, dr = s["dx"].to(d).reshape(B, -1, C), s["dr"].to(d).reshape(B, -1, C)
    q = dx * pre
    dr = dr + q / lr - r * ((q * r).sum(2, keepdim=True) / (C * lr ** 3))
    p = dr * gate * post
    dy = p / ly - y * ((p * y).sum(2, keepdim=True) / (C * ly ** 3))
    dgate = None if s["gate"] is None else (dr * post * y / ly).sum(1).reshape(s["gate"].shape)
    return ((s["scale"] * dr).reshape(R, C), dy.reshape(R, C), (dr * gate * y / ly).sum((0, 1)),
            (dx * r / lr).sum((0, 1)), dgate)
