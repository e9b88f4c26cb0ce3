"""8-bit feed-forward operators: token/channel-scaled int8 products, the gated projection
and the fused block norm, each with its backward pass.

Activations are int8 codes [..., K] with one float32 scale a token, as quantize_activations()
and block_norm(int8=True) return them; weights are packed once by pack_channel() or
pack_gated().  One sub-layer, forward:

    r, (q, s) = block_norm(r, y, post_weight=..., pre_weight=..., gate=..., int8=True)
    h = gated_i8(q, s, gated_weight)
    y = linear_i8(*quantize_activations(h), down_weight)

The weights are frozen: the backward passes give the gradients of the activations (the
quantisation passed straight through), of the pre-activations, norm weights and gates.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass

import torch

import bit_weight_only_offline_amd as _Q

__all__ = [
    "ChannelWeight", "GatedWeight", "pack_channel", "unpack_channel", "pack_gated", "unpack_gated", "GATE_ACTS",
    "i8_packed_bytes", "i8_default_schedule", "i8_workspace_bytes", "i8_backward_workspace_bytes", "linear_i8", "linear_i8_backward",
    "gated_i8", "gated_i8_backward", "block_norm_backward_workspace_bytes", "block_norm", "block_norm_backward",
]

GATE_ACTS = {"silu": 0, "gelu": 1}
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}


def bind(L: ctypes.CDLL) -> None:
    """Argument types of the entry points this module calls."""
    i64, sz, vp, ci, cf = ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    psz = ctypes.POINTER(sz)
    for name, args in {
        "qlinear_i8_packed_bytes": [i64, i64, ci, psz, psz],
        "qlinear_i8_pack": [i64, i64, vp, vp, vp, vp, vp, vp, vp],
        "qlinear_i8_unpack": [i64, i64, vp, vp, vp, vp, vp, vp, vp],
        "qlinear_i8_default_schedule": [i64, i64, i64, ci, ci, ctypes.POINTER(_Q.Schedule)],
        "qlinear_i8_workspace_bytes": [i64, i64, i64, ci, psz],
        "qlinear_i8_backward_workspace_bytes": [i64, i64, i64, ci, psz],
        "qlinear_i8_forward": [vp, vp, i64, i64, i64, vp, vp, vp, vp, ci, vp, sz, vp],
        "qlinear_i8_gated_forward": [vp, vp, i64, i64, i64, vp, vp, vp, ci, vp, ci, vp, vp, sz, vp],
        "qlinear_i8_backward": [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp],
        "qlinear_i8_gated_backward": [vp, vp, i64, i64, i64, vp, vp, ci, vp, vp, vp, sz, vp],
        "qlinear_block_norm": [vp, ci, vp, vp, vp, vp, ci, i64, cf, cf, i64, i64, vp, vp, vp, vp, vp],
        "qlinear_block_norm_backward_workspace_bytes": [i64, i64, i64, psz],
        "qlinear_block_norm_backward": [vp, vp, vp, ci, vp, vp, vp, vp, ci, i64, cf, cf, i64, i64, vp, vp, vp, vp, vp,
                                        vp, sz, vp],
    }.items():
        f = getattr(L, name)
        f.restype = ci
        f.argtypes = args


# A decoded token's product takes a few microseconds on the GPU, so the wrappers are written
# for few Python operations: messages are built only when a check fails, and the stream and
# the current device are read without building objects.

def _call(name: str, device: torch.device, *args) -> None:
    """One entry point on the device's current stream, with that device current."""
    index = device.index
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(name, device, *args)
    status = getattr(_Q._lib or _Q.lib(), name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        _Q._check(status, name)


def _fail(message: str):
    raise _Q.QLinearError(message)


def _need(ok: bool, message: str) -> None:
    if not ok:
        raise _Q.QLinearError(message)


def _tensor(t, name: str, dtypes, device=None) -> torch.Tensor:
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and not t.requires_grad and t.is_cuda
            and (device is None or t.device == device)):
        return t
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        _fail(f"{name} must be a tensor of {' or '.join(str(d).replace('torch.', '') for d in dtypes)}")
    if t.requires_grad:
        _fail(f"{name} must not require grad: call the backward functions")
    if not t.is_cuda:
        _fail("the library runs on a HIP device only")
    _fail(f"{name} must be on {device}")


def _out(out, shape, dtype, device, name="out") -> torch.Tensor:
    if out is None:
        return torch.empty(*shape, dtype=dtype, device=device)   # (shape,) takes 0.35 us longer to parse
    if (not isinstance(out, torch.Tensor) or out.dtype != dtype or out.shape != shape or not out.is_contiguous()
            or out.device != device):
        _fail(f"{name} must be a contiguous {tuple(shape)} tensor of {dtype} on {device}")
    if out.requires_grad:
        _fail(f"{name} must not require grad: it is written without a record of it")
    return out


def _space(workspace, need: int, device):
    """The caller's workspace, or a new one; None where none is needed.  It is held until the
    call has queued its work."""
    return None if need == 0 else _Q._space(workspace, need, device)


def _aligned(t: torch.Tensor) -> torch.Tensor:
    """Contiguous, and on a 16-byte boundary (a view may start anywhere)."""
    if not t.is_contiguous():
        t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


@functools.lru_cache(maxsize=4096)
def _sizes(name: str, *args) -> int:
    n = ctypes.c_size_t()
    _Q._check(getattr(_Q.lib(), name)(*args, ctypes.byref(n)), name)
    return n.value


def i8_packed_bytes(N: int, K: int, gated: bool = False):
    """(w_bytes, s_bytes) of a packed weight."""
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    _Q._check(_Q.lib().qlinear_i8_packed_bytes(N, K, int(gated), ctypes.byref(w), ctypes.byref(s)),
              "qlinear_i8_packed_bytes")
    return w.value, s.value


def i8_default_schedule(M: int, N: int, K: int, gated: bool = False, backward: bool = False):
    """The Schedule (tile, splits) that a product, or its backward pass, takes at these sizes."""
    s = _Q.Schedule()
    _Q._check(_Q.lib().qlinear_i8_default_schedule(M, N, K, int(gated), int(backward), ctypes.byref(s)),
              "qlinear_i8_default_schedule")
    return s


def i8_workspace_bytes(M: int, N: int, K: int, gated: bool = False) -> int:
    return _sizes("qlinear_i8_workspace_bytes", M, N, K, int(gated))


def i8_backward_workspace_bytes(M: int, N: int, K: int, gated: bool = False) -> int:
    return _sizes("qlinear_i8_backward_workspace_bytes", M, N, K, int(gated))


def block_norm_backward_workspace_bytes(R: int, C: int, gates: int = 0) -> int:
    return _sizes("qlinear_block_norm_backward_workspace_bytes", R, C, gates)


@dataclass
class ChannelWeight:
    """An int8 weight [N, K] with one float32 scale a channel, in operand order."""
    N: int
    K: int
    w: torch.Tensor
    s: torch.Tensor
    gated = False

    def __post_init__(self):
        self.device = self.w.device


@dataclass
class GatedWeight:
    """Two such weights (up and gate, [N, K] each), interleaved."""
    N: int
    K: int
    w: torch.Tensor
    s: torch.Tensor
    gated = True

    def __post_init__(self):
        self.device = self.w.device


def _canonical(codes, scales, name, device=None, shape=None):
    _tensor(codes, f"{name} codes", (torch.int8,), device)
    _tensor(scales, f"{name} scales", (torch.float32,), codes.device)
    _need(codes.dim() == 2 and scales.shape == codes.shape[:1], f"{name}: codes [N, K] and scales [N]")
    _need(shape is None or codes.shape == shape, "up and gate must have the same shape")
    return codes.contiguous(), scales.contiguous()


def _pack(cls, up, gate):
    N, K = up[0].shape
    dev = up[0].device
    wb, sb = i8_packed_bytes(N, K, gate is not None)
    w = torch.empty(wb, dtype=torch.uint8, device=dev)
    s = torch.empty(sb, dtype=torch.uint8, device=dev)
    g = (None, None) if gate is None else (gate[0].data_ptr(), gate[1].data_ptr())
    _call("qlinear_i8_pack", dev, N, K, up[0].data_ptr(), up[1].data_ptr(), *g, w.data_ptr(), s.data_ptr())
    return cls(N, K, w, s)


def pack_channel(codes: torch.Tensor, scales: torch.Tensor) -> ChannelWeight:
    """Pack int8 codes [N, K] and float32 channel scales [N] (quantize_activations() of a
    bf16 weight gives both), once."""
    return _pack(ChannelWeight, _canonical(codes, scales, "weight"), None)


def pack_gated(up_codes: torch.Tensor, up_scales: torch.Tensor, gate_codes: torch.Tensor,
               gate_scales: torch.Tensor) -> GatedWeight:
    """Pack the up and gate projections of a gated feed-forward block together."""
    up = _canonical(up_codes, up_scales, "up")
    return _pack(GatedWeight, up, _canonical(gate_codes, gate_scales, "gate", up[0].device, up[0].shape))


def _unpack(pw):
    outs = []
    for _ in range(2 if pw.gated else 1):
        outs += [torch.empty((pw.N, pw.K), dtype=torch.int8, device=pw.device),
                 torch.empty((pw.N,), dtype=torch.float32, device=pw.device)]
    ptrs = [t.data_ptr() for t in outs] + [None] * (4 - len(outs))
    _call("qlinear_i8_unpack", pw.device, pw.N, pw.K, pw.w.data_ptr(), pw.s.data_ptr(), *ptrs)
    return tuple(outs)


def unpack_channel(pw: ChannelWeight):
    """(codes, scales), exactly as packed."""
    _need(isinstance(pw, ChannelWeight), "a ChannelWeight is needed")
    return _unpack(pw)


def unpack_gated(pw: GatedWeight):
    """(up_codes, up_scales, gate_codes, gate_scales), exactly as packed."""
    _need(isinstance(pw, GatedWeight), "a GatedWeight is needed")
    return _unpack(pw)


def _activations(codes, scales, pw):
    _tensor(codes, "codes", (torch.int8,), pw.device)
    _tensor(scales, "scales", (torch.float32,), pw.device)
    shape = codes.shape
    if not shape or shape[-1] != pw.K:
        _fail(f"codes must be [..., {pw.K}]")
    M = codes.numel() // pw.K
    lead, given = shape[:-1], scales.shape
    # one value a token, in the tokens' shape or in a row, ones aside; another shape as large holds
    # them in another order
    if given != lead:
        long = [d for d in given if d != 1]
        if long != [d for d in lead if d != 1] and long != ([M] if M != 1 else []):
            _fail(f"scales must be {tuple(lead)}")
    return lead, M, _aligned(codes), scales.contiguous()


def _bias(bias, n, pw):
    if bias is None:
        return None
    _tensor(bias, "bias", (torch.bfloat16,), pw.device)
    if bias.numel() != n:
        _fail(f"bias must have {n} values")
    return bias.contiguous()


def linear_i8(codes: torch.Tensor, scales: torch.Tensor, pw: ChannelWeight, bias: torch.Tensor | None = None,
              out_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None) -> torch.Tensor:
    """y[..., N] = (codes . q^T) * scales * channel scales + bias, summed exactly in int32.

    codes int8 [..., K], scales float32 [...] (or one row of them), bias bf16 [N]; out_dtype bf16
    or float32."""
    _need(isinstance(pw, ChannelWeight), "pw must be a ChannelWeight")
    _need(out_dtype in _DTYPES, "out_dtype must be bfloat16 or float32")
    lead, M, codes, scales = _activations(codes, scales, pw)
    bias = _bias(bias, pw.N, pw)
    out = _out(out, (*lead, pw.N), out_dtype, pw.device)
    need = i8_workspace_bytes(M, pw.N, pw.K)
    ws = _space(workspace, need, pw.device)
    _call("qlinear_i8_forward", pw.device, codes.data_ptr(), scales.data_ptr(), M, pw.N, pw.K, pw.w.data_ptr(),
          pw.s.data_ptr(), None if bias is None else bias.data_ptr(), out.data_ptr(), _DTYPES[out_dtype], _p(ws), need)
    return out


def gated_i8(codes: torch.Tensor, scales: torch.Tensor, pw: GatedWeight, bias: torch.Tensor | None = None,
             act: str = "silu", keep_raw: bool = False, out_dtype: torch.dtype = torch.bfloat16,
             out: torch.Tensor | None = None, raw: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """h[..., N] = act(gate) * up, both projections of codes in one kernel.

    bias bf16 [2N] = [up | gate]; act "silu" or "gelu" (tanh form).  keep_raw: returns
    (h, raw) with raw bf16 [..., 2N] = [up | gate] before the activation, which
    gated_i8_backward() reads (`raw` may also be given to be written into)."""
    _need(isinstance(pw, GatedWeight), "pw must be a GatedWeight")
    if act not in GATE_ACTS:
        _fail(f"act must be one of {sorted(GATE_ACTS)}")
    _need(out_dtype in _DTYPES, "out_dtype must be bfloat16 or float32")
    lead, M, codes, scales = _activations(codes, scales, pw)
    bias = _bias(bias, 2 * pw.N, pw)
    out = _out(out, (*lead, pw.N), out_dtype, pw.device)
    if keep_raw or raw is not None:
        raw = _out(raw, (*lead, 2 * pw.N), torch.bfloat16, pw.device, "raw")
    need = i8_workspace_bytes(M, pw.N, pw.K, True)
    ws = _space(workspace, need, pw.device)
    _call("qlinear_i8_gated_forward", pw.device, codes.data_ptr(), scales.data_ptr(), M, pw.N, pw.K, pw.w.data_ptr(),
          pw.s.data_ptr(), None if bias is None else bias.data_ptr(), GATE_ACTS[act], out.data_ptr(),
          _DTYPES[out_dtype], None if raw is None else raw.data_ptr(), _p(ws), need)
    return out if raw is None else (out, raw)


def linear_i8_backward(dy: torch.Tensor, pw: ChannelWeight, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dx bf16 [..., K] = (dy * channel scales) . q for dy bf16 [..., N]: the gradient of the
    dequantised activations.  The gradient of a bias is dy summed over the tokens."""
    _need(isinstance(pw, ChannelWeight), "pw must be a ChannelWeight")
    _tensor(dy, "dy", (torch.bfloat16,), pw.device)
    if not dy.shape or dy.shape[-1] != pw.N:
        _fail(f"dy must be [..., {pw.N}]")
    dy = _aligned(dy)
    M = dy.numel() // pw.N
    out = _out(out, (*dy.shape[:-1], pw.K), torch.bfloat16, pw.device)
    need = i8_backward_workspace_bytes(M, pw.N, pw.K)
    ws = _space(workspace, need, pw.device)
    _call("qlinear_i8_backward", pw.device, dy.data_ptr(), M, pw.N, pw.K, pw.w.data_ptr(), pw.s.data_ptr(),
          out.data_ptr(), _p(ws), need)
    return out


def gated_i8_backward(dh: torch.Tensor, raw: torch.Tensor, pw: GatedWeight, act: str = "silu",
                      out: torch.Tensor | None = None, draw: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None):
    """(dx bf16 [..., K], draw bf16 [..., 2N]) for dh bf16 [..., N] and the raw [up | gate]
    that gated_i8(keep_raw=True) returned; draw is the gradient of raw, and its sum over the
    tokens that of the bias."""
    _need(isinstance(pw, GatedWeight), "pw must be a GatedWeight")
    if act not in GATE_ACTS:
        _fail(f"act must be one of {sorted(GATE_ACTS)}")
    _tensor(dh, "dh", (torch.bfloat16,), pw.device)
    _tensor(raw, "raw", (torch.bfloat16,), pw.device)
    lead = dh.shape[:-1]
    if not dh.shape or dh.shape[-1] != pw.N:
        _fail(f"dh must be [..., {pw.N}]")
    if raw.shape != (*lead, 2 * pw.N):
        _fail(f"raw must be {(*lead, 2 * pw.N)}")
    dh, raw = _aligned(dh), _aligned(raw)
    M = dh.numel() // pw.N
    out = _out(out, (*lead, pw.K), torch.bfloat16, pw.device)
    draw = _out(draw, (*lead, 2 * pw.N), torch.bfloat16, pw.device, "draw")
    need = i8_backward_workspace_bytes(M, pw.N, pw.K, True)
    ws = _space(workspace, need, pw.device)
    _call("qlinear_i8_gated_backward", pw.device, dh.data_ptr(), raw.data_ptr(), M, pw.N, pw.K, pw.w.data_ptr(),
          pw.s.data_ptr(), GATE_ACTS[act], out.data_ptr(), draw.data_ptr(), _p(ws), need)
    return out, draw


_FLOATS = (torch.bfloat16, torch.float32)


def _norm_args(residual, y, post_weight, pre_weight, gate, eps):
    """Checked arguments of both directions: (rows, C, gates, parameter dtype)."""
    _tensor(residual, "residual", _FLOATS)
    shape, dev = residual.shape, residual.device
    if not shape or shape[-1] == 0:
        _fail("residual must be [..., C]")
    C = shape[-1]
    R = residual.numel() // C
    if y is not None:
        _tensor(y, "y", (torch.bfloat16,), dev)
        if y.shape != shape:
            _fail("y must have the residual's shape")
    elif post_weight is not None or gate is not None:
        _fail("post_weight and gate need y")
    dtype, gates = None, 0
    allowed = _FLOATS
    for p in (post_weight, pre_weight, gate):
        if p is None:
            continue
        _tensor(p, "weights and gate", allowed, dev)
        if dtype is None:
            dtype = p.dtype
            allowed = (dtype,)
    for p in (post_weight, pre_weight):
        if p is not None and p.shape != (C,):
            _fail("a norm weight must be [C]")
    if gate is not None:
        if gate.dim() not in (1, 2) or gate.shape[-1] != C:
            _fail("gate must be [C] or [B, C]")
        gates = 1 if gate.dim() == 1 else gate.shape[0]
        if gates == 0 or R % gates:
            _fail("the rows must divide evenly among the gates")
    if not eps > 0.0:
        _fail("eps must be positive")
    return R, C, gates, 1 if dtype is None else _DTYPES[dtype]


def _c(t):
    """Contiguous, or None."""
    return t if t is None or t.is_contiguous() else t.contiguous()


def _p(t):
    return None if t is None else t.data_ptr()


def block_norm(residual: torch.Tensor, y: torch.Tensor | None = None, *, post_weight: torch.Tensor | None = None,
               pre_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, residual_scale: float = 1.0,
               eps: float = 1e-6, int8: bool = False, residual_out: torch.Tensor | None = None):
    """The step between two blocks: (r', x) with

        r' = residual_scale * residual + gate * rms_norm(y) * post_weight
        x  = rms_norm(r') * pre_weight

    residual bf16 or float32 [..., C], y bf16 [..., C] (the finished block's output; None
    before the first block); post_weight None: y enters unnormed; pre_weight None: x is None.
    gate [C], or [B, C] with one gate for each of B equal runs of rows.  x is bf16, or with
    int8=True the pair (codes int8 [..., C], scales float32 [...]) that linear_i8() and
    gated_i8() take.  residual_out may be the residual itself (in place)."""
    R, C, gates, dt = _norm_args(residual, y, post_weight, pre_weight, gate, eps)
    shape, dev = residual.shape, residual.device
    residual, y, post_weight, pre_weight, gate = _c(residual), _c(y), _c(post_weight), _c(pre_weight), _c(gate)
    if int8 and pre_weight is None:
        _fail("int8 output needs pre_weight")
    r_out = torch.empty_like(residual) if residual_out is None else \
        _out(residual_out, shape, residual.dtype, dev, "residual_out")
    x = codes = scales = None
    if pre_weight is not None:
        if int8:
            codes = torch.empty_like(residual, dtype=torch.int8)
            scales = residual.new_empty(shape[:-1], dtype=torch.float32)
        else:
            x = torch.empty_like(residual, dtype=torch.bfloat16)
    _call("qlinear_block_norm", dev, residual.data_ptr(), _DTYPES[residual.dtype], _p(y), _p(post_weight),
          _p(pre_weight), _p(gate), dt, gates, residual_scale, eps, R, C, r_out.data_ptr(), _p(x), _p(codes), _p(scales))
    return r_out, ((codes, scales) if int8 else x)


def block_norm_backward(dx: torch.Tensor | None, dresidual: torch.Tensor | None, residual_out: torch.Tensor,
                        y: torch.Tensor | None = None, *, post_weight: torch.Tensor | None = None,
                        pre_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None,
                        residual_scale: float = 1.0, eps: float = 1e-6, workspace: torch.Tensor | None = None):
    """Gradients (residual, y, post_weight, pre_weight, gate) of block_norm().

    dx bf16 [..., C]: gradient of x (None without pre_weight; for int8 output the gradient of
    the dequantised x); dresidual: gradient of r' from the rest of the network (its dtype), or
    None; residual_out and y as the forward pass returned and took them.  Parameter gradients
    are float32, None for parameters that are not given; their sums have a fixed order."""
    R, C, gates, dt = _norm_args(residual_out, y, post_weight, pre_weight, gate, eps)
    dev = residual_out.device
    residual_out, y, post_weight, pre_weight, gate = (_c(residual_out), _c(y), _c(post_weight), _c(pre_weight),
                                                      _c(gate))
    _need((dx is not None) == (pre_weight is not None), "dx and pre_weight go together")
    if dx is not None:
        _tensor(dx, "dx", (torch.bfloat16,), dev)
        _need(dx.shape == residual_out.shape, "dx must have the residual's shape")
        dx = dx.contiguous()
    if dresidual is not None:
        _tensor(dresidual, "dresidual", (residual_out.dtype,), dev)
        _need(dresidual.shape == residual_out.shape, "dresidual must have the residual's shape")
        dresidual = dresidual.contiguous()
    dr = torch.empty_like(residual_out)
    dy = None if y is None else torch.empty_like(y)
    dpost, dpre, dgate = [None if t is None else torch.empty_like(t, dtype=torch.float32)
                          for t in (post_weight, pre_weight, gate)]
    need = block_norm_backward_workspace_bytes(R, C, gates)
    ws = _space(workspace, need, dev)
    _call("qlinear_block_norm_backward", dev, _p(dx), _p(dresidual), _p(residual_out), _DTYPES[residual_out.dtype],
          _p(y), _p(post_weight), _p(pre_weight), _p(gate), dt, gates, residual_scale, eps, R, C, _p(dr), _p(dy),
          _p(dpost), _p(dpre), _p(dgate), _p(ws), need)
    return dr, dy, dpost, dpre, dgate
