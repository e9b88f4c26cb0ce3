"""The 8-bit feed-forward entry points without a GPU: sizes, and refusals before any work is
queued (no call here reaches a kernel launch).  Pointers are addresses that are never
dereferenced."""
import ctypes

import pytest

OK, ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = range(6)
P = 1 << 20
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    import bit_weight_only_offline_amd as Q
    return Q.lib()


def _bytes(f, *args):
    n = ctypes.c_size_t(77)
    return f(*args, ctypes.byref(n)), n.value


def test_packed_bytes(L):
    def sizes(N, K, gated):
        w, s = ctypes.c_size_t(), ctypes.c_size_t()
        return L.qlinear_i8_packed_bytes(N, K, gated, ctypes.byref(w), ctypes.byref(s)), w.value, s.value
    assert sizes(4096, 14336, 0) == (OK, 4096 * 14336, 4096 * 4)
    assert sizes(14336, 4096, 1) == (OK, 2 * 14336 * 4096, 2 * 14336 * 4)
    assert sizes(17, 96, 0) == (OK, 2 * 2 * 1024, 256)              # whole tiles of 16 x 64
    assert sizes(17, 96, 1) == (OK, 4 * 2 * 1024, 256)
    for bad in ((0, 64, 0), (16, 0, 0), (16, 48, 0), (16, 131072, 0), ((1 << 20) + 1, 64, 0), (-1, 64, 0)):
        assert sizes(*bad)[0] == SHAPE, bad
    assert sizes(16, 64, 2)[0] == ARG
    assert L.qlinear_i8_packed_bytes(16, 64, 0, None, None) == ARG


def test_workspaces(L):
    assert _bytes(L.qlinear_i8_workspace_bytes, 0, 64, 64, 0) == (OK, 0)
    assert _bytes(L.qlinear_i8_workspace_bytes, 16, 4096, 4096, 0) == (OK, 0)      # few rows: no split
    assert _bytes(L.qlinear_i8_workspace_bytes, 5, 64, 100, 0)[0] == SHAPE
    assert _bytes(L.qlinear_i8_workspace_bytes, -1, 64, 64, 0)[0] == SHAPE
    st, n = _bytes(L.qlinear_i8_backward_workspace_bytes, 100, 40, 64, 0)
    assert st == OK and n >= 100 * 40 * 2                                          # the scaled gradients
    st, n = _bytes(L.qlinear_i8_backward_workspace_bytes, 100, 37, 64, 1)
    assert st == OK and n >= 100 * 48 * 4
    st, n = _bytes(L.qlinear_block_norm_backward_workspace_bytes, 1000, 64, 1)
    assert st == OK and n > 0
    assert _bytes(L.qlinear_block_norm_backward_workspace_bytes, 0, 64, 1)[0] == OK
    for bad in ((10, 0, 1), (10, 32769, 1), (-1, 64, 1), (10, 64, 3), (10, 64, -1)):
        assert _bytes(L.qlinear_block_norm_backward_workspace_bytes, *bad)[0] == SHAPE, bad


def test_pack_refusals(L):
    def pack(N=32, K=64, c=P, s=P, gc=None, gs=None, w=P, ps=P):
        return L.qlinear_i8_pack(N, K, c, s, gc, gs, w, ps, None)
    assert pack(K=40) == SHAPE
    for kw in ({"c": None}, {"s": None}, {"w": None}, {"ps": None}, {"gc": P}, {"gs": P}):
        assert pack(**kw) == ARG, kw
    for kw in ({"s": P + 2}, {"w": P + 8}, {"ps": P + 4}, {"gc": P, "gs": P + 1}):
        assert pack(**kw) == ALIGN, kw
    assert L.qlinear_i8_unpack(32, 64, P, P, None, P, None, None, None) == ARG


def test_forward_refusals(L):
    def lin(M=70, N=64, K=64, x=P, xs=P, w=P, ps=P, b=None, out=P, dt=BF16, ws=P, nws=1 << 30):
        return L.qlinear_i8_forward(x, xs, M, N, K, w, ps, b, out, dt, ws, nws, None)
    assert lin(M=-1) == SHAPE and lin(K=65) == SHAPE and lin(N=0) == SHAPE
    assert lin(dt=2) == ARG and lin(x=None) == ARG and lin(xs=None) == ARG and lin(out=None) == ARG and lin(w=None) == ARG
    assert lin(x=P + 8) == ALIGN and lin(out=P + 1) == ALIGN and lin(out=P + 2, dt=F32) == ALIGN and lin(b=P + 1) == ALIGN
    assert lin(M=0, x=None, xs=None, out=None, ws=None, nws=0) == OK               # no rows: nothing to do
    M, N, K = 65, 1024, 14336                                                      # a split input dimension
    need = _bytes(L.qlinear_i8_workspace_bytes, M, N, K, 0)[1]
    assert need > 0
    assert lin(M, N, K, ws=None) == WORKSPACE and lin(M, N, K, nws=need - 1) == WORKSPACE
    assert lin(M, N, K, ws=P + 16) == ALIGN
    assert L.qlinear_i8_gated_forward(P, P, 4, 64, 64, P, P, None, 2, P, BF16, None, None, 0, None) == ARG
    assert L.qlinear_i8_gated_forward(P, P, 4, 64, 64, P, P, None, 0, P, BF16, P + 1, None, 0, None) == ALIGN


def test_backward_refusals(L):
    def back(M=4, N=64, K=64, dy=P, w=P, ps=P, dx=P, ws=P, nws=1 << 30):
        return L.qlinear_i8_backward(dy, M, N, K, w, ps, dx, ws, nws, None)
    assert back(K=10) == SHAPE and back(dy=None) == ARG and back(dx=None) == ARG and back(w=None) == ARG
    assert back(dy=P + 4) == ALIGN and back(dx=P + 8) == ALIGN
    assert back(ws=None) == WORKSPACE and back(nws=16) == WORKSPACE and back(ws=P + 64) == ALIGN
    assert back(M=0, dy=None, dx=None, ws=None, nws=0) == OK
    def gated(raw=P, draw=P, act=0):
        return L.qlinear_i8_gated_backward(P, raw, 4, 64, 64, P, P, act, P, draw, P, 1 << 30, None)
    assert gated(raw=None) == ARG and gated(draw=None) == ARG and gated(act=3) == ARG and gated(raw=P + 2) == ALIGN


def _norm(L, r=P, rdt=F32, y=P, post=P, pre=P, gate=P, pdt=F32, gates=1, scale=1.0, eps=1e-6, R=4, C=64, out=P, x=P,
          codes=None, scales=None):
    return L.qlinear_block_norm(r, rdt, y, post, pre, gate, pdt, gates, scale, eps, R, C, out, x, codes, scales, None)


def test_block_norm_refusals(L):
    for kw in ({"R": -1}, {"C": 0}, {"C": 32769}, {"gates": 3}, {"gates": -1}):
        assert _norm(L, **kw) == SHAPE, kw
    for kw in ({"eps": 0.0}, {"eps": -1.0}, {"eps": float("nan")}, {"scale": float("inf")}, {"rdt": 5}, {"pdt": -1},
               {"gates": 0}, {"gate": None}, {"y": None}, {"codes": P}, {"codes": P, "scales": P}, {"x": None},
               {"pre": None}, {"r": None}, {"out": None}):
        assert _norm(L, **kw) == ARG, kw
    for kw in ({"r": P + 2}, {"y": P + 1}, {"post": P + 2}, {"x": P + 1}, {"x": None, "codes": P, "scales": P + 2}):
        assert _norm(L, **kw) == ALIGN, kw
    assert _norm(L, R=0, r=None, out=None, x=None, y=None) == OK


def test_block_norm_backward_refusals(L):
    def back(dx=P, dres=P, r=P, rdt=F32, y=P, post=P, pre=P, gate=P, gates=1, eps=1e-6, R=4, C=64, dr=P, dy=P, dpost=P,
             dpre=P, dgate=P, ws=P, nws=1 << 30):
        return L.qlinear_block_norm_backward(dx, dres, r, rdt, y, post, pre, gate, F32, gates, 1.0, eps, R, C, dr, dy,
                                             dpost, dpre, dgate, ws, nws, None)
    for kw in ({"dx": None}, {"pre": None, "dpre": None}, {"dpost": None}, {"dgate": None}, {"dy": None}, {"dr": None},
               {"y": None}, {"r": None}, {"eps": 0.0}, {"gates": 0}):
        assert back(**kw) == ARG, kw
    assert back(ws=None) == WORKSPACE and back(nws=100) == WORKSPACE and back(ws=P + 8) == ALIGN
    assert back(dr=P + 2) == ALIGN and back(dpre=P + 1) == ALIGN and back(C=40000) == SHAPE


def test_wrappers_refuse_tensors_off_the_gpu():
    torch = pytest.importorskip("torch")
    import bit_weight_only_offline_amd as Q
    codes, scales = torch.zeros((32, 64), dtype=torch.int8), torch.ones(32)
    for call in (lambda: Q.pack_channel(codes, scales), lambda: Q.pack_gated(codes, scales, codes, scales),
                 lambda: Q.block_norm(torch.zeros(4, 8)),
                 lambda: Q.block_norm_backward(None, None, torch.zeros(4, 8))):
        with pytest.raises(Q.QLinearError):
            call()
    with pytest.raises(Q.QLinearError):
        Q.linear_i8(codes, scales, None)
