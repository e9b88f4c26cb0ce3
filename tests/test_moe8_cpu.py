"""The mixture-of-experts entry points without a GPU: sizes, and refusals before any work is queued (no call here reaches
a kernel launch).  Pointers are addresses that are never dereferenced."""
import ctypes

import pytest

OK, ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = range(6)
P = 1 << 20
BF16, F32 = 0, 1
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def L():
    import bit_weight_only_offline_amd as Q
    return Q.lib()


def _bytes(f, *args):
    n = ctypes.c_size_t(77)
    return f(*args, ctypes.byref(n)), n.value


def test_packed_bytes(L):
    assert _bytes(L.qlinear_f8_packed_bytes, 1, 4096, 14336) == (OK, 4096 * 14336)
    assert _bytes(L.qlinear_f8_packed_bytes, 8, 17, 160) == (OK, 8 * 2 * 2 * 2048)      # whole tiles of 16 x 128
    for bad in ((0, 16, 64), (1, 0, 64), (1, 16, 0), (1, 16, 48), (1, 16, 131072), (1, (1 << 20) + 1, 64), (65537, 16, 64)):
        assert _bytes(L.qlinear_f8_packed_bytes, *bad)[0] == SHAPE, bad
    assert L.qlinear_f8_packed_bytes(1, 16, 64, None) == ARG


def test_workspaces(L):
    def forward(dtype):
        return lambda *a: L.qlinear_f8_workspace_bytes(*a[:-1], dtype, a[-1])
    assert L.qlinear_f8_workspace_bytes(5, 1, 64, 64, 0, 2, ctypes.byref(ctypes.c_size_t())) == ARG
    for f in (forward(BF16), forward(F32), L.qlinear_f8_backward_workspace_bytes):
        assert _bytes(f, 0, 1, 64, 64, 0) == (OK, 0)
        for bad in ((-1, 1, 64, 64, 0), (5, 1, 64, 100, 0), (5, 2, 64, 64, 0), (1 << 31, 1, 64, 64, 0), (5, 0, 64, 64, 1)):
            assert _bytes(f, *bad)[0] == SHAPE, bad
        assert _bytes(f, 5, 1, 64, 64, 2)[0] == ARG
        assert f(5, 1, 64, 64, 0, None) == ARG
        for M in (1, 1 << 24, BIG):
            for N in (1, 40, 300):
                for E, grouped in ((1, 0), (1, 1), (60, 1)):
                    assert _bytes(f, M, E, N, 32, grouped)[0] == OK
    st, n = _bytes(L.qlinear_f8_backward_workspace_bytes, 100, 3, 37, 64, 1)
    assert st == OK and n >= 100 * 40 * 2                                              # rows of 37 copied to rows of 40
    assert _bytes(L.qlinear_expert_order_workspace_bytes, 1000, 64) == (OK, 0)
    st, n = _bytes(L.qlinear_expert_order_workspace_bytes, 100000, 64)
    assert st == OK and n > 0
    for bad in ((-1, 4), (1 << 31, 4), (10, 0), (10, 1025)):
        assert _bytes(L.qlinear_expert_order_workspace_bytes, *bad)[0] == SHAPE, bad


def test_default_schedule(L):
    def f(M, E, N, K, grouped, backward, s, dtype=BF16):
        return L.qlinear_f8_default_schedule(M, E, N, K, grouped, backward, dtype, s)
    import bit_weight_only_offline_amd as Q
    s = Q.Schedule()
    assert f(4, 1, 64, 64, 0, 0, ctypes.byref(s)) == OK and s.tile in (0, 1) and s.splits == 1
    assert f(0, 1, 64, 64, 0, 0, ctypes.byref(s)) == SHAPE
    assert f(4, 1, 64, 64, 0, 2, ctypes.byref(s)) == ARG and f(4, 1, 64, 64, 0, 0, None) == ARG
    assert f(4, 8, 64, 64, 0, 0, ctypes.byref(s)) == SHAPE and f(4, 8, 64, 64, 1, 1, ctypes.byref(s)) == OK
    assert f(4, 1, 64, 64, 0, 0, ctypes.byref(s), F32) == OK and f(4, 1, 64, 64, 0, 0, ctypes.byref(s), 2) == ARG


def test_forward_refusals(L):
    def fwd(M=4, E=1, N=32, K=64, x=P, xs=P, cnt=None, w=P, ws=P, b=None, out=P, dt=BF16, space=None, n=0):
        return L.qlinear_f8_forward(x, xs, M, cnt, E, N, K, w, ws, b, out, dt, space, n, None)
    assert fwd(M=0, x=None, xs=None, out=None) == OK
    for kw in ({"x": None}, {"xs": None}, {"w": None}, {"ws": None}, {"out": None}, {"dt": 2}):
        assert fwd(**kw) == ARG, kw
    for kw in ({"K": 48}, {"K": 0}, {"N": 0}, {"M": -1}, {"M": 1 << 31}, {"E": 2}, {"E": 0, "cnt": P}):
        assert fwd(**kw) == SHAPE, kw
    for kw in ({"x": P + 8}, {"w": P + 8}, {"xs": P + 2}, {"ws": P + 2}, {"b": P + 1}, {"out": P + 1}, {"out": P + 2, "dt": F32},
               {"cnt": P + 2}):
        assert fwd(**kw) == ALIGN, kw
    assert fwd(M=BIG, N=1 << 20, K=32) == SHAPE                                        # no grid holds the tiles


def test_backward_refusals(L):
    def back(M=4, E=1, N=32, K=64, dy=P, cnt=None, w=P, ws=P, dx=P, space=P, n=1 << 40):
        return L.qlinear_f8_backward(dy, M, cnt, E, N, K, w, ws, dx, space, n, None)
    assert back(M=0, dy=None, dx=None) == OK
    for kw in ({"dy": None}, {"dx": None}, {"w": None}, {"ws": None}):
        assert back(**kw) == ARG, kw
    for kw in ({"K": 48}, {"N": 0}, {"M": -1}, {"E": 3}):
        assert back(**kw) == SHAPE, kw
    for kw in ({"dy": P + 2}, {"dx": P + 8}, {"w": P + 1}, {"ws": P + 1}, {"cnt": P + 1}):
        assert back(**kw) == ALIGN, kw
    assert back(N=37, space=None, n=0) == WORKSPACE and back(N=37, n=10) == WORKSPACE and back(N=37, space=P + 16) == ALIGN
    assert back(M=BIG, N=8, K=131040) == SHAPE


def test_quantiser_refusals(L):
    q = L.qlinear_f8_quantize
    assert q(None, BF16, 0, 0, 64, None, None, None) == OK
    assert q(P, 2, 0, 4, 64, P, P, None) == ARG and q(P, BF16, 2, 4, 64, P, P, None) == ARG
    assert q(P, BF16, 0, 4, 40, P, P, None) == SHAPE and q(P, BF16, 0, -1, 64, P, P, None) == SHAPE
    assert q(None, BF16, 0, 4, 64, P, P, None) == ARG and q(P, BF16, 0, 4, 64, None, P, None) == ARG
    assert q(P + 8, BF16, 0, 4, 64, P, P, None) == ALIGN and q(P, BF16, 0, 4, 64, P + 4, P, None) == ALIGN
    b = L.qlinear_f8_quantize_backward
    assert b(P, P, 4, 40, P, None) == SHAPE and b(P, None, 4, 64, P, None) == ARG and b(P, P + 2, 4, 64, P, None) == ALIGN
    d = L.qlinear_f8_dequantize
    assert d(P, P, 4, 40, P, BF16, None) == SHAPE and d(P, P, 4, 64, P, 5, None) == ARG and d(P, None, 4, 64, P, BF16, None) == ARG
    assert d(P + 4, P, 4, 64, P, BF16, None) == ALIGN
    w = L.qlinear_f8_quantize_weight
    assert w(P, BF16, 1, 4, 40, P, P, None) == SHAPE and w(P, 3, 1, 4, 64, P, P, None) == ARG and w(P + 2, BF16, 1, 4, 64, P, P, None) == ALIGN
    for f in (L.qlinear_f8_pack, L.qlinear_f8_unpack):
        assert f(1, 4, 40, P, P, None) == SHAPE and f(1, 4, 64, None, P, None) == ARG and f(1, 4, 64, P + 8, P, None) == ALIGN


def test_expert_order_refusals(L):
    def order(ids=P, size=8, n=100, E=8, c=P, r=P, s=P, space=None, b=0):
        return L.qlinear_expert_order(ids, size, n, E, c, r, s, space, b, None)
    for kw in ({"ids": None}, {"size": 2}, {"c": None}, {"r": None}, {"s": None}):
        assert order(**kw) == ARG, kw
    for kw in ({"n": -1}, {"n": 1 << 31}, {"E": 0}, {"E": 1025}):
        assert order(**kw) == SHAPE, kw
    for kw in ({"ids": P + 4}, {"ids": P + 2, "size": 4}, {"r": P + 2}):
        assert order(**kw) == ALIGN, kw
    assert order(n=1 << 20) == WORKSPACE and order(n=1 << 20, space=P + 16, b=1 << 30) == ALIGN


def test_row_refusals(L):
    def dispatch(x=P, dt=BF16, rows=P, T=4, k=2, D=64, out=P, codes=None, scales=None):
        return L.qlinear_dispatch(x, dt, rows, T, k, D, out, codes, scales, None)
    assert dispatch(T=0, x=None, rows=None, out=None) == OK
    for kw in ({"x": None}, {"rows": None}, {"out": None}, {"dt": 2}, {"codes": P}, {"scales": P}, {"codes": P, "scales": P}):
        assert dispatch(**kw) == ARG, kw
    for kw in ({"T": -1}, {"k": 0}, {"k": 257}, {"D": 0}, {"D": (1 << 24) + 1}, {"T": 1 << 30}, {"D": 40, "out": None, "codes": P, "scales": P}):
        assert dispatch(**kw) == SHAPE, kw
    for kw in ({"x": P + 1}, {"rows": P + 2}, {"out": P + 2, "dt": F32}, {"out": None, "codes": P + 4, "scales": P}):
        assert dispatch(**kw) == ALIGN, kw

    def combine(y=P, dt=BF16, rows=P, w=P, T=4, k=2, D=64, out=P):
        return L.qlinear_combine(y, dt, rows, w, T, k, D, out, None)
    assert combine(T=0) == OK
    for kw in ({"y": None}, {"rows": None}, {"out": None}, {"dt": 9}):
        assert combine(**kw) == ARG, kw
    assert combine(k=0) == SHAPE and combine(w=P + 2) == ALIGN

    def back(g=P, y=P, dt=BF16, rows=P, w=P, T=4, k=2, D=64, dy=P, dw=P):
        return L.qlinear_combine_backward(g, y, dt, rows, w, T, k, D, dy, dw, None)
    assert back(T=0) == OK
    for kw in ({"g": None}, {"y": None}, {"rows": None}, {"w": None}, {"dy": None}, {"dw": None}):
        assert back(**kw) == ARG, kw
    assert back(D=0) == SHAPE and back(dw=P + 1) == ALIGN


def test_python_refuses_cpu_tensors():
    torch = pytest.importorskip("torch")
    import bit_weight_only_offline_amd as Q
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    for call in (lambda: Q.quantize_f8(x), lambda: Q.quantize_weight_f8(x), lambda: Q.expert_order(torch.zeros((4, 2), dtype=torch.int32), 4),
                 lambda: Q.pack_f8(x.to(torch.float8_e4m3fn), torch.ones((1, 1)))):
        with pytest.raises(Q.QLinearError):
            call()
