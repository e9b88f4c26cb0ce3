"""Shapes at the launch limits of the 8-bit entry points, without a GPU: what no grid holds is
refused before anything is queued.  Pointers are addresses that are never dereferenced."""
import ctypes

import pytest

OK, ARG, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, HIP = range(7)
P = 1 << 20
BIG = (1 << 31) - 1


@pytest.fixture(scope="module")
def L():
    import bit_weight_only_offline_amd as Q
    return Q.lib()


def test_products_that_no_grid_holds(L):
    """2^32 threads of a backward product: tiles of 256 rows by 256 inputs, 512 threads each."""
    def back(M, N, K):
        return L.qlinear_i8_backward(P, M, N, K, P, P, P, P, 1 << 62, None)
    assert back(BIG, 8, 32) == SHAPE                               # 2^23 tiles
    assert back(BIG // 2, 8, 288) == SHAPE                         # 2^22, twice
    assert L.qlinear_i8_gated_backward(P, P, BIG, 8, 32, P, P, 0, P, P, P, 1 << 62, None) == SHAPE


def test_forward_tiles_past_what_an_index_holds(L):
    def lin(M, N, K):
        return L.qlinear_i8_forward(P, P, M, N, K, P, P, None, P, 0, P, 1 << 62, None)
    assert lin(BIG, 1 << 20, 32) == SHAPE
    assert L.qlinear_i8_gated_forward(P, P, BIG, 1 << 20, 32, P, P, None, 0, P, 0, None, P, 1 << 62, None) == SHAPE


def test_gates_past_what_an_index_holds(L):
    n = ctypes.c_size_t()
    assert L.qlinear_block_norm_backward_workspace_bytes(0, 64, 1 << 31, ctypes.byref(n)) == SHAPE
    assert L.qlinear_block_norm_backward_workspace_bytes(0, 64, BIG, ctypes.byref(n)) == OK


@pytest.mark.parametrize("gated", [0, 1])
def test_no_schedule_past_the_limit(L, gated):
    """Rows by the billion, few channels: tiles that would need too many workgroups are not
    chosen where larger ones fit, so the workspace query has an answer for every shape."""
    n = ctypes.c_size_t()
    for M in (1 << 24, 1 << 28, BIG):
        for N in (1, 16, 40, 300):
            for f in (L.qlinear_i8_workspace_bytes, L.qlinear_i8_backward_workspace_bytes):
                assert f(M, N, 32, gated, ctypes.byref(n)) == OK


def test_default_schedule(L):
    import bit_weight_only_offline_amd as Q
    s = Q.i8_default_schedule(1, 4096, 14336)
    assert (s.tile, s.splits) == (0, 1)
    assert Q.i8_default_schedule(4, 14336, 4096, gated=True).tile == 1
    s = Q.i8_default_schedule(2048, 14336, 4096, gated=True, backward=True)
    assert (s.tile, s.splits) == (0, 2)
    out = Q.Schedule()
    f = L.qlinear_i8_default_schedule
    assert f(4, 64, 64, 0, 2, ctypes.byref(out)) == ARG and f(4, 64, 64, 2, 0, ctypes.byref(out)) == ARG
    assert f(4, 64, 64, 0, 0, None) == ARG
    assert f(0, 64, 64, 0, 0, ctypes.byref(out)) == SHAPE and f(4, 64, 40, 0, 1, ctypes.byref(out)) == SHAPE
    for gated in (0, 1):
        for M in (1, 16, 17, 100, 3000):                      # a workspace exactly where the forward splits
            n = ctypes.c_size_t()
            assert L.qlinear_i8_workspace_bytes(M, 4099, 12000, gated, ctypes.byref(n)) == OK
            assert f(M, 4099, 12000, gated, 0, ctypes.byref(out)) == OK and (n.value > 0) == (out.splits > 1)
