"""Host checks of the dense product's workspaces and sizes, on the CPU."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def lib():
    from combine_moe_layout_03_amd import capi

    return capi.lib()


D, NULL = C.c_void_p(256), None
SHAPE, WORKSPACE = -2, -6


@pytest.mark.parametrize("T,N,Cc", [(7, 4096, 264), (1001, 264, 520)])  # d_x, d_w in parts
def test_gradients_refuse_a_small_workspace(lib, T, N, Cc):
    need = lib.moe_linear_grad_workspace_bytes(T, N, Cc)
    assert need > 0

    def call(ws, n, dx=D, dw=D):
        return lib.moe_linear_grad(T, N, Cc, D, D, D, dx, dw, ws, n, None)

    for kw in ({}, dict(dx=NULL), dict(dw=NULL)):
        assert call(D, need - 1, **kw) == WORKSPACE
        assert call(NULL, need, **kw) == WORKSPACE
        assert call(D, 0, **kw) == WORKSPACE


def test_refused_sizes_need_no_workspace(lib):
    """T*N, T*C and N*C are at most 2^36; the workspace of a refused size is 0."""
    big = 1 << 20
    for T, N, Cc in ((1 << 17, big, 8), (1 << 17, 8, big), (8, big, 1 << 17), (-1, 8, 8),
                     (8, 12, 8), (8, 8, 12)):
        assert lib.moe_linear(T, N, Cc, D, D, None, None, D, None, 0, None, 0, None) == SHAPE
        assert lib.moe_linear_grad(T, N, Cc, D, D, D, D, D, None, 0, None) == SHAPE
        assert lib.moe_linear_workspace_bytes(T, N, Cc, 0) == 0
        assert lib.moe_linear_grad_workspace_bytes(T, N, Cc) == 0
    assert lib.moe_linear_act_grad(1 << 17, big, D, D, D, D, 1, None, 0, None) == SHAPE
    assert lib.moe_linear_act_grad_workspace_bytes(1 << 17, big, 1) == 0
