"""Sizes of the routers' workspaces: they do not fall as the batch grows, each entry point asks for its own."""
import ctypes as C

import pytest


def _lib():
    import fine_grained_blockwise_amd as fgb
    return fgb.lib()


@pytest.mark.parametrize("E", [1, 8, 32, 33, 64, 128, 129, 256, 384, 512, 513, 1024])
def test_sizes_never_fall(E):
    L = _lib()
    for size in (L.moe_router_workspace_size, L.moe_router_grouped_workspace_size):
        last = 0
        for T in list(range(0, 4200)) + [5000, 8191, 8192, 10000, 12288, 12289, 50000, 2 ** 31 - 1]:
            n = size(T, E)
            assert n >= last, T
            last = n
        assert size(-1, E) == 0 and size(5, 0) == 0 and size(5, 1025) == 0
    for T in (0, 1, 33, 1000, 5000):
        assert L.moe_router_grouped_workspace_size(T, E) >= L.moe_router_workspace_size(T, E)


def test_plain_sizes():
    """256 / lanes tokens a workgroup, 768 of them at most; E <= 32 is added by one workgroup."""
    L = _lib()
    assert L.moe_router_workspace_size(1000, 256) == 17 * 8 + 63 * 513 * 4 == 129412
    assert L.moe_router_workspace_size(1500, 256) == 17 * 8 + 94 * 513 * 4 == 193024
    assert L.moe_router_workspace_size(32, 8) == 0 and L.moe_router_workspace_size(33, 8) == 2 * 8 + 2 * 17 * 4
    assert L.moe_router_grouped_workspace_size(32, 8) == 0
    assert L.moe_router_grouped_workspace_size(1000, 256) == 17 * 8 + 250 * 513 * 4


def test_one_byte_less_is_refused():
    L = _lib()
    f = C.c_void_p(0x1000)
    for T, E in ((1000, 256), (33, 8), (5000, 384)):
        n = L.moe_router_workspace_size(T, E)
        assert L.moe_router(f, 0, T, E, E, 2, None, 0, 0, 1.0, 0.0, f, f, f, None, f, n - 1, None) == 3
        assert f"workspace of {n} bytes".encode() in L.fgb_last_error()
        assert L.moe_router_grouped(f, 0, T, E, E, 2, None, f, 1, 1, 0, 0, 1.0, 0.0, f, f, f, None, f, n - 1, None) == 3
        assert f"workspace of {n} bytes".encode() in L.fgb_last_error()
        assert L.moe_router_grouped(f, 0, T, E, E, 2, None, f, 1, 1, 0, 0, 1.0, 0.0, f, f, f, None, None, 1 << 30, None) == 3
