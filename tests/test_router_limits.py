"""Row counts past the limits are refused before anything else is looked at (no GPU needed)."""
import ctypes
import os

import pytest

from moe_variable_size_amd import _lib

LIMIT = 7
P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


@pytest.mark.parametrize("T,k", [(1 << 31, 1), (1 << 30, 2), (1 << 61, 8), (1 << 62, 4), ((1 << 63) - 1, 2)])
def test_rows_times_slots_past_2_31(lib, T, k):
    """Products that wrap around 64 bits among them."""
    assert lib.moe_route_fwd(P, None, T, 8, k, 0, 1, 1, 0, 1, 1.0, P, P, 0, None) == LIMIT
    assert lib.moe_route_bwd(P, P, P, P, T, 8, k, 0, 1, 1.0, P, 0, None) == LIMIT
    assert lib.moe_router_loss_fwd(P, P, T, 8, k, 0, P, P, 0, P, 1 << 40, None) == LIMIT
    if T >= 1 << 31:
        assert lib.moe_router_loss_bwd(P, P, P, T, 8, 0, P, 0, None) == LIMIT
        assert lib.moe_router_loss_workspace_bytes(T, 8) == 0
