"""NULL pointers in the descriptor of 4-bit weights, and in the place of one, are refused by every call that takes it, on the
host before any launch (no GPU needed)."""
import ctypes
import os

import pytest

from moe_variable_size_amd import _lib

P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


@pytest.mark.parametrize("name", ["linear", "fused", "token", "quantize", "dequantize"])
def test_w4_descriptor(lib, name):
    s = _lib.MoeSchedule()
    for field, kind in _lib.MoeSchedule._fields_:
        setattr(s, field, P.value if kind is ctypes.c_void_p else 0)
    s.T, s.S, s.R, s.k, s.E, s.phases = 10, 20, 20, 2, 1, 0
    call = {"linear": lambda w: lib.moe_linear_w4_fwd(P, w, None, None, P, 10, 0, 1, None),
            "fused": lambda w: lib.moe_fused_fwd_w4(P, w, ctypes.byref(s), P, None),
            "token": lambda w: lib.moe_token_fwd_w4(P, w, P, None, 10, 2, P, None),
            "quantize": lambda w: lib.moe_w4_quantize(P, w, 0, None),
            "dequantize": lambda w: lib.moe_w4_dequantize(w, P, 0, None)}[name]
    assert call(None) == 1
    for field in ("codes", "scales"):
        f = dict(codes=P.value, scales=P.value, zeros=None, N=40, K=136, E=1, group=32)
        f[field] = None
        assert call(ctypes.byref(_lib.MoeW4Weight(**f))) == 1, field
