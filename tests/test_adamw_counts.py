"""Refusals of the AdamW step with a count for every tensor, on the host before any launch (no GPU needed)."""
import ctypes
import os

import pytest

from moe_variable_size_amd import _lib

P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def call():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    lib = _lib.load()

    def run(counts=P, steps=5, count=1, tensors=None, b1=0.9, lr=1e-3, lr_dev=None, scale=None, bits=32, **fields):
        if tensors is None:
            base = dict(param=P.value, grad=P.value, m=P.value, v=P.value, n=8, number=4)
            tensors = (_lib.MoeAdamwTensor * 1)(_lib.MoeAdamwTensor(**{**base, **fields}))
        return lib.moe_adamw_step_counts(tensors, count, lr, lr_dev, b1, 0.99, 1e-8, 0.0, counts, steps, scale, 0, 0, 0, bits, None)

    return run


def test_rejects_before_launch(call):
    assert call(count=0, counts=None) == 0 and call(n=0, number=-3) == 0
    assert call(counts=None) == 1
    assert call(number=5) == 2 and call(number=-1) == 2 and call(steps=4) == 2 and call(steps=-1) == 2 and call(steps=1 << 31) == 2
    assert call(number=1 << 40) == 2
    assert call(counts=ctypes.c_void_p(P.value + 2)) == 4
    # what the step with one number refuses
    assert call(count=-1) == 2 and call(n=-1) == 2 and call(n=(1 << 34) + 1) == 7 and call(param=None) == 1
    assert call(b1=1.0) == 8 and call(lr=float("nan")) == 8 and call(bits=16) == 8 and call(bits=8) == 1
    assert call(master=P.value) == 3 and call(grad=P.value + 1) == 4 and call(scale=ctypes.c_void_p(P.value + 1)) == 4
