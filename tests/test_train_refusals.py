"""Refusals of the optimizer's step, the linear cross entropy and the 4-bit products, on the host before any
launch (no GPU needed), and pins of their oracle."""
import ctypes
import os

import numpy as np
import pytest
import torch

from moe_variable_size_amd import _lib
from oracle import train_oracle as O

P = ctypes.c_void_p(1 << 20)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def adamw(lib, tensors=None, count=None, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1, step_dev=None,
          scale=None, pd=0, gd=0, bits=32, **fields):
    if tensors is None:
        base = dict(param=P.value, grad=P.value, m=P.value, v=P.value, n=8)
        tensors = (_lib.MoeAdamwTensor * 1)(_lib.MoeAdamwTensor(**{**base, **fields}))
        count = 1 if count is None else count
    return lib.moe_adamw_step(tensors, count, lr, None, b1, b2, eps, wd, step, step_dev, scale, 0, pd, gd, bits, None)


def test_adamw_rejects_before_launch(lib):
    assert adamw(lib, count=0) == 0                       # nothing to do
    assert adamw(lib, n=0, param=None) == 0
    assert adamw(lib, count=-1) == 2
    assert adamw(lib, n=-1) == 2
    assert adamw(lib, n=(1 << 34) + 1) == 7
    for name in ("param", "grad", "m", "v"):
        assert adamw(lib, **{name: None}) == 1
    assert adamw(lib, bits=8) == 1                        # no scales
    assert adamw(lib, pd=2) == 3 and adamw(lib, gd=7) == 3
    assert adamw(lib, master=P.value) == 3                # of fp32 parameters
    assert adamw(lib, bits=16) == 8
    for bad in (dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=float("nan")), dict(eps=-1.0), dict(eps=float("inf")),
                dict(lr=float("nan")), dict(wd=float("inf")), dict(step=0), dict(step=1 << 31)):
        assert adamw(lib, **bad) == 8, bad
    for name in ("param", "grad", "m", "v"):
        assert adamw(lib, **{name: ODD.value}) == 4
    assert adamw(lib, scale=ODD) == 4 and adamw(lib, step_dev=ODD) == 4
    assert adamw(lib, bits=8, m_scale=ODD.value, v_scale=P.value) == 4
    assert lib.moe_adamw_step(None, 1, 1e-3, None, 0.9, 0.99, 1e-8, 0.0, 1, None, None, 0, 0, 0, 32, None) == 1


def test_linear_ce_rejects_before_launch(lib):
    def fwd(x=P, W=P, t=P, bits=32, M=10, K=8, V=20, z=0.0, loss=P, lse=P, total=None, dt=1, ws=P, nb=1 << 40):
        return lib.moe_linear_ce_fwd(x, W, t, bits, M, K, V, z, loss, lse, total, dt, ws, nb, None)

    def bwd(g=P, red=0, total=None, x=P, W=P, t=P, bits=64, lse=P, M=10, K=8, V=20, z=0.0, dX=P, dW=P, dt=0, ws=P, nb=1 << 40):
        return lib.moe_linear_ce_bwd(g, red, total, x, W, t, bits, lse, M, K, V, z, dX, dW, dt, ws, nb, None)

    for call in (fwd, bwd):
        for name in ("x", "W", "t", "lse"):
            assert call(**{name: None}) == 1
            assert call(**{name: ODD}) == 4
        assert call(K=0) == 2 and call(V=0) == 2 and call(M=-1) == 2
        assert call(M=(1 << 24) + 1) == 7 and call(K=(1 << 22) + 1) == 7 and call(V=(1 << 22) + 1) == 7
        assert call(dt=2) == 3 and call(bits=16) == 3
        assert call(z=float("inf")) == 8
        assert call(ws=None) == 5 and call(nb=8) == 5 and call(ws=ODD) == 4
    assert fwd(loss=None) == 1 and fwd(total=ODD) == 4
    assert bwd(g=None) == 1 and bwd(red=3) == 8 and bwd(red=2) == 1 and bwd(dX=ODD) == 4 and bwd(dW=ODD) == 4
    assert bwd(dX=None, dW=None) == 0 and fwd(M=0, x=None, W=None, t=None) == 0
    for q in (lib.moe_linear_ce_fwd_workspace_bytes, lib.moe_linear_ce_bwd_workspace_bytes):
        assert q(10, 0, 20, 1) == 0 and q(10, 8, 20, 3) == 0 and q(0, 8, 20, 1) == 0
        assert q(10, 8, 20, 1) > 0 and q(10, 8, 20, 1) % 256 == 0
    # no logits: 8192 x 65536 of them would be a GiB in bf16
    assert lib.moe_linear_ce_fwd_workspace_bytes(8192, 4096, 65536, 1) < 1 << 27
    assert lib.moe_linear_ce_bwd_workspace_bytes(8192, 4096, 65536, 1) < 1 << 29


def test_oracle_linear_ce_against_differences_and_torch():
    rng = np.random.default_rng(0)
    x, W = rng.standard_normal((7, 5)), rng.standard_normal((11, 5))
    t, g = np.array([0, 10, -1, 11, 3, 4, 5]), rng.standard_normal(7)
    loss, lse, total = O.linear_ce(x, W, t, 0.01)
    assert loss[2] == loss[3] == 0 and total[1] == 5
    want = torch.nn.functional.cross_entropy(torch.from_numpy(x @ W.T), torch.from_numpy(np.where(t < 11, t, -1)),
                                             ignore_index=-1, reduction="none").numpy()
    assert np.allclose(loss, want + np.where((t >= 0) & (t < 11), 0.01 * lse ** 2, 0), rtol=1e-12)
    dX, dW, _ = O.linear_ce_bwd(g, x, W, t, 0.01)
    u, v, h = rng.standard_normal(x.shape), rng.standard_normal(W.shape), 1e-5

    def f(s):
        return (g * O.linear_ce(x + s * h * u, W + s * h * v, t, 0.01)[0]).sum()

    assert abs((f(1) - f(-1)) / (2 * h) - (dX * u).sum() - (dW * v).sum()) < 1e-8


def test_oracle_e4m3_is_the_format():
    c = torch.arange(256, dtype=torch.uint8)
    want = c.view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(O.e4m3(c.numpy()), want, equal_nan=True)


def test_oracle_adamw_is_torch_s():
    gen = torch.Generator().manual_seed(0)
    p = torch.randn(50, generator=gen, dtype=torch.float64).requires_grad_()
    opt = torch.optim.AdamW([p], lr=1e-2, betas=(0.9, 0.98), eps=1e-8, weight_decay=0.1)
    w, m, v = p.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        p.grad = torch.randn(50, generator=gen, dtype=torch.float64)
        w, m, v = O.adamw(w, p.grad.numpy(), m, v, t, 1e-2, (0.9, 0.98), 1e-8, 0.1)
        opt.step()
        assert np.allclose(p.detach().numpy(), w, rtol=1e-12, atol=0)


def test_rounding_numbers_are_even_and_apart():
    """The hash's halves: even over 256 bins, without correlation between neighbours, halves, steps and tensors."""
    n = 1 << 16
    a = O.dither(np.arange(n), 0, 0, 1)
    others = [O.dither(np.arange(n), 1, 0, 1), O.dither(np.arange(n), 0, 1, 1), O.dither(np.arange(n), 0, 0, 2)]
    for u in (a[0], a[1]):
        bins = np.bincount((u * 256).astype(int), minlength=256)
        assert ((bins - n / 256) ** 2 / (n / 256)).sum() < 255 + 6 * np.sqrt(2 * 255)
        for lag in (1, 2, 8, 256, 2048):
            assert abs(np.corrcoef(u[lag:], u[:-lag])[0, 1]) < 6 / np.sqrt(n)
    pairs = [(a[0], a[1])] + [(a[i], o[i]) for o in others for i in (0, 1)]
    for x, y in pairs:
        assert abs(np.corrcoef(x, y)[0, 1]) < 6 / np.sqrt(n)
