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


def test_w4_rejects_before_launch(lib):
    def w(**f):
        return ctypes.byref(_lib.MoeW4Weight(**{**dict(codes=P.value, scales=P.value, zeros=None, N=40, K=136, E=1, group=32), **f}))

    s = _lib.MoeSchedule()
    for name, kind in _lib.MoeSchedule._fields_:
        setattr(s, name, P.value if kind is ctypes.c_void_p else 0)
    s.T, s.S, s.R, s.k, s.E, s.phases = 10, 20, 20, 2, 1, 0

    def lin(x=P, ww=None, bias=None, res=None, out=P, M=10, act=0, od=1):
        return lib.moe_linear_w4_fwd(x, ww or w(), bias, res, out, M, act, od, None)

    calls = [lambda ww, **k: lin(ww=ww, **k), lambda ww, **k: lib.moe_fused_fwd_w4(k.get("x", P), ww, ctypes.byref(s), P, None),
             lambda ww, **k: lib.moe_token_fwd_w4(k.get("x", P), ww, P, None, 10, 2, P, None),
             lambda ww, **k: lib.moe_w4_quantize(P, ww, 0, None), lambda ww, **k: lib.moe_w4_dequantize(ww, P, 0, None)]
    for call in calls:
        assert call(w(codes=None)) == 1 and call(w(scales=None)) == 1 and call(None) == 1 or call is calls[0]
        assert call(w(N=0)) == 2 and call(w(K=0)) == 2 and call(w(E=0)) == 2
        assert call(w(group=48)) == 8
        assert call(w(N=(1 << 22) + 1)) == 7 and call(w(K=(1 << 22) + 8)) == 7 and call(w(E=1025)) == 7
        assert call(w(N=1 << 20, K=4096)) == 7  # 2^31 bytes of codes
        assert call(w(codes=P.value + 8)) == 4 and call(w(scales=P.value + 2)) == 4 and call(w(zeros=P.value + 1)) == 4
    for call in calls[:3]:
        assert call(w(K=132)) == 2
        assert call(w(), x=None) == 1 and call(w(), x=ctypes.c_void_p(P.value + 8)) == 4
    assert lin(out=None) == 1 and lin(M=-1) == 2 and lin(M=1 << 23) == 7 and lin(act=5) == 8 and lin(od=2) == 3 and lin(ww=w(E=2)) == 2
    assert lin(bias=ODD) == 4 and lin(res=ODD) == 4 and lin(out=ODD) == 4 and lin(M=0, x=None, out=None) == 0
    assert lib.moe_fused_fwd_w4(P, w(E=2), ctypes.byref(s), P, None) == 2
    assert lib.moe_fused_fwd_w4(P, w(), ctypes.byref(s), None, None) == 1 and lib.moe_fused_fwd_w4(P, w(), None, P, None) == 1
    tok = lib.moe_token_fwd_w4
    assert tok(P, w(), None, None, 10, 2, P, None) == 1 and tok(P, w(), P, None, 10, 2, None, None) == 1
    assert tok(P, w(), P, None, 10, 0, P, None) == 2 and tok(P, w(), P, None, 10, 65, P, None) == 2
    assert tok(P, w(), ODD, None, 10, 2, P, None) == 4 and tok(P, w(), P, ODD, 10, 2, P, None) == 4
    assert tok(None, w(), None, None, 0, 2, None, None) == 0
    assert lib.moe_w4_quantize(None, w(), 0, None) == 1 and lib.moe_w4_quantize(P, w(), 3, None) == 3
    assert lib.moe_w4_dequantize(w(), None, 0, None) == 1 and lib.moe_w4_dequantize(w(), ODD, 1, None) == 4


def test_oracle_w4_places_every_code_once():
    """256 elements: every nibble of their 128 bytes is one of them; a block alone fills its 64 bytes."""
    seen = {O.w4_place(k) for k in range(256)}
    assert seen == {(b, s) for b in range(128) for s in (0, 4)}
    assert {O.w4_place(k)[0] // 64 for k in range(128)} == {0}
    W = np.random.default_rng(1).standard_normal((3, 70))
    for symmetric in (True, False):
        q, s, z = O.w4_quantize(W, 32, symmetric)
        g = np.arange(70) // 32
        assert (abs((q - z[:, g]) * s[:, g] - W) <= s[:, g] * 1.07).all()


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
