"""The router and linear-layer oracle against differences, identities and worked
examples, and the refusals of the router and linear calls (no GPU needed)."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from moe_variable_size_amd import _lib, api
from oracle import router_oracle as R


def _diff(f, x, h=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        d[i] = (f(a) - f(b)) / (2 * h)
    return d


def test_worked_routing_example():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0]]))
    ids, w = R.route(l, 2)
    assert ids.tolist() == [[1, 2]] and np.allclose(w, [[4 / 6, 2 / 6]])
    ids, w = R.route(l, 2, renormalize=False, scale=2.0)
    assert np.allclose(w, [[1.0, 0.5]])
    # the bias moves the choice, not the weight; equal values go to the lower expert
    ids, w = R.route(l, 2, bias=[0.5, 0.0, 0.0, 0.5], renormalize=False)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[1 / 8, 1 / 8]])
    # groups {0, 1}, {2, 3}: by the best 1 wins, by the sum of two likewise; one group stays
    assert R.route(l, 1, groups=2, topk_groups=1)[0].tolist() == [[1]]
    assert R.route(np.log([[3.0, 3.0, 4.0, 1.0]]), 1, groups=2, topk_groups=1)[0].tolist() == [[2]]
    assert R.route(np.log([[3.0, 3.0, 4.0, 1.0]]), 1, groups=2, topk_groups=1,
                   group_score="top2")[0].tolist() == [[0]]


def test_barred_experts_and_empty_rows():
    inf = math.inf
    ids, w = R.route(np.array([[-inf, 1.0, -inf], [-inf, -inf, -inf]]), 2)
    assert ids.tolist() == [[1, -1], [-1, -1]] and w.tolist() == [[1.0, 0.0], [0.0, 0.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_is_the_difference_quotient(score, renorm):
    rng = np.random.default_rng(3)
    l, g = rng.standard_normal((3, 7)), rng.standard_normal((3, 3))
    opts = dict(score=score, renormalize=renorm, scale=1.7)
    ids, _ = R.route(l, 3, **opts)
    d = R.route_grad(l, ids, g, **opts)
    num = _diff(lambda x: float((R.route(x, 3, **opts)[1] * g).sum()), l)
    assert np.abs(d - num).max() < 1e-8


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_loss_gradient_is_the_difference_quotient(score):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((5, 6))
    ids = rng.integers(-1, 6, (5, 2)).astype(np.int32)
    gl = (0.7, 0.3)

    def f(x):
        b, z, _, _ = R.router_losses(x, ids, score)
        return gl[0] * b + gl[1] * z

    assert np.abs(R.router_losses_grad(l, ids, gl, score) - _diff(f, l)).max() < 1e-8


def test_even_load_balances_at_one():
    ids = np.arange(8, dtype=np.int32).reshape(4, 2)
    assert abs(R.router_losses(np.zeros((4, 8)), ids)[0] - 1.0) < 1e-12


@pytest.mark.parametrize("kind", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_gradient_is_the_difference_quotient(kind):
    rng = np.random.default_rng(5)
    x, W, b = rng.standard_normal((3, 4)), rng.standard_normal((5, 4)), rng.standard_normal(5)
    dy = rng.standard_normal((3, 5))
    _, z = R.linear(x, W, b, kind)
    dX, dW, db = R.linear_grad(dy, x, W, z, kind)
    assert np.abs(dX - _diff(lambda v: float((R.linear(v, W, b, kind)[0] * dy).sum()), x)).max() < 1e-7
    assert np.abs(dW - _diff(lambda v: float((R.linear(x, v, b, kind)[0] * dy).sum()), W)).max() < 1e-7
    assert np.abs(db - _diff(lambda v: float((R.linear(x, W, v, kind)[0] * dy).sum()), b)).max() < 1e-7


# ---- refusals -----------------------------------------------------------------------------------

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, LIMIT, OPTION = 1, 2, 3, 4, 5, 7, 8
P = ctypes.c_void_p(1 << 20)     # never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 1)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        pytest.skip("library not built (run __graft_entry__.build())")
    return _lib.load()


def _fwd(lib, logits=P, bias=None, T=4, E=8, k=2, score=0, groups=1, keep=1, gs=0, renorm=1,
         scale=1.0, ids=P, w=P, dtype=0):
    return lib.moe_route_fwd(logits, bias, T, E, k, score, groups, keep, gs, renorm, scale, ids, w,
                             dtype, None)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), NULL), (dict(ids=None), NULL), (dict(w=None), NULL),
    (dict(T=-1), SHAPE), (dict(E=0), SHAPE), (dict(k=0), SHAPE), (dict(k=9), SHAPE),
    (dict(E=128, k=65), SHAPE), (dict(E=1025), LIMIT), (dict(T=1 << 30), LIMIT),
    (dict(dtype=2), DTYPE), (dict(score=2), OPTION), (dict(gs=2), OPTION),
    (dict(groups=3), OPTION), (dict(groups=0), OPTION), (dict(groups=2, keep=3), OPTION),
    (dict(groups=4, keep=1, k=3), OPTION), (dict(groups=8, keep=8, gs=1), OPTION),
    (dict(E=130, groups=65, keep=65), OPTION), (dict(scale=0.0), OPTION),
    (dict(scale=math.inf), OPTION), (dict(scale=math.nan), OPTION),
    (dict(logits=ODD), ALIGN), (dict(bias=ODD), ALIGN), (dict(ids=ODD), ALIGN), (dict(w=ODD), ALIGN),
    (dict(logits=ODD, dtype=1), ALIGN),
    (dict(T=0, logits=None, ids=None, w=None), 0),
])
def test_route_forward_refuses(lib, kw, code):
    assert _fwd(lib, **kw) == code


def test_route_backward_refuses(lib):
    def call(g=P, l=P, i=P, w=P, T=4, E=8, k=2, score=0, renorm=1, scale=1.0, d=P, dtype=0):
        return lib.moe_route_bwd(g, l, i, w, T, E, k, score, renorm, scale, d, dtype, None)
    for kw, code in ((dict(g=None), NULL), (dict(l=None), NULL), (dict(i=None), NULL),
                     (dict(w=None), NULL), (dict(d=None), NULL), (dict(k=9), SHAPE),
                     (dict(scale=-1.0), OPTION), (dict(dtype=7), DTYPE), (dict(d=ODD), ALIGN),
                     (dict(score=-1), OPTION), (dict(T=0, g=None, l=None, i=None, w=None, d=None), 0)):
        assert call(**kw) == code, kw


def test_router_loss_refuses(lib):
    n = lib.moe_router_loss_workspace_bytes(100, 8)
    assert n > 0 and n % 256 == 0
    assert lib.moe_router_loss_workspace_bytes(0, 8) == 0
    assert lib.moe_router_loss_workspace_bytes(100, 0) == 0
    assert lib.moe_router_loss_workspace_bytes(100, 1025) == 0

    def call(l=P, i=P, T=100, E=8, k=2, score=0, out=P, stats=P, dtype=0, ws=P, nb=n):
        return lib.moe_router_loss_fwd(l, i, T, E, k, score, out, stats, dtype, ws, nb, None)
    for kw, code in ((dict(l=None), NULL), (dict(i=None), NULL), (dict(out=None), NULL),
                     (dict(stats=None), NULL), (dict(ws=None), WORKSPACE), (dict(nb=n - 1), WORKSPACE),
                     (dict(ws=ODD), ALIGN), (dict(E=1025), LIMIT), (dict(score=3), OPTION),
                     (dict(dtype=2), DTYPE), (dict(k=0), SHAPE), (dict(T=-1), SHAPE)):
        assert call(**kw) == code, kw

    def back(g=P, l=P, stats=P, T=100, E=8, score=0, d=P, dtype=0):
        return lib.moe_router_loss_bwd(g, l, stats, T, E, score, d, dtype, None)
    for kw, code in ((dict(g=None), NULL), (dict(l=None), NULL), (dict(stats=None), NULL),
                     (dict(d=None), NULL), (dict(d=ODD), ALIGN), (dict(E=0), SHAPE),
                     (dict(T=0, g=None, l=None, d=None), 0)):
        assert back(**kw) == code, kw


def test_linear_refuses(lib):
    big = 1 << 40

    def call(x=P, W=P, b=None, r=None, out=P, z=None, M=4, K=8, N=8, act=0, dt=1, odt=1, ws=P, nb=big):
        return lib.moe_linear_fwd(x, W, b, r, out, z, M, K, N, act, dt, odt, ws, nb, None)
    for kw, code in ((dict(x=None), NULL), (dict(W=None), NULL), (dict(out=None), NULL),
                     (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(N=0), SHAPE),
                     (dict(M=1 << 31), LIMIT), (dict(K=(1 << 22) + 1), LIMIT),
                     (dict(N=(1 << 22) + 1), LIMIT), (dict(act=5), OPTION), (dict(act=-1), OPTION),
                     (dict(dt=0, odt=1), DTYPE), (dict(dt=2), DTYPE), (dict(odt=2), DTYPE),
                     (dict(x=ODD), ALIGN), (dict(b=ODD), ALIGN), (dict(r=ODD), ALIGN),
                     (dict(z=ODD), ALIGN), (dict(out=ODD), ALIGN), (dict(M=0, x=None, out=None), 0)):
        assert call(**kw) == code, kw
    need = lib.moe_linear_bwd_workspace_bytes(4, 8, 8, 1, 1, 1)
    assert need > 0
    assert lib.moe_linear_bwd_workspace_bytes(4, 0, 8, 1, 1, 1) == 0
    assert lib.moe_linear_bwd_workspace_bytes(4, 8, 8, 9, 1, 1) == 0

    def back(g=P, x=P, W=P, z=P, dX=P, dW=P, db=P, M=4, K=8, N=8, act=1, dt=1, odt=1, ws=P, nb=big):
        return lib.moe_linear_bwd(g, x, W, z, dX, dW, db, M, K, N, act, dt, odt, ws, nb, None)
    for kw, code in ((dict(g=None), NULL), (dict(x=None), NULL), (dict(W=None), NULL),
                     (dict(z=None), NULL), (dict(ws=None), WORKSPACE), (dict(nb=need - 1), WORKSPACE),
                     (dict(ws=ODD), ALIGN), (dict(dX=ODD), ALIGN), (dict(dW=ODD), ALIGN),
                     (dict(db=ODD), ALIGN), (dict(z=ODD), ALIGN), (dict(act=8), OPTION),
                     (dict(dt=0, odt=1), DTYPE), (dict(N=0), SHAPE)):
        assert back(**kw) == code, kw


def test_binding_refuses_host_tensors_and_unknown_options(lib):
    l = torch.zeros(3, 8)
    with pytest.raises(ValueError):
        api.moe_route_fwd(l, 2)
    with pytest.raises(ValueError):
        api.moe_linear_fwd(l, l)
    with pytest.raises(ValueError):
        api._option(api.MOE_SCORES, "tanh", "score")
    with pytest.raises(ValueError):
        api._option(api.MOE_ACTS, None, "act")
