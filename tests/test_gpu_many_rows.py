"""Calls of more rows than one launch can hold (2^32 work-items): routing, its gradient and the linear
layer's products run them as several launches, and every row gets its own result."""
import pytest
import torch

from moe_variable_size_amd import api
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16 = torch.bfloat16
RUN = 1 << 25  # rows of a routing launch


def test_routing_of_2_28_rows():
    T, E = (1 << 28) + 3, 8
    log(f"route T={T}")
    edge = torch.tensor([0, 1, RUN - 1, RUN, RUN + 1, 5 * RUN - 1, 5 * RUN, T - 4, T - 3, T - 2, T - 1], device="cuda")
    l = torch.zeros((T, E), dtype=BF16, device="cuda")
    best = (torch.arange(edge.numel(), device="cuda") * 5 + 3) % E
    l[edge, best] = 2.0
    ids = torch.full((T, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, 1), float("nan"), device="cuda")
    api.moe_route_fwd(l, 1, renormalize=False, expert_ids=ids, topk_weights=w)
    torch.cuda.synchronize()
    assert torch.equal(ids[edge, 0].long(), best)
    e2 = torch.tensor(2.0, dtype=torch.float64).exp()
    p = float(e2 / (e2 + 7))
    # a plain weight: an exponential and a sum of 8, 40 u and 2 u of the argument's rounding
    assert float((w[edge, 0].double() - p).abs().max()) <= 42 * U * p
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[edge] = False
    assert not bool(ids[rest].any())
    assert float((w[rest] - 0.125).abs().max()) <= 40 * U * 0.125
    log("route bwd")
    g = torch.zeros((T, 1), device="cuda")
    g[edge] = 1.0
    d = torch.full((T, E), float("nan"), dtype=BF16, device="cuda")
    api.moe_route_bwd(g, l, ids, w, renormalize=False, d_logits=d)
    torch.cuda.synchronize()
    assert not bool(d[rest].any())
    q = (1 - p) / 7
    ref = torch.full((edge.numel(), E), -p * q, dtype=torch.float64, device="cuda")
    ref[torch.arange(edge.numel(), device="cuda"), best] = p * (1 - p)
    err = (d[edge].double() - ref).abs()
    assert bool((err <= 200 * U * p + 2.0 ** -8 * ref.abs()).all())


def test_streamed_product_of_2_26_rows():
    M, K, N = (1 << 26) + 5, 8, 8
    log(f"linear M={M} streamed")
    x = torch.empty((M, K), device="cuda", dtype=BF16).normal_()
    W = torch.eye(N, K, device="cuda", dtype=BF16) * 2   # out = 2 x, exactly
    o = torch.full((M, N), float("nan"), device="cuda", dtype=BF16)
    api.moe_linear_fwd(x, W, out=o)
    torch.cuda.synchronize()
    assert torch.equal(o, x * 2)
    o.fill_(float("nan"))
    api.moe_linear_fwd(x, W, act="relu", residual=x, out=o)
    torch.cuda.synchronize()
    for r in range(0, M, 1 << 24):
        v = x[r:r + (1 << 24)].float()
        assert torch.equal(o[r:r + (1 << 24)], (torch.relu(v * 2) + v).bfloat16())


def test_staged_products_of_2_30_rows():
    M = (1 << 30) + 7
    log(f"linear M={M} fp32")
    x = torch.empty((M, 1), device="cuda").normal_()
    W = torch.full((1, 1), 1.5, device="cuda")
    want = x * 1.5
    o = torch.full((M, 1), float("nan"), device="cuda")
    api.moe_linear_fwd(x, W, out=o)
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    del o
    log("dX")
    dX, dW, db = api.moe_linear_bwd(x, x, W, dw=False, dbias=False)
    torch.cuda.synchronize()
    assert dW is None and db is None and torch.equal(dX, want)
