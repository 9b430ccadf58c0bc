"""The linear cross entropy's gradients where rows share the factor g of their loss: a mean, a sum, sequences that weigh their
tokens alike.  What g's rounding to the operands' type would do to one row it would do to all of them, in the same direction, and
nothing of it would average out.

In norm a rounding to bf16 is 2^-8 sqrt(1 / 3) at most where many are evenly spread below half a step (see
test_gpu_cross_entropy.py): the outputs' own is one, that of dl (of x, where rows differ in g and dW needs it) another.
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api

pytestmark = pytest.mark.gpu

H32, H16 = 2.0 ** -24, 2.0 ** -8
BF = torch.bfloat16


def make(M, K, V, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((M, K), generator=gen, device="cuda").to(BF)
    W = (torch.randn((V, K), generator=gen, device="cuda") / K ** 0.5).to(BF)
    return x, W, torch.randint(0, V, (M,), generator=gen, device="cuda")


def reference(x, W, t, g, z=0.0):
    """(dX, dW) in 64 bits"""
    x, W = x.double(), W.double()
    l = x @ W.t()
    lse = torch.logsumexp(l, 1)
    ok = (t >= 0) & (t < W.shape[0])
    g = torch.where(ok, g.double(), 0.0)
    d = torch.exp(l - lse[:, None]) * (g * (1 + 2 * z * lse))[:, None]
    d.scatter_add_(1, torch.where(ok, t, 0)[:, None], -g[:, None])
    return d @ W, d.t() @ x


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


LIMIT = H16 * (2 / 3) ** 0.5


@pytest.mark.parametrize("rows,count", [(1020, 1020), (1024, 920), (2040, 2040), (4096, 4080), (513, 513), (700, 509)])
@pytest.mark.parametrize("K,V,z", [(512, 4001, 0.0), (264, 8192, 1e-4), (129, 2003, 0.0)])
def test_means_are_off_by_independent_roundings(rows, count, K, V, z):
    """Counts just below a power of two, where 1 / count is furthest from a number of 8 bits; as a mean, as a sum of that
    weight and as a gradient for each row."""
    x, W, t = make(rows, K, V, rows + K)
    t[:rows - count] = -100
    total = torch.empty(3, device="cuda")
    _, lse = api.moe_linear_ce_fwd(x, W, t, z_weight=z, total=total)
    one = torch.ones(1, device="cuda")
    want = reference(x, W, t, torch.full((rows,), 1.0 / count, device="cuda", dtype=torch.double), z)
    got = api.moe_linear_ce_bwd(one, x, W, t, lse, z_weight=z, reduction="mean", total=total)
    for a, b in zip(got, want):
        assert off(a, b) <= LIMIT
    w = one / count
    for again in (api.moe_linear_ce_bwd(w, x, W, t, lse, z_weight=z, reduction="sum"),
                  api.moe_linear_ce_bwd(w.expand(rows).contiguous(), x, W, t, lse, z_weight=z)):
        for a, b in zip(again, got):
            assert torch.equal(a, b)


def test_sequences_that_weigh_their_tokens_alike():
    lens = (1020, 508, 2036, 250)
    x, W, t = make(sum(lens), 512, 4001, 1)
    g = torch.cat([torch.full((n,), 1.0 / n, device="cuda") for n in lens])
    _, lse = api.moe_linear_ce_fwd(x, W, t)
    for s in (1.0, -1.0, 1e-3):
        for a, b in zip(api.moe_linear_ce_bwd(s * g, x, W, t, lse), reference(x, W, t, s * g)):
            assert off(a, b) <= LIMIT
    # of very different size: the rows' gradients one by one
    g[:1020] *= 1e-6
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse)
    want = reference(x, W, t, g)
    assert float(((dX.double() - want[0]).norm(dim=1) / want[0].norm(dim=1)).max()) <= 1.3 * H16
    assert off(dW, want[1]) <= LIMIT


@pytest.mark.parametrize("K,offset", [(64, 0), (64, 1), (63, 0)])
def test_rows_that_do_not_count(K, offset):
    """Their upstream gradient may be anything; none that counts, weights of 0 and weights that are all 0 give zeros."""
    M, V = 600, 1003
    x, W, t = make(M, K, V, 2)
    if offset:
        x = torch.empty(M * K + offset, dtype=BF, device="cuda")[offset:].view(M, K).copy_(x)
    t[:50], t[550:] = -100, V
    g = torch.linspace(-1, 2, M, device="cuda")
    g[100:120] = 0
    _, lse = api.moe_linear_ce_fwd(x, W, t)
    clean = api.moe_linear_ce_bwd(g, x, W, t, lse)
    for a, b in zip(clean, reference(x, W, t, g)):
        assert off(a, b) <= LIMIT
    assert not clean[0][:50].any() and not clean[0][550:].any() and not clean[0][100:120].any()
    for bad in (float("nan"), float("inf"), 3e38):
        h = g.clone()
        h[:50], h[550:] = bad, -bad
        for a, b in zip(api.moe_linear_ce_bwd(h, x, W, t, lse), clean):
            assert torch.equal(a, b)
    for a in api.moe_linear_ce_bwd(torch.zeros_like(g), x, W, t, lse):
        assert not a.any()
    none, total = torch.full_like(t, -1), torch.empty(3, device="cuda")
    _, lse = api.moe_linear_ce_fwd(x, W, none, total=total)
    for reduction in ("sum", "mean"):
        for a in api.moe_linear_ce_bwd(g[:1], x, W, none, lse, reduction=reduction, total=total):
            assert not a.any()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_gradients_that_are_not_finite_reach_their_rows(reduction):
    M, V = 600, 500
    x, W, t = make(M, 64, V, 3)
    t[7] = -100
    total = torch.empty(3, device="cuda")
    _, lse = api.moe_linear_ce_fwd(x, W, t, total=total)
    for bad in (float("nan"), float("inf")):
        g = torch.full((M if reduction == "none" else 1,), 0.5, device="cuda")
        g[0] = bad
        dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse, reduction=reduction, total=total)
        assert not dX[7].any() and not torch.isfinite(dX[0]).any()
        assert bool(torch.isfinite(dX[1:]).all()) == (reduction == "none")
        assert not torch.isfinite(dW).all()


@pytest.mark.parametrize("M,K,V", [(600, 64, 3001), (600, 65, 3001), (2049, 128, 70001), (1500, 2048, 520), (5000, 16, 100), (640, 5, 40)])
def test_factors_in_every_way_through_the_products(M, K, V):
    """Whole and staged tiles, several pieces, reductions in ranges (with their join), rows of 8 and of less than 16 columns."""
    x, W, t = make(M, K, V, M + V)
    _, lse = api.moe_linear_ce_fwd(x, W, t)
    g = torch.tensor([0.3, 0.7, 1.1], device="cuda").repeat(M // 3 + 1)[:M].contiguous()
    for h in (g, torch.full_like(g, 0.7)):
        want = reference(x, W, t, h)
        for a, b in zip(api.moe_linear_ce_bwd(h, x, W, t, lse), want):
            assert off(a, b) <= LIMIT
        dX, _ = api.moe_linear_ce_bwd(h, x, W, t, lse, dw=False)
        _, dW = api.moe_linear_ce_bwd(h, x, W, t, lse, dx=False)
        assert off(dX, want[0]) <= LIMIT and off(dW, want[1]) <= LIMIT


def test_captured_and_replayed():
    M, K, V = 700, 64, 2001
    x, W, t = make(M, K, V, 4)
    g = torch.rand(M, device="cuda")

    def call():
        _, lse = api.moe_linear_ce_fwd(x, W, t)
        return api.moe_linear_ce_bwd(g, x, W, t, lse)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (5, 6, 7):
        for a, b in zip((x, W, t), make(M, K, V, seed)):
            a.copy_(b)
        g.copy_(torch.rand(M, device="cuda") * 10 ** (seed - 6))
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


def test_mean_of_a_trained_model():
    """Targets' probabilities between 0 and 1: their entries p - 1 differ, and so do their roundings."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    M, K, V = 1020, 512, 2003
    W = torch.randn((V, K), generator=gen, device="cuda") / K ** 0.5
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    x = torch.randn((M, K), generator=gen, device="cuda") + W[t] * torch.linspace(0, 25, M, device="cuda")[:, None]
    x, W = x.to(BF), W.to(BF)
    loss = api.linear_cross_entropy(x.requires_grad_(), W.requires_grad_(), t)
    got = torch.autograd.grad(loss, (x, W))
    p = torch.exp(-api.moe_linear_ce_fwd(x.detach(), W.detach(), t)[0])
    assert float(p.min()) < 0.01 and float(p.max()) > 0.99
    for a, b in zip(got, reference(x.detach(), W.detach(), t, torch.full((M,), 1.0 / M, device="cuda"))):
        assert off(a, b) <= LIMIT
