"""GPU parity of expert routing and the router losses against the float64 oracle.

Tolerances, in units of u = 2^-24 (half a step of fp32), per element:
  * a score is an exponential of l - m, whose argument carries a rounding of
    |l - m| u and whose evaluation and the following sum (<= 1024 positive terms
    added 16 per lane, then over 64 lanes: 22 additions deep), quotient and
    scaling add at most 40 u: relative error (|l|max-range + 40) u =: R;
  * a gradient is a sum of products of such values: R times the sum of the
    absolute values of its terms, doubled for the dot product's own additions;
  * a bf16 gradient is rounded once more: 2^-8 relative;
  * the oracle's gradient of a renormalised softmax leaves, where the exact value is
    0, what is left of ds - sum(ds s): E <= 1024 = 2^10 roundings of 2^-53 of terms of
    the size of a row's largest, times s <= 1: 2^-43 of that.
Ids have to be equal.
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from oracle import router_oracle as R
from tests.gpu_util import host, log

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
INF = float("inf")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _logits(T, E, dtype, seed, std=2.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((T, E), generator=g) * std).to(DT[dtype])


def _rel(l):
    fin = l[np.isfinite(l)]
    return ((fin.max() - fin.min() if fin.size else 0.0) + 40.0) * U


def _check_route(l, k, what, **opts):
    """Runs l (a host tensor) through the library and compares with the oracle."""
    log(f"route {what} {tuple(l.shape)} {l.dtype} k={k} {opts}")
    T = l.shape[0]
    o = dict(opts)
    if o.get("bias") is not None:
        o["bias"] = torch.from_numpy(o["bias"]).cuda()
    ids0 = torch.full((T, k), 77, dtype=torch.int32, device="cuda")
    w0 = torch.full((T, k), float("nan"), device="cuda")
    ids, w = api.moe_route_fwd(l.cuda(), k, expert_ids=ids0, topk_weights=w0, **o)
    torch.cuda.synchronize()
    lf = l.float().numpy()
    ri, rw = R.route(lf, k, **opts)
    assert np.array_equal(host(ids), ri), what
    got = host(w)
    assert np.array_equal(np.isnan(got), np.isnan(rw)), what
    ok = ~np.isnan(rw)
    # a plain softmax weight below fp32's smallest normal is flushed or rounded coarsely
    tol = _rel(lf) * np.abs(rw) + 2.0 ** -126
    near = np.abs(got - rw)[ok] <= tol[ok]
    assert near.all(), (what, np.max((np.abs(got - rw) / tol)[ok]))
    return ids, w


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (65, 8, 2), (129, 60, 4), (40, 64, 8), (37, 65, 6),
          (33, 128, 8), (70, 160, 6), (21, 257, 13), (18, 512, 64), (9, 1000, 17), (6, 1024, 64)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route(T, E, k, score, dtype):
    l = _logits(T, E, dtype, T * 7 + E)
    bias = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.2
    for renorm in (True, False):
        _check_route(l, k, "plain", score=score, renormalize=renorm, scale=1.0 if renorm else 2.5)
        _check_route(l, k, "bias", score=score, renormalize=renorm, bias=bias)


@pytest.mark.parametrize("T,E,k,groups,keep", [(50, 256, 8, 8, 4), (31, 60, 6, 4, 2), (17, 12, 3, 6, 3),
                                               (23, 128, 4, 64, 5), (12, 1024, 20, 2, 1),
                                               (9, 33, 7, 3, 3), (64, 160, 6, 8, 3), (5, 64, 1, 64, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_groups(T, E, k, groups, keep, score, group_score):
    if group_score == "top2" and E == groups:
        pytest.skip("one expert a group has no two best")
    bias = np.random.default_rng(T).standard_normal(E).astype(np.float32) * 0.1
    for dtype in ("f32", "bf16"):
        l = _logits(T, E, dtype, T + E)
        for b in (None, bias):
            _check_route(l, k, "groups", score=score, groups=groups, topk_groups=keep,
                         group_score=group_score, bias=b)


def test_ties_go_to_the_lower_expert():
    l = torch.zeros((4, 96))
    l[1, 40:] = 1.0
    l[2, ::2] = -0.0
    l[3] = torch.tensor([float(i % 3) for i in range(96)])
    for opts in (dict(), dict(bias=np.zeros(96, np.float32)), dict(score="sigmoid"),
                 dict(groups=4, topk_groups=2), dict(groups=4, topk_groups=2, group_score="top2"),
                 dict(groups=8, topk_groups=3, group_score="top2", bias=np.ones(96, np.float32))):
        _check_route(l, 10, "ties", **opts)


def test_values_next_to_each_other_under_a_bias():
    """Scores that differ by less than fp32 resolves, told apart in 64 bits: steps of
    one in the logit's last place near l = 4 change the sigmoid by 4e-9, under a tenth
    of fp32's step near 1; a bias moves them past each other."""
    base = np.float32(4.0)
    step = np.spacing(base)
    rng = np.random.default_rng(8)
    l = torch.from_numpy((base + step * rng.permuted(np.tile(np.arange(64), (30, 1)), axis=1)).astype(np.float32))
    bias = np.full(64, 0.25, np.float32)
    for score in ("sigmoid", "softmax"):
        _check_route(l, 9, "close", score=score, bias=bias)
        _check_route(l, 9, "close groups", score=score, bias=bias, groups=8, topk_groups=2,
                     group_score="top2")
        _check_route(l, 9, "close groups, no bias", score=score, groups=8, topk_groups=2,
                     group_score="top2")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_barred_experts_empty_rows_and_lowest_values(score, renorm):
    lo = torch.finfo(torch.float32).min
    l = _logits(7, 70, "f32", 5)
    l[0] = -INF                       # nothing to choose
    l[1, 3:] = -INF                   # fewer than k left
    l[2, ::2] = -INF
    l[3] = lo                         # the lowest finite value is a value
    l[4, 10:] = lo
    l[5] = -200.0 - torch.arange(70)  # scores that underflow in fp32
    bias = np.zeros(70, np.float32)
    bias[5] = -np.inf
    o = dict(score=score, renormalize=renorm)
    _check_route(l, 6, "barred", **o)
    _check_route(l[[0, 1, 2, 6]], 6, "barred, groups", groups=7, topk_groups=2, group_score="top2", **o)
    _check_route(l[[0, 1, 2, 6]], 6, "barred, bias", bias=bias, groups=7, topk_groups=6, **o)


def test_nan_and_infinite_logits():
    l = _logits(5, 64, "f32", 6)
    l[0, 17] = float("nan")
    l[1, [3, 50]] = float("nan")
    l[2, 9] = INF
    l[3] = float("nan")
    for k in (1, 2, 6):
        for renorm in (True, False):
            _check_route(l[[0, 1, 3, 4]], k, "nan", renormalize=renorm)
            _check_route(l, k, "nan sigmoid", score="sigmoid", renormalize=renorm)
            # +inf: the softmax of its row is NaN
            ids, w = api.moe_route_fwd(l[2:3].cuda(), k, renormalize=renorm)
            assert int(ids[0, 0]) == 9 and bool(w.isnan().all())


# ---- backward -----------------------------------------------------------------------------------

def _grad_tol(l, terms, dtype, ref):
    t = 2 * _rel(l) * terms + 2.0 ** -126
    return t + 2.0 ** -8 * np.abs(ref) if dtype == "bf16" else t


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_backward(T, E, k, score, renorm):
    for dtype in ("f32", "bf16"):
        l = _logits(T, E, dtype, T + 3 * E)
        if E > 3 and k < E - 2:
            l[0, 1:3] = -INF
        if T > 2:
            l[1] = -INF
        o = dict(score=score, renormalize=renorm, scale=1.5)
        log(f"route bwd {T} {E} {k} {o} {dtype}")
        ids, w = api.moe_route_fwd(l.cuda(), k, **o)
        g = torch.randn((T, k), generator=torch.Generator().manual_seed(9))
        d0 = torch.full((T, E), float("nan"), dtype=DT[dtype], device="cuda")
        d = api.moe_route_bwd(g.cuda(), l.cuda(), ids, w, d_logits=d0, **o)
        torch.cuda.synchronize()
        lf, gi, idn = l.float().numpy(), g.double().numpy(), host(ids)
        live = ~np.all(lf == -np.inf, axis=1)
        ref = np.zeros((T, E))
        ref[live] = R.route_grad(lf[live], idn[live], gi[live], **o)
        # |w_j g_j| and w_j (or p_i) times sum |g w|
        wn = np.abs(host(w)).astype(np.float64)
        terms = np.zeros((T, E))
        gw = (np.abs(gi) * wn).sum(1, keepdims=True)
        for t in range(T):
            on = idn[t] >= 0
            np.add.at(terms[t], idn[t][on], wn[t][on] * (np.abs(gi[t][on]) + gw[t] / 1.5))
            if live[t] and not renorm and score == "softmax":
                terms[t] += R.softmax(lf[t]) * gw[t]
        err = np.abs(host(d) - ref)
        ok = err <= _grad_tol(lf, terms, dtype, ref) + 2.0 ** -43 * terms.max(1, keepdims=True)
        assert ok.all(), (dtype, err.max())


def test_route_backward_repeated_and_foreign_ids():
    """An id a row repeats gets the sum of its slots; ids outside [0, E) count for nothing."""
    l = _logits(3, 10, "f32", 1)
    ids = torch.tensor([[4, 4, 2], [-1, 10, 3], [-5, -1, 1 << 30]], dtype=torch.int32)
    w = torch.tensor([[0.2, 0.3, 0.5]] * 3)
    g = torch.tensor([[1.0, -2.0, 0.5]] * 3)
    d = host(api.moe_route_bwd(g.cuda(), l.cuda(), ids.cuda(), w.cuda()))
    ref = np.zeros((3, 10))
    D = float((w[0] * g[0]).sum())
    for j, e in enumerate((4, 4, 2)):
        ref[0, e] += float(w[0, j]) * (float(g[0, j]) - D)
    ref[1, 3] = 0.5 * (0.5 - 0.25)
    assert np.abs(d - ref).max() <= 16 * U


# ---- losses -------------------------------------------------------------------------------------

def _loss_case(T, E, k, score, dtype, seed):
    l = _logits(T, E, dtype, seed)
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(-1, E, (T, k), generator=g, dtype=torch.int32)
    if T > 4:
        l[2] = -INF
        ids[2] = -1
        if E > 2:
            l[3, : E // 2] = -INF
    return l, ids


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (7, 3, 2), (300, 60, 6), (1025, 128, 8),
                                   (65, 257, 3), (50, 512, 8), (33, 1024, 64), (2100, 8, 2), (700, 1024, 8),
                                   (4500, 600, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_losses(T, E, k, score, dtype):
    log(f"losses {T} {E} {k} {score} {dtype}")
    l, ids = _loss_case(T, E, k, score, dtype, T + E)
    losses, stats = api.moe_router_loss_fwd(l.cuda(), ids.cuda(), score=score)
    gl = torch.tensor([0.7, 0.2])
    d0 = torch.full((T, E), float("nan"), dtype=DT[dtype], device="cuda")
    d = api.moe_router_loss_bwd(gl.cuda(), l.cuda(), stats, score=score, d_logits=d0)
    torch.cuda.synchronize()
    lf, idn = l.float().numpy(), ids.numpy()
    b, z, f, inv = R.router_losses(lf, idn, score)
    # per-lane sums of <= T / 4 probabilities over the blocks, joined in 64 bits
    rel = _rel(lf) + (T / 4.0 + 8) * U
    got = host(losses)
    assert abs(got[0] - b) <= rel * abs(b) and abs(got[1] - z) <= 2 * rel * abs(z) + 1e-30
    st = host(stats)
    assert np.allclose(st[:E], f, rtol=4 * U, atol=0) and abs(st[E] - inv) <= 2 * U * inv
    ref = R.router_losses_grad(lf, idn, gl.double().numpy(), score)
    terms = np.zeros((T, E))
    for t in range(T):
        if np.all(lf[t] == -np.inf):
            continue
        p = R.softmax(lf[t])
        s = p if score == "softmax" else R._sigmoid(lf[t])
        q = s / s.sum()
        m = lf[t].max()
        lse = m + np.log(np.exp(lf[t].astype(np.float64) - m).sum())
        terms[t] = inv * (0.7 * q * (f + (f * q).sum()) + 0.4 * (abs(lse) + 1) * p)
    err = np.abs(host(d) - ref)
    ok = err <= _grad_tol(lf, terms, dtype, ref)
    assert ok.all(), (err.max(), np.max(err / (terms + 1e-30)))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_losses_of_nothing(score):
    """No rows at all, or none with a usable logit: both losses and the gradient are 0."""
    l0 = torch.empty((0, 12), device="cuda")
    i0 = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    losses, stats = api.moe_router_loss_fwd(l0, i0, score=score)
    assert host(losses).tolist() == [0.0, 0.0] and not host(stats).any()
    l = torch.full((5, 12), -INF, device="cuda")
    i = torch.full((5, 2), -1, dtype=torch.int32, device="cuda")
    losses, stats = api.moe_router_loss_fwd(l, i, score=score)
    assert host(losses).tolist() == [0.0, 0.0] and not host(stats).any()
    d = api.moe_router_loss_bwd(torch.ones(2, device="cuda"), l, stats, score=score)
    assert not host(d).any()
    ids, w = api.moe_route_fwd(l0, 3)
    assert ids.shape == (0, 3) and w.shape == (0, 3)


# ---- together -----------------------------------------------------------------------------------

def _sublayer(x, Wr, br, W, Ws, bias):
    """Router logits -> routing -> routed experts, plus a shared expert, and the losses."""
    logits = api.linear(x, Wr, br, out_dtype=torch.float32)
    ids, w = api.route(logits, 2, score="sigmoid", bias=bias, scale=1.5)
    y = api.moe(x, W, ids, w)
    y = api.linear(x, Ws, None, act="silu", residual=y, out_dtype=torch.float32)
    return y, api.router_loss(logits, ids, score="sigmoid"), ids


def test_sublayer_and_its_gradients():
    """The set as a layer uses it, every gradient against float64 autograd of the same
    formulas on the CPU with the ids the library chose.  x, the weights and their
    gradients are bf16: dy (rounded on its way into the products), dz and each gradient
    are rounded once, 2^-8 each, against sums of like size: 3e-2 of the largest element
    and 1e-2 in norm."""
    T, K, N, E = 260, 128, 96, 12
    g = torch.Generator().manual_seed(12)

    def r(*s, std=1.0):
        return (torch.randn(s, generator=g) * std).bfloat16()

    x, Wr, br = r(T, K), r(E, K, std=K ** -0.5), r(E, std=0.1)
    W, Ws = r(E, N, K, std=K ** -0.5), r(N, K, std=K ** -0.5)
    bias = (torch.randn(E, generator=g) * 0.1).float()
    dY, gl = torch.randn((T, N), generator=g), torch.tensor([3.0, 0.5])
    leaves = [t.cuda().requires_grad_() for t in (x, Wr, br, W, Ws)]
    y, losses, ids = _sublayer(*leaves, bias.cuda())
    ((y * dY.cuda()).sum() + (losses * gl.cuda()).sum()).backward()
    torch.cuda.synchronize()

    ref = [t.double().requires_grad_() for t in (x, Wr, br, W, Ws)]
    xd, Wrd, brd, Wd, Wsd = ref
    l = xd @ Wrd.t() + brd
    s = torch.sigmoid(l)
    idl = ids.cpu().long()
    w = s.gather(1, idl)
    w = 1.5 * w / w.sum(1, keepdim=True)
    z = xd @ Wsd.t()
    yd = z * torch.sigmoid(z)
    for j in range(2):
        yd = yd + w[:, j:j + 1] * torch.matmul(Wd[idl[:, j]], xd.unsqueeze(2)).squeeze(2)
    f = torch.bincount(idl.flatten(), minlength=E).double() * E / idl.numel()
    q = s / s.sum(1, keepdim=True)
    ld = torch.stack([(f * q.mean(0)).sum(), torch.logsumexp(l, 1).pow(2).mean()])
    ((yd * dY.double()).sum() + (ld * gl.double()).sum()).backward()
    assert np.allclose(host(losses.detach()), ld.detach().numpy(), rtol=1e-5)
    want = torch.topk((s + bias.double()).detach(), 2, dim=1).indices
    assert torch.equal(torch.sort(want, 1)[0], torch.sort(idl, 1)[0])
    err = (y.detach().cpu().double() - yd.detach()).abs().max() / yd.detach().abs().max()
    assert err < 1e-2
    for name, a, b in zip(("x", "Wr", "br", "W", "Ws"), leaves, ref):
        d = a.grad.cpu().double() - b.grad
        log(f"sublayer grad {name}: max {float(d.abs().max() / b.grad.abs().max()):.2e} "
            f"norm {float(d.norm() / b.grad.norm()):.2e}")
        assert d.abs().max() <= 3e-2 * b.grad.abs().max() and d.norm() <= 1e-2 * b.grad.norm(), name


def test_padded_batch_reaches_no_expert():
    """Rows of -inf logits (padding) come out of the routed layer as zeros and give
    nothing to any gradient."""
    T, K, N, E = 64, 64, 64, 8
    g = torch.Generator().manual_seed(3)
    x = torch.randn((T, K), generator=g).bfloat16().cuda().requires_grad_()
    W = (torch.randn((E, N, K), generator=g) * K ** -0.5).bfloat16().cuda().requires_grad_()
    l = torch.randn((T, E), generator=g)
    l[40:] = -INF
    logits = l.cuda().requires_grad_()
    ids, w = api.route(logits, 2)
    y = api.moe(x, W, ids, w)
    (y.sum() + api.router_loss(logits, ids).sum()).backward()
    assert bool((ids[40:] == -1).all()) and not host(y.detach()[40:]).any()
    assert not host(x.grad[40:]).any() and not host(logits.grad[40:]).any()
    sched = api.moe_build_schedule(ids, w.detach(), E)
    assert int(sched.status[0]) == 24 * 2 and int(sched.counts.sum()) == 80


def test_side_stream_and_two_calls_at_once():
    l = [_logits(3000, 128, "f32", s).cuda() for s in (1, 2)]
    want = [api.moe_route_fwd(v, 8) for v in l]
    wl = [api.moe_router_loss_fwd(v, i)[0] for v, (i, _) in zip(l, want)]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for v, s in zip(l, st):
        s.wait_stream(torch.cuda.current_stream())
        ids, w = api.moe_route_fwd(v, 8, stream=s)
        got.append((ids, w, api.moe_router_loss_fwd(v, ids, stream=s)[0]))
    torch.cuda.synchronize()
    for (i, w), (gi, gw, gl), ll in zip(want, got, wl):
        assert torch.equal(i, gi) and torch.equal(w, gw) and torch.equal(gl, ll)


def test_graph_replays_match_eager():
    """Routing, losses and both backwards captured once and replayed over changing
    logits, with eager work in between."""
    T, E, k = 700, 96, 6
    l = _logits(T, E, "f32", 1).cuda()
    g = torch.randn((T, k), generator=torch.Generator().manual_seed(2)).cuda()
    gl = torch.tensor([1.0, 0.1], device="cuda")

    def step(v):
        ids, w = api.moe_route_fwd(v, k, score="sigmoid", groups=8, topk_groups=3, group_score="top2")
        losses, stats = api.moe_router_loss_fwd(v, ids)
        return (ids, w, losses, api.moe_route_bwd(g, v, ids, w, score="sigmoid"),
                api.moe_router_loss_bwd(gl, v, stats))

    step(l)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(l)
    for seed in (3, 4, 5, 6):
        l.copy_(_logits(T, E, "f32", seed))
        want = step(l)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,E,k", [(20, 64, 64), (11, 100, 40), (33, 200, 17), (6, 513, 16), (40, 17, 16),
                                   (9, 256, 16), (5, 300, 32), (7, 300, 33)])
def test_route_many_slots(T, E, k):
    """More slots than the lanes that share a row, as many, and every expert chosen."""
    l = _logits(T, E, "f32", T + k)
    bias = np.random.default_rng(k).standard_normal(E).astype(np.float32) * 0.2
    for score in ("softmax", "sigmoid"):
        _check_route(l, k, "many", score=score)
        _check_route(l, k, "many, bias", score=score, bias=bias)


def test_bias_of_nan_and_infinity():
    l = _logits(9, 48, "f32", 2)
    bias = np.zeros(48, np.float32)
    bias[[3, 30]] = np.nan
    bias[7] = np.inf
    bias[[0, 1, 47]] = -np.inf
    for o in (dict(), dict(score="sigmoid"), dict(groups=6, topk_groups=3, group_score="top2"),
              dict(score="sigmoid", groups=4, topk_groups=2)):
        _check_route(l, 5, "bias", bias=bias, **o)


@pytest.mark.parametrize("seed", range(12))
def test_route_sweep(seed):
    rng = np.random.default_rng(1000 + seed)
    E = int(rng.integers(2, 600))
    groups = int(rng.choice([1, 1, 2, 3, 4, 8, 16]))
    E = max(2, E // groups) * groups
    keep = int(rng.integers(1, groups + 1))
    k = int(rng.integers(1, min(64, keep * (E // groups)) + 1))
    T = int(rng.integers(1, 90))
    l = _logits(T, E, ["f32", "bf16"][seed % 2], seed, std=float(rng.choice([0.01, 1.0, 8.0])))
    l[torch.from_numpy(rng.random((T, E)) < rng.choice([0.0, 0.3, 0.95]))] = -INF
    bias = rng.standard_normal(E).astype(np.float32) * 0.1 if rng.random() < 0.6 else None
    _check_route(l, k, f"sweep {seed}", score=str(rng.choice(["softmax", "sigmoid"])), bias=bias, groups=groups,
                 topk_groups=keep, group_score=str(rng.choice(["max", "top2"])),
                 renormalize=bool(rng.integers(2)), scale=float(rng.choice([1.0, 2.5])))


def test_rows_past_two_gigabytes():
    """Logits of more than 2^32 bytes: the last rows are routed, and their gradients and
    losses formed, from their own place."""
    T, E, k = (1 << 22) + 5, 260, 3
    l = torch.zeros((T, E), device="cuda")
    assert l.numel() * 4 > 1 << 32
    tail = _logits(7, E, "f32", 4)
    l[-7:] = tail.cuda()
    ids, w = api.moe_route_fwd(l, k)
    ri, rw = R.route(tail.numpy(), k)
    assert np.array_equal(host(ids[-7:]), ri) and np.abs(host(w[-7:]) - rw).max() <= _rel(tail.numpy())
    assert host(ids[:3]).tolist() == [[0, 1, 2]] * 3
    g = torch.zeros((T, k), device="cuda")
    g[-7:] = torch.randn((7, k), generator=torch.Generator().manual_seed(1)).cuda()
    d = api.moe_route_bwd(g, l, ids, w)
    ref = R.route_grad(tail.numpy(), ri, host(g[-7:]).astype(np.float64))
    assert np.abs(host(d[-7:]) - ref).max() <= 4 * _rel(tail.numpy()) * np.abs(host(g[-7:])).max()
    losses, stats = api.moe_router_loss_fwd(l, ids)
    api.moe_router_loss_bwd(torch.tensor([0.0, 1.0], device="cuda") * T, l, stats, d_logits=d)
    p = np.stack([R.softmax(r) for r in tail.numpy()])
    m = tail.numpy().astype(np.float64).max(1, keepdims=True)
    lse = m + np.log(np.exp(tail.numpy() - m).sum(1, keepdims=True))
    assert np.abs(host(d[-7:]) - 2 * lse * p).max() <= 4 * _rel(tail.numpy()) * np.abs(2 * lse * p).max()


def test_captured_forward_and_backward_of_the_sublayer():
    """The differentiable calls captured with torch.autograd.grad, replayed over new
    inputs, against the eager pass."""
    T, K, N, E = 96, 64, 72, 8
    g = torch.Generator().manual_seed(5)

    def r(*s, std=1.0):
        return (torch.randn(s, generator=g) * std).bfloat16().cuda()

    x = r(T, K)
    p = [r(E, K, std=K ** -0.5), r(E, std=0.1), r(E, N, K, std=K ** -0.5), r(N, K, std=K ** -0.5)]
    p = [t.requires_grad_() for t in p]
    bias = (torch.randn(E, generator=g) * 0.1).cuda()

    def step():
        y, losses, ids = _sublayer(x, *p, bias)
        return (y.detach(), losses.detach()) + torch.autograd.grad(y.square().sum() + losses.sum(), p)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (6, 7, 8):
        x.copy_(torch.randn((T, K), generator=torch.Generator().manual_seed(seed)).bfloat16())
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            # two atomic additions per output commute; sums of the losses are ordered
            assert torch.allclose(a.float(), b.float(), rtol=2 ** -7, atol=1e-6)


def test_refusals_of_the_router_binding():
    l = torch.zeros((4, 8), device="cuda")
    ids, w = api.moe_route_fwd(l, 2)
    for kw in (dict(score="tanh"), dict(group_score="sum"), dict(bias=torch.zeros(7, device="cuda")),
               dict(bias=torch.zeros(8)), dict(expert_ids=torch.zeros((4, 3), dtype=torch.int32, device="cuda")),
               dict(topk_weights=torch.zeros((3, 2), device="cuda"))):
        with pytest.raises(ValueError):
            api.moe_route_fwd(l, 2, **kw)
    for bad in (l.double(), l.half()):
        with pytest.raises(TypeError):
            api.moe_route_fwd(bad, 2)
    with pytest.raises(ValueError):
        api.moe_route_fwd(l.t(), 2)
    for kw in (dict(groups=3), dict(groups=2, topk_groups=3), dict(scale=0.0)):
        with pytest.raises(api._lib.MoeError):
            api.moe_route_fwd(l, 2, **kw)
    with pytest.raises(api._lib.MoeError):
        api.moe_route_fwd(l, 9)
    with pytest.raises(ValueError):
        api.moe_route_bwd(w[:3], l, ids, w)
    with pytest.raises(TypeError):
        api.moe_route_bwd(w.bfloat16(), l, ids, w)
    with pytest.raises(TypeError):
        api.moe_router_loss_fwd(l, ids.long())
    with pytest.raises(ValueError):
        api.moe_router_loss_fwd(l, ids[:3])
    losses, stats = api.moe_router_loss_fwd(l, ids)
    with pytest.raises(ValueError):
        api.moe_router_loss_bwd(losses, l, stats[:8])


def _off(t):
    """The same values in a dense view that begins one element into its storage."""
    s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = s[1:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_rows_off_their_lines(dtype):
    """Logits, bias, outputs and gradients that begin between lines of four elements."""
    T, E, k = 50, 64, 6
    l = _logits(T, E, dtype, 3)
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.1)
    lc, bc = l.cuda(), bias.cuda()
    ids, w = api.moe_route_fwd(lc, k, bias=bc, groups=4, topk_groups=2, group_score="top2")
    ids2, w2 = api.moe_route_fwd(_off(lc), k, bias=_off(bc), groups=4, topk_groups=2, group_score="top2",
                                 expert_ids=_off(ids), topk_weights=_off(w))
    assert torch.equal(ids, ids2) and torch.equal(w, w2)
    g = torch.randn((T, k), device="cuda")
    for renorm in (True, False):
        d = api.moe_route_bwd(g, lc, ids, w, renormalize=renorm)
        assert torch.equal(d, api.moe_route_bwd(_off(g), _off(lc), ids2, w2, renormalize=renorm, d_logits=_off(d)))
    losses, stats = api.moe_router_loss_fwd(lc, ids)
    l2, s2 = api.moe_router_loss_fwd(_off(lc), ids2)
    assert torch.equal(losses, l2) and torch.equal(stats, s2)
    d = api.moe_router_loss_bwd(losses, lc, stats)
    assert torch.equal(d, api.moe_router_loss_bwd(losses, _off(lc), stats, d_logits=_off(d)))
