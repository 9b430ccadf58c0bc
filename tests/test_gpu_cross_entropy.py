"""Linear cross entropy on the GPU against a plain computation in 64 bits.

x holds small whole numbers and W multiples of 2^-6, so that every logit is exact in fp32 and what is
off comes from the exponentials, the sums and the roundings, counted in half steps (2^-24 in fp32, 2^-8 in
bf16):
  lse   an exponential of d is off by 2 |d| (its argument's product and constant) and 2, and a sum by one
        per addition, at most 80 in a tile and one for each of the parts (columns / 64 at most), then the
        logarithm and the sum with the largest: 3 |lse|
  loss  those of lse times 1 + 2 |z lse|, and 3 of each of its terms
  dl    p by lse's and its own, then one rounding to the type
  dX    (dW) dl's over sum |dl| |W|, V (M) additions in fp32, and one rounding of its own
In norm a rounding to bf16 is 2^-8 sqrt(1 / 3) at most where many are evenly spread below half a step.  The
output's are; of dl's, the target's carries most of a row's gradient, (1 - p) g against p of the others, so
there are only as many as rows.  The square of one, over 2^-16, is 1 / 3 in the mean and off by sqrt(4 / 45) =
0.3, the mean of M by 0.3 / sqrt M: six times that is allowed, and never more than 1 (see norm_limit).
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import _lib, api
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

H32, H16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def norm_limit(rows):
    return H16 * (min(1.0, 1 / 3 + 1.8 / max(1, rows) ** 0.5) + 1 / 3) ** 0.5


def make(M, K, V, dtype, seed=0, ignore=0.2, wide=True, spread=2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randint(-spread, spread + 1, (M, K), generator=gen, device="cuda").to(dtype)
    # about unit variance of the logits
    step = max(2.0 ** -6, 2.0 ** round(np.log2(0.5 / K ** 0.5 / spread)))
    W = (torch.randint(-2, 3, (V, K), generator=gen, device="cuda").float() * step).to(dtype)
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t = torch.where(torch.rand(M, generator=gen, device="cuda") < ignore, torch.full_like(t, -100), t)
    g = torch.randn(M, generator=gen, device="cuda")
    return x, W, t if wide else t.int(), g


def reference(x, W, t, z, g=None):
    """(loss, lse, E |d|) and with g (dX, dW, |dl| |W|, |dl| |x|), in 64 bits."""
    x, W, t = x.double(), W.double(), t.long()
    l = x @ W.t()
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    ok = (t >= 0) & (t < W.shape[0])
    at = torch.where(ok, t, 0)[:, None]
    lt = l.gather(1, at)[:, 0]
    loss = torch.where(ok, lse - lt + z * lse ** 2, 0.0)
    far = (p * (l.amax(1, keepdim=True) - l)).sum(1)
    if g is None:
        return loss, lse, far, lt
    gg = torch.where(ok, g.double(), 0.0)
    d = p * (gg * (1 + 2 * z * lse))[:, None]
    d.scatter_add_(1, at, -gg[:, None])
    size = (p * (gg * (1 + 2 * z * lse)).abs()[:, None]).scatter_add_(1, at, gg.abs()[:, None])
    return loss, lse, far, lt, d @ W, d.t() @ x, d.abs() @ W.abs(), d.abs().t() @ x.abs(), size @ W.abs(), size.t() @ x.abs()


def check(x, W, t, g, z=0.0, grad=True, **k):
    M, V, half = x.shape[0], W.shape[0], H16 if x.dtype == BF else H32
    loss, lse = api.moe_linear_ce_fwd(x, W, t, z_weight=z)
    r = reference(x, W, t, z, g if grad else None)
    tol = H32 * (2 * r[2] + 80 + V / 64 + 3 * r[1].abs())
    assert ((lse - r[1]).abs() <= tol).all(), (lse - r[1]).abs().max()
    tl = tol * (1 + (2 * z * r[1]).abs()) + 3 * H32 * (r[1].abs() + r[3].abs() + z * r[1] ** 2)
    assert ((loss - r[0]).abs() <= tl).all(), (loss - r[0]).abs().max()
    if not grad:
        return
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse, z_weight=z)
    # p is off by lse's error, its exponential's and, in its scale, z's
    dp = float(tol.max()) + H32 * (2 * float(r[2].max() + 40) + 8)
    for name, got, want, room, size, n in (("dX", dX, r[4], r[6], r[8], V), ("dW", dW, r[5], r[7], r[9], M)):
        assert got.dtype == x.dtype and got.shape == want.shape
        off = (got.double() - want).abs()
        lim = half * room * 1.01 + (dp + n * H32) * size + half * want.abs() * 1.01 + 1e-30
        assert (off <= lim).all(), (name, float((off / lim).max()))
        if x.dtype == BF and want.numel() > 1000:
            assert float(off.norm()) <= norm_limit(int((t >= 0).sum())) * float(want.norm()), name


# (sizes that the tiles of 128 x 128, 256 x 128 and 256 x 256 take; edges of a tile, of its halves, odd vocabularies)
@pytest.mark.parametrize("M,K,V", [
    (17, 64, 300), (64, 512, 1000), (130, 128, 129), (128, 128, 128), (256, 64, 256), (257, 72, 5003), (300, 264, 40000),
    (255, 8, 1), (100, 64, 2), (2048, 256, 33001), (2049, 128, 8191), (1000, 1024, 20000)])
def test_tiles(M, K, V):
    check(*make(M, K, V, BF, seed=M + V), z=1e-3)


# few rows (streamed), rows off 16-byte lines, short vocabularies whose reduction is split
@pytest.mark.parametrize("M,K,V", [
    (1, 64, 7), (1, 512, 32000), (2, 2048, 5000), (16, 256, 4099), (5, 128, 50257), (33, 100, 700), (64, 8192, 500),
    (40, 1, 60), (77, 33, 2049), (3, 7, 4097), (129, 36, 130), (600, 1001, 999)])
def test_logits_in_memory(M, K, V):
    check(*make(M, K, V, BF, seed=M + V), z=1e-3)


@pytest.mark.parametrize("M,K,V", [(1, 64, 7), (1, 512, 3000), (16, 30, 2049), (130, 65, 257), (777, 101, 5003), (64, 4096, 300)])
def test_fp32(M, K, V):
    check(*make(M, K, V, F32, seed=M + V), z=1e-3)


def test_more_than_one_piece():
    """dl of 4096 x 40001 and of 300 x 2^19 goes by in pieces whose dX add up; so does fp32's."""
    check(*make(4096, 64, 40001, BF, seed=1))
    check(*make(300, 32, (1 << 19) + 9, BF, seed=2))
    check(*make(3000, 24, 50003, F32, seed=3))
    check(*make(12, 40, (1 << 22) - 1, BF, seed=4))


def test_weights_past_2_gib():
    x, W, t, g = make(32, 16384, 70001, BF, seed=5)
    assert W.numel() * 2 > 1 << 31
    check(x, W, t, g)


def test_rows_past_2_gib():
    x, W, t, g = make((1 << 18) + 300, 4096, 260, BF, seed=6)
    assert x.numel() * 2 > 1 << 31
    check(x, W, t, g)


@pytest.mark.parametrize("M,K,V", [(40, 64, 3001), (300, 128, 5000)])
@pytest.mark.parametrize("off", [1, 4])
def test_off_the_lines(M, K, V, off):
    """x and W that begin between 16-byte lines."""
    x, W, t, g = make(M, K, V, BF, seed=7)

    def shifted(a):
        b = torch.empty(a.numel() + off, dtype=a.dtype, device="cuda")[off:].view(a.shape)
        return b.copy_(a)

    check(shifted(x), W, t, g)
    check(x, shifted(W), t, g)


@pytest.mark.parametrize("M,K,V,dtype", [(40, 64, 301, BF), (4, 64, 301, BF), (40, 65, 301, F32)])
def test_targets(M, K, V, dtype):
    x, W, t, g = make(M, K, V, dtype, seed=8, ignore=0.0)
    t[:4] = torch.tensor([0, V - 1, V, -1], device="cuda")
    check(x, W, t, g)
    check(x, W, t.int(), g)
    far = t.clone()
    far[2], far[3] = 1 << 40, -(1 << 40)
    a, b = (api.moe_linear_ce_fwd(x, W, v)[0] for v in (t, far))
    assert torch.equal(a, b) and a[2] == a[3] == 0
    none = torch.full_like(t, -100)
    total = torch.full((3,), 7.0, device="cuda")
    loss, lse = api.moe_linear_ce_fwd(x, W, none, total=total)
    assert not loss.any() and torch.equal(total, torch.zeros(3, device="cuda"))
    one = torch.ones(1, device="cuda")
    dX, dW = api.moe_linear_ce_bwd(one, x, W, none, lse, reduction="mean", total=total)
    assert not dX.any() and not dW.any()


@pytest.mark.parametrize("M,V", [(50, 300), (8, 300), (3000, 600)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_total_and_reductions(M, V, dtype):
    x, W, t, _ = make(M, 64, V, dtype, seed=9)
    total = torch.empty(3, device="cuda")
    loss, lse = api.moe_linear_ce_fwd(x, W, t, total=total)
    count = int(((t >= 0) & (t < V)).sum())
    assert total[1] == count
    # 64-bit sums, rounded once
    s = loss.double().sum()
    assert abs(total[0] - s) <= H32 * s and abs(total[2] - s / count) <= H32 * s / count
    g = torch.tensor([0.7], device="cuda")
    for reduction, each in (("sum", g), ("mean", g / count)):
        a = api.moe_linear_ce_bwd(g, x, W, t, lse, reduction=reduction, total=total)
        b = api.moe_linear_ce_bwd(each.expand(M).contiguous(), x, W, t, lse)
        for u, v in zip(a, b):
            assert torch.equal(u, v)


def test_one_gradient_alone():
    x, W, t, g = make(300, 64, 1000, BF, seed=10)
    _, lse = api.moe_linear_ce_fwd(x, W, t)
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse)
    a = api.moe_linear_ce_bwd(g, x, W, t, lse, dw=False)
    b = api.moe_linear_ce_bwd(g, x, W, t, lse, dx=False)
    assert a[1] is None and b[0] is None and torch.equal(a[0], dX) and torch.equal(b[1], dW)
    assert api.moe_linear_ce_bwd(g, x, W, t, lse, dx=False, dw=False) == (None, None)


def test_no_rows():
    x, W = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(50, 64, dtype=BF, device="cuda")
    t = torch.empty(0, dtype=torch.int64, device="cuda")
    total = torch.full((3,), 7.0, device="cuda")
    loss, lse = api.moe_linear_ce_fwd(x, W, t, total=total)
    assert loss.shape == lse.shape == (0,) and not total.any()
    dX, dW = api.moe_linear_ce_bwd(torch.ones(1, device="cuda"), x, W, t, lse, reduction="sum")
    assert dX.shape == (0, 64) and not dW.any()


@pytest.mark.parametrize("M,K,dtype", [(40, 64, BF), (4, 64, BF), (40, 33, F32)])
def test_far_out_logits(M, K, dtype):
    """Logits of tens of thousands: p is 0 or 1, nothing overflows; all equal: lse is that plus log V."""
    V = 700
    x, W, t, g = make(M, K, V, dtype, seed=11, spread=1)
    x *= 1 << 13
    loss, lse = api.moe_linear_ce_fwd(x, W, t)
    r = reference(x, W, t, 0.0)
    assert torch.isfinite(loss).all() and ((lse - r[1]).abs() <= H32 * (4 * r[1].abs() + 200)).all()
    W.fill_(1.0)
    loss, lse = api.moe_linear_ce_fwd(x, W, t)
    want = x.double().sum(1) + np.log(V)
    assert ((lse - want).abs() <= H32 * (4 * want.abs() + 200)).all()
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse)
    assert torch.isfinite(dX).all() and torch.isfinite(dW).all()


@pytest.mark.parametrize("M,K,dtype", [(40, 64, BF), (4, 64, BF), (40, 33, F32)])
def test_rows_that_are_not_finite_stay_alone(M, K, dtype):
    x, W, t, g = make(M, K, 700, dtype, seed=12, ignore=0.0)
    a, la = api.moe_linear_ce_fwd(x, W, t)
    x[2, 5] = float("nan")
    b, lb = api.moe_linear_ce_fwd(x, W, t)
    keep = torch.arange(M, device="cuda") != 2
    assert torch.isnan(b[2]) and torch.equal(a[keep], b[keep])
    dX, _ = api.moe_linear_ce_bwd(g, x, W, t, lb, dw=False)
    assert torch.isnan(dX[2]).all() and torch.isfinite(dX[keep]).all()


def test_random_inputs_in_norm():
    """Inputs as a model has them: fp32 products of bf16 values, 2048 additions of a row's."""
    gen = torch.Generator(device="cuda").manual_seed(13)
    M, K, V = 1500, 2048, 9001
    x = torch.randn(M, K, generator=gen, device="cuda").bfloat16()
    W = (torch.randn(V, K, generator=gen, device="cuda") / K ** 0.5 * 1.5).bfloat16()
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    g = torch.full((M,), 1.0 / M, device="cuda")
    loss, lse = api.moe_linear_ce_fwd(x, W, t, z_weight=1e-4)
    r = reference(x, W, t, 1e-4, g)
    # a logit: below sqrt(K) roundings of sum |x w| / sqrt(K) ~ 1.5, in fp32
    assert float((loss - r[0]).abs().max()) <= 2048 ** 0.5 * H32 * 1.5 * 2 + 200 * H32
    for got, want in zip(api.moe_linear_ce_bwd(g, x, W, t, lse, z_weight=1e-4), r[4:6]):
        assert float((got.double() - want).norm() / want.norm()) <= norm_limit(M)


def test_differences():
    """The gradient against central differences of the loss in the 64-bit reference, and against autograd."""
    x, W, t, g = make(37, 24, 211, F32, seed=14)
    _, lse = api.moe_linear_ce_fwd(x, W, t, z_weight=1e-2)
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, lse, z_weight=1e-2)
    gen = torch.Generator(device="cuda").manual_seed(15)
    u, v = torch.randn(x.shape, generator=gen, device="cuda"), torch.randn(W.shape, generator=gen, device="cuda")
    h = 1e-4

    def f(s):
        return (reference(x.double() + s * h * u, W.double() + s * h * v, t, 1e-2)[0] * g).sum()

    slope = float((f(1) - f(-1)) / (2 * h))
    got = float((dX.double() * u).sum() + (dW.double() * v).sum())
    # h^2 of third derivatives, and fp32's roundings of 6000 terms of about 1
    assert abs(got - slope) <= 1e-5 * max(1.0, abs(slope)) * 10


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype,M,K,V", [(BF, 70, 64, 501), (BF, 5, 64, 501), (F32, 70, 33, 501)])
def test_autograd(reduction, dtype, M, K, V):
    x, W, t, _ = make(M, K, V, dtype, seed=16)
    x = x.t().contiguous().t().requires_grad_()  # (columns contiguous)
    W.requires_grad_()
    loss = api.linear_cross_entropy(x, W, t, z_weight=1e-3, reduction=reduction)
    up = torch.linspace(0.5, 1.5, M, device="cuda") if reduction == "none" else torch.tensor(1.3, device="cuda")
    gx, gw = torch.autograd.grad(loss, (x, W), up)
    xd, Wd = x.detach().double().requires_grad_(), W.detach().double().requires_grad_()
    l = xd @ Wd.t()
    lse = torch.logsumexp(l, 1)
    ok = t >= 0
    rows = torch.where(ok, lse - l.gather(1, t.clamp(min=0)[:, None])[:, 0] + 1e-3 * lse ** 2, 0.0)
    want = rows if reduction == "none" else rows.sum() if reduction == "sum" else rows.sum() / ok.sum()
    assert torch.allclose(loss.double(), want, rtol=300 * H32, atol=300 * H32)
    for got, ref in zip((gx, gw), torch.autograd.grad(want, (xd, Wd), up.double())):
        rel = float((got.double() - ref).norm() / ref.norm())
        assert rel <= (norm_limit(int(ok.sum())) if dtype == BF else 2000 * H32), rel
    with pytest.raises(ValueError):
        api.linear_cross_entropy(x, W, t, reduction="avg")


@pytest.mark.parametrize("M,K,V,dtype", [(300, 64, 2000, BF), (4, 64, 2000, BF), (70, 33, 501, F32)])
def test_captured_and_replayed(M, K, V, dtype):
    x, W, t, g = make(M, K, V, dtype, seed=17)
    total = torch.empty(3, device="cuda")

    def call():
        loss, lse = api.moe_linear_ce_fwd(x, W, t, total=total)
        return (loss, lse, total) + api.moe_linear_ce_bwd(g[:1], x, W, t, lse, reduction="mean", total=total)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (18, 19, 20):
        for a, b in zip((x, W, t, g), make(M, K, V, dtype, seed=seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        for a, b in zip(got, call()):
            assert torch.equal(a, b)


def test_streams_and_repeats():
    x, W, t, g = make(500, 128, 3000, BF, seed=21)

    def call(stream=None):
        loss, lse = api.moe_linear_ce_fwd(x, W, t, stream=stream)
        return (loss, lse) + api.moe_linear_ce_bwd(g, x, W, t, lse, stream=stream)

    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [call(s) for s in streams for _ in range(2)]
    torch.cuda.synchronize()
    for got in both:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_outputs_end_where_they_end():
    """Rows behind the outputs keep what they hold (the library is given exactly its buffers)."""
    x, W, t, g = make(130, 64, 333, BF, seed=22)
    lib = _lib.load()
    big = [torch.full((n,), 7.0, dtype=d, device="cuda") for n, d in ((130 + 64, F32), (130 + 64, F32), (131 * 64, BF), (334 * 64, BF))]
    n = max(lib.moe_linear_ce_fwd_workspace_bytes(130, 64, 333, 1), lib.moe_linear_ce_bwd_workspace_bytes(130, 64, 333, 1))
    ws = torch.full((n + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert lib.moe_linear_ce_fwd(x.data_ptr(), W.data_ptr(), t.data_ptr(), 64, 130, 64, 333, 0.0, big[0].data_ptr(), big[1].data_ptr(),
                                 None, 1, ws.data_ptr(), n, st) == 0
    assert lib.moe_linear_ce_bwd(g.data_ptr(), 0, None, x.data_ptr(), W.data_ptr(), t.data_ptr(), 64, big[1].data_ptr(), 130, 64, 333,
                                 0.0, big[2].data_ptr(), big[3].data_ptr(), 1, ws.data_ptr(), n, st) == 0
    loss, lse = api.moe_linear_ce_fwd(x, W, t)
    for a, b in zip(big, (loss, lse) + api.moe_linear_ce_bwd(g, x, W, t, lse)):
        assert torch.equal(a[:b.numel()], b.flatten()) and (a[b.numel():] == 7).all()
    assert (ws[n:] == 0xAB).all()


def test_refusals_on_device_tensors():
    x, W, t, g = make(20, 64, 100, BF, seed=23)
    fwd, bwd = api.moe_linear_ce_fwd, api.moe_linear_ce_bwd
    _, lse = fwd(x, W, t)
    for bad in (lambda: fwd(x, W[:, :32].contiguous(), t), lambda: fwd(x, W, t[:5]), lambda: fwd(x, W.t(), t), lambda: fwd(x, W, t.cpu()),
                lambda: bwd(g[:3], x, W, t, lse), lambda: bwd(g, x, W, t, lse, reduction="mean"),
                lambda: bwd(g[:1], x, W, t, lse, reduction="mean"), lambda: bwd(g, x, W, t, lse[:4]),
                lambda: fwd(x, W, t, total=torch.empty(2, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: fwd(x, W.float(), t), lambda: fwd(x, W, t.float()), lambda: fwd(x.half(), W.half(), t),
                lambda: bwd(g.double(), x, W, t, lse)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(_lib.MoeError):
        fwd(x, W, t, z_weight=float("nan"))


@pytest.mark.parametrize("M,K,V", [
    (17, 4, 33), (70, 5, 300), (65, 67, 130), (100, 130, 515), (40, 600, 333),  # small tiles; odd ends in every direction
    (777, 101, 5003), (300, 258, 3070), (1027, 35, 8191),                      # 128 x 128 too
    (33, 4100, 700), (200, 2633, 900),                                         # reductions in ranges, the logits' among them
    (3, 100, 301), (5, 1030, 77), (19, 3, 50), (50, 2, 7), (40, 64, 3), (30, 9, 2),  # few rows; fewer than four of something
])
def test_fp32_of_any_value(M, K, V):
    """Numbers of all 24 bits, rows of very different size.  Each product is off by two half steps at most, its sums by one
    per addition (8 at the joins); what follows as above."""
    gen = torch.Generator(device="cuda").manual_seed(M + V)
    x = torch.randn((M, K), generator=gen, device="cuda") * 10 ** torch.linspace(-3, 0.5, M, device="cuda")[:, None]
    W = torch.randn((V, K), generator=gen, device="cuda") * 10 ** torch.linspace(-3, 0, V, device="cuda")[:, None] / K ** 0.5
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    t[M // 2] = -1
    g = torch.randn(M, generator=gen, device="cuda")
    xd, Wd, z = x.double(), W.double(), 1e-3
    l, size = xd @ Wd.t(), xd.abs() @ Wd.abs().t()
    off = (K + 10) * H32 * size
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    # of an exponential: its argument's and its own; of the sum: its terms', one per addition
    exps = (2 * (l - lse[:, None]).abs() + 4) * H32
    lse_off = (p * (off + exps)).sum(1) + (90 + V / 32 + 3 * lse.abs()) * H32
    got, got_lse = api.moe_linear_ce_fwd(x, W, t, z_weight=z)
    assert ((got_lse.double() - lse).abs() <= lse_off).all()
    ok = t >= 0
    at = t.clamp(min=0)[:, None]
    want = torch.where(ok, lse - l.gather(1, at)[:, 0] + z * lse ** 2, 0.0)
    lim = lse_off * (1 + 2 * z * lse.abs()) + off.gather(1, at)[:, 0] + 4 * H32 * (lse.abs() + l.gather(1, at)[:, 0].abs() + z * lse ** 2)
    assert ((got.double() - want).abs() <= lim).all() and float(got[M // 2]) == 0
    gg = torch.where(ok, g.double(), 0.0)
    f = gg * (1 + 2 * z * lse)
    d = p * f[:, None]
    d_off = d.abs() * (off + exps + lse_off[:, None]) + (p * gg[:, None]).abs() * (2 * z * lse_off)[:, None] + 6 * H32 * d.abs()
    d.scatter_add_(1, at, -gg[:, None])
    d_off += 2 * H32 * d.abs()
    dX, dW = api.moe_linear_ce_bwd(g, x, W, t, got_lse, z_weight=z)
    for a, b, e, s in ((dX, d @ Wd, d_off @ Wd.abs(), (V + 20) * (d.abs() @ Wd.abs())),
                       (dW, d.t() @ xd, d_off.t() @ xd.abs(), (M + 20) * (d.abs().t() @ xd.abs()))):
        assert ((a.double() - b).abs() <= 1.01 * e + H32 * s).all()


def test_fp32_that_is_not_finite():
    """An infinite or NaN value of x stays in its row, one of W in every row that is not left out."""
    M, K, V = 70, 33, 300
    x, W, t, g = make(M, K, V, F32, seed=31, ignore=0)
    want, lse = api.moe_linear_ce_fwd(x, W, t)
    x[7, 3], x[50, 32] = float("inf"), float("nan")
    got, lse2 = api.moe_linear_ce_fwd(x, W, t)
    bad = torch.zeros(M, dtype=torch.bool, device="cuda")
    bad[7] = bad[50] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], want[~bad])
    dX, _ = api.moe_linear_ce_bwd(g, x, W, t, lse2)
    assert torch.isnan(dX[bad]).all() and torch.isfinite(dX[~bad]).all()
    W[299, 0] = -float("inf")
    assert torch.isnan(api.moe_linear_ce_fwd(x, W, t)[0]).all()


@pytest.mark.parametrize("M,K,V", [(1, 1880, 708), (1, 64, 300), (2, 997, 1698), (5, 33, 4097), (16, 2072, 2183), (60, 136, 5000), (128, 256, 3001),
                                   (300, 264, 20011), (512, 64, 1000), (400, 65, 3001)])
def test_few_rows_lose_nothing_in_dl(M, K, V):
    """Gradients of few rows are off by their own rounding alone: half a step of each element, beside what lse, the exponentials
    and the sums leave (dl's second part ends at 2^-16 of it, 2^8 half steps of fp32)."""
    gen = torch.Generator(device="cuda").manual_seed(M + K)
    x = torch.randn((M, K), generator=gen, device="cuda").to(BF)
    W = (torch.randn((V, K), generator=gen, device="cuda") / K ** 0.5).to(BF)
    t = torch.randint(0, V, (M,), generator=gen, device="cuda")
    g = torch.randn(M, generator=gen, device="cuda")
    _, lse = api.moe_linear_ce_fwd(x, W, t)
    got = api.moe_linear_ce_bwd(g, x, W, t, lse)
    xd, Wd = x.double(), W.double()
    d = torch.softmax(xd @ Wd.t(), 1) * g.double()[:, None]
    # the logits' sums and lse (as off as they) in p, 4 half steps per unit of exponent
    far = float((xd.abs() @ Wd.abs().t()).max())
    spread = d.abs() * (2 * K * far + 200) * H32
    d.scatter_add_(1, t[:, None], -g.double()[:, None])
    for a, want, room, n in ((got[0], d @ Wd, (spread + 2 ** 8 * H32 * d.abs()) @ Wd.abs() + V * H32 * (d.abs() @ Wd.abs()), V),
                             (got[1], d.t() @ xd, (spread + 2 ** 8 * H32 * d.abs()).t() @ xd.abs() + 2 * M * H32 * (d.abs().t() @ xd.abs()), M)):
        assert ((a.double() - want).abs() <= H16 * want.abs() * 1.01 + 1.01 * room + 1e-37).all()
        # a rounding is 2^-8 sqrt(1 / 3) in norm at most, of many evenly spread ones
        assert float((a.double() - want).norm()) <= H16 * (1 / 3) ** 0.5 * float(want.norm()) + float(room.norm())
