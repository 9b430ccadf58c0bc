"""GPU parity of the dense linear layer (moe_linear_fwd / _bwd) against float64.

Tolerances per element, u = 2^-24 (half a step of fp32), v = 2^-8 (of bf16):
  * a product sum over n terms a_i b_i accumulates roundings of its partial sums,
    whose size is at most about S = sqrt(sum (a b)^2) times a random walk: 8 u
    sqrt(n) S (eight standard deviations of n roundings of at most u S each), and
    n u max|a b| for short sums;
  * an activation has slope at most 1.13 and is evaluated within 8 u (1 + |z|);
  * an output is rounded once: v or u times its value;
  * the backward rounds dz to the inputs' type before the products: independent
    errors of at most v |dz|, so 4 v sqrt(sum (dz b)^2) in their sum.
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from oracle import router_oracle as R
from tests.gpu_util import host, log

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def _rand(shape, dtype, gen, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(DT[dtype])


def _sum_tol(A, B, n):
    """Accumulation error of A @ B over n terms."""
    S = np.sqrt(np.square(A) @ np.square(B))
    return 8 * U * np.sqrt(n) * S + n * U * (np.abs(A).max(initial=0.0) * np.abs(B).max(initial=0.0)) * min(1.0, 16.0 / n)


def _round(dtype):
    return V if dtype == "bf16" else U


def _inputs(M, K, N, dtype, out, bias, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x, W = _rand((M, K), dtype, g), _rand((N, K), dtype, g, K ** -0.5)
    b = _rand((N,), dtype, g, 0.3) if bias else None
    r = _rand((M, N), out, g) if residual else None
    return x, W, b, r


def _cu(t):
    return None if t is None else t.cuda()


def _f64(t):
    return None if t is None else t.double().numpy()


def _check_fwd(M, K, N, dtype="bf16", out="bf16", act="none", bias=True, residual=True, seed=0, x=None):
    log(f"linear fwd M={M} K={K} N={N} {dtype}->{out} {act} bias={bias} residual={residual}")
    xi, W, b, r = _inputs(M, K, N, dtype, out, bias, residual, seed)
    x = xi if x is None else x
    o0 = torch.full((M, N), float("nan"), dtype=DT[out], device="cuda")
    z0 = torch.full((M, N), float("nan"), dtype=DT[dtype], device="cuda")
    o, z = api.moe_linear_fwd(x.cuda(), W.cuda(), bias=_cu(b), act=act, residual=_cu(r),
                              out_dtype=DT[out], out=o0, z=z0)
    o2 = api.moe_linear_fwd(x.cuda(), W.cuda(), bias=_cu(b), act=act, residual=_cu(r), out_dtype=DT[out])
    torch.cuda.synchronize()
    ro, rz = R.linear(_f64(x), _f64(W), _f64(b), act, _f64(r))
    tz = _sum_tol(_f64(x), _f64(W).T, K) + 2 * U * np.abs(rz)
    ez = np.abs(host(z) - rz)
    ok = ez <= tz + _round(dtype) * (np.abs(rz) + tz)
    assert ok.all(), ("z", ez.max())
    to = 1.13 * tz + 8 * U * (1 + np.abs(rz)) + 2 * U * np.abs(ro)
    eo = np.abs(host(o) - ro)
    ok = eo <= to + _round(out) * (np.abs(ro) + to)
    assert ok.all(), ("out", eo.max())
    assert torch.equal(o, o2)


def _check_bwd(M, K, N, dtype="bf16", out="bf16", act="silu", seed=0, **skip):
    log(f"linear bwd M={M} K={K} N={N} {dtype}/{out} {act} {skip}")
    x, W, _, _ = _inputs(M, K, N, dtype, out, False, False, seed)
    g = torch.Generator().manual_seed(seed + 1)
    d, z = _rand((M, N), out, g), _rand((M, N), dtype, g, 1.5)
    got = api.moe_linear_bwd(d.cuda(), x.cuda(), W.cuda(), act=act, z=z.cuda() if act != "none" else None, **skip)
    torch.cuda.synchronize()
    dz = _f64(d) * R.act_grad(_f64(z), act)
    refs = R.linear_grad(_f64(d), _f64(x), _f64(W), _f64(z), act)
    rounded = V if dtype == "bf16" and (act != "none" or out != dtype) else 0.0
    # the derivative's own evaluation: 16 u, against |d_out| times its largest value
    ev = 16 * U * np.abs(_f64(d)) * 1.13
    xf, Wf = _f64(x), _f64(W)
    tols = (_sum_tol(dz, Wf, N) + 4 * rounded * np.sqrt(np.square(dz) @ np.square(Wf)) + ev @ np.abs(Wf),
            _sum_tol(dz.T, xf, M) + 4 * rounded * np.sqrt(np.square(dz.T) @ np.square(xf)) + ev.T @ np.abs(xf),
            _sum_tol(np.ones((1, M)), dz, M)[0] + ev.sum(0))
    for name, flag, o, ref, t in zip(("dX", "dW", "db"), ("dx", "dw", "dbias"), got, refs, tols):
        if skip.get(flag) is False:
            assert o is None
            continue
        e = np.abs(host(o) - ref)
        ok = e <= t + _round(dtype) * (np.abs(ref) + t)  # false for a NaN
        assert ok.all(), (name, e.max())


# tokens from one up, widths around every tile edge, reduction lengths from one
FWD = [(1, 1, 1), (1, 64, 8), (1, 4096, 512), (2, 72, 24), (5, 200, 333), (16, 1000, 64), (17, 1024, 96),
       (33, 7, 130), (64, 2048, 192), (100, 136, 8), (127, 129, 131), (128, 512, 2048), (129, 64, 264),
       (255, 1016, 257), (256, 256, 256), (300, 88, 520), (513, 320, 64), (700, 40, 1), (1030, 2048, 16)]


@pytest.mark.parametrize("M,K,N", FWD)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_forward(M, K, N, dtype, out):
    _check_fwd(M, K, N, dtype, out, act=ACTS[(M + N) % 5], bias=(M + K) % 3 != 0, residual=(K + N) % 2 == 0,
               seed=M + N)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(3, 96, 40), (70, 64, 136), (384, 128, 520), (90, 33, 50)])
def test_forward_activations(act, M, K, N):
    for dtype, out in (("bf16", "bf16"), ("f32", "f32")):
        _check_fwd(M, K, N, dtype, out, act=act, seed=7)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 64, 8), (2, 72, 24), (16, 1000, 64), (33, 7, 130),
                                   (64, 2048, 192), (127, 129, 131), (256, 256, 256), (255, 1016, 264),
                                   (513, 320, 64), (700, 40, 1), (1030, 520, 16), (600, 264, 776)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_backward(M, K, N, dtype, out):
    _check_bwd(M, K, N, dtype, out, act=ACTS[(M + K) % 5], seed=K)


@pytest.mark.parametrize("act", ACTS)
def test_backward_activations_and_skipped_outputs(act):
    for dtype in ("bf16", "f32"):
        _check_bwd(90, 72, 136, dtype, dtype, act=act, seed=3)
        _check_bwd(90, 72, 136, dtype, dtype, act=act, seed=3, dx=False)
        _check_bwd(90, 72, 136, dtype, dtype, act=act, seed=3, dw=False)
        _check_bwd(90, 72, 136, dtype, dtype, act=act, seed=3, dbias=False)
        _check_bwd(90, 72, 136, dtype, dtype, act=act, seed=3, dx=False, dw=False)


def test_no_rows():
    x, W = torch.empty((0, 24), device="cuda"), torch.randn(16, 24, device="cuda")
    assert api.moe_linear_fwd(x, W, act="silu").shape == (0, 16)
    dX, dW, db = api.moe_linear_bwd(torch.empty((0, 16), device="cuda"), x, W)
    assert dX.shape == (0, 24) and not host(dW).any() and not host(db).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_inputs_that_start_between_16_byte_lines(dtype):
    """Views that begin one element into their storage take the element-aligned path."""
    M, K, N = 65, 64, 72
    base = torch.randn(M * K + 1, generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    x = base[1:].view(M, K)
    W = (torch.randn((N, K), generator=torch.Generator().manual_seed(2)) * 0.1).to(DT[dtype])
    xd = base.cuda()[1:].view(M, K)
    assert xd.data_ptr() % 16 != 0
    o = api.moe_linear_fwd(xd, W.cuda())
    ref = _f64(x) @ _f64(W).T
    t = _sum_tol(_f64(x), _f64(W).T, K)
    assert (np.abs(host(o) - ref) <= t + _round(dtype) * (np.abs(ref) + t)).all()
    d = torch.randn((M, N), generator=torch.Generator().manual_seed(3)).to(DT[dtype])
    _, dW, _ = api.moe_linear_bwd(d.cuda(), xd, W.cuda())
    ref = _f64(d).T @ _f64(x)
    t = _sum_tol(_f64(d).T, _f64(x), M)
    assert (np.abs(host(dW) - ref) <= t + _round(dtype) * (np.abs(ref) + t)).all()


def test_residual_in_place_and_guard_rows():
    """out may be the residual's buffer; memory behind the last row stays as it was."""
    M, K, N = 130, 64, 136
    g = torch.Generator().manual_seed(4)
    x, W = _rand((M, K), "bf16", g), _rand((N, K), "bf16", g, 0.1)
    buf = torch.randn((M + 3, N), generator=g).cuda()
    keep = buf.clone()
    want = api.moe_linear_fwd(x.cuda(), W.cuda(), residual=keep[:M].contiguous(), out_dtype=torch.float32)
    out = buf[:M]
    got = api.moe_linear_fwd(x.cuda(), W.cuda(), residual=out, out=out, out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(buf[M:], keep[M:])


def test_nan_and_infinity_reach_the_output():
    x = torch.ones((4, 64)).bfloat16()
    x[1, 5] = float("nan")
    x[2, 5] = float("inf")
    W = torch.ones((8, 64)).bfloat16()
    for act in ("none", "relu"):
        o = host(api.moe_linear_fwd(x.cuda(), W.cuda(), act=act))
        assert np.isnan(o[1]).all() and np.isposinf(o[2]).all() and (o[[0, 3]] == 64).all()


def test_extreme_pre_activations():
    """Activations and their derivatives far out: no NaN where the limit is finite."""
    z = torch.tensor([[-3e38, -1e20, -1e4, -100.0, -20.0, -5.0, -0.0, 0.0, 5.0, 20.0, 100.0, 1e4, 1e20, 3e38]])
    n = z.shape[1]
    x, W = torch.zeros((1, 1)), torch.zeros((n, 1))
    for act in ACTS:
        o = host(api.moe_linear_fwd(x.cuda(), W.cuda(), bias=z[0].cuda(), act=act))
        with np.errstate(all="ignore"):
            ref = R.act(z.double().numpy(), act)
        assert (np.abs(o - ref) <= 1e-6 * np.abs(ref) + 1e-6).all(), (act, o, ref)
        _, _, db = api.moe_linear_bwd(torch.ones((1, n), device="cuda"), x.cuda(), W.cuda(), act=act, z=z.cuda())
        with np.errstate(all="ignore"):
            rg = R.act_grad(np.clip(z.double().numpy(), -1e4, 1e4), act)
        assert (np.abs(host(db) - rg[0]) <= 1e-6 * (1 + np.abs(rg[0]))).all(), (act, host(db), rg)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_autograd(dtype):
    """api.linear's gradients, the residual's among them, against the library's own
    calls; leaves that ask for none get none."""
    M, K, N = 77, 64, 48
    g = torch.Generator().manual_seed(9)
    x, W, b, r = (_rand(s, dtype, g, 0.5).cuda() for s in ((M, K), (N, K), (N,), (M, N)))
    d = _rand((M, N), dtype, g).cuda()
    leaves = [t.clone().requires_grad_() for t in (x, W, b, r)]
    y = api.linear(leaves[0], leaves[1], leaves[2], act="gelu", residual=leaves[3])
    y.backward(d)
    out, z = api.moe_linear_fwd(x, W, bias=b, act="gelu", residual=r, save_z=True)
    want = api.moe_linear_bwd(d, x, W, act="gelu", z=z) + (d,)
    assert torch.equal(y.detach(), out)
    for a, w in zip(leaves, want):
        assert torch.equal(a.grad, w)
    x2 = x.clone().requires_grad_()
    api.linear(x2, W, b, act="silu").backward(d)
    W2 = W.clone().requires_grad_()
    api.linear(x.t().contiguous().t(), W2).backward(d.t().contiguous().t())
    assert x2.grad is not None and W2.grad is not None


def test_refusals_of_the_binding():
    x, W = torch.zeros((4, 8), device="cuda"), torch.zeros((6, 8), device="cuda")
    for kw in (dict(bias=torch.zeros(5, device="cuda")), dict(residual=torch.zeros((4, 5), device="cuda")),
               dict(act="tanh"), dict(out=torch.zeros((4, 7), device="cuda"))):
        with pytest.raises(ValueError):
            api.moe_linear_fwd(x, W, **kw)
    for kw in (dict(bias=torch.zeros(6, device="cuda").bfloat16()), dict(out_dtype=torch.float16),
               dict(residual=torch.zeros((4, 6), device="cuda").bfloat16())):
        with pytest.raises(TypeError):
            api.moe_linear_fwd(x, W, **kw)
    with pytest.raises(api._lib.MoeError):
        api.moe_linear_fwd(x, W, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.moe_linear_fwd(x, W.t())
    with pytest.raises(ValueError):
        api.moe_linear_bwd(torch.zeros((4, 6), device="cuda"), x, W, act="silu")


@pytest.mark.parametrize("M,K,N", [(8, 1024, 128), (130, 512, 256), (520, 264, 520)])
def test_graph_replays_match_eager(M, K, N):
    g = torch.Generator().manual_seed(M)
    x, W, b = _rand((M, K), "bf16", g).cuda(), _rand((N, K), "bf16", g, 0.05).cuda(), _rand((N,), "bf16", g).cuda()
    d = _rand((M, N), "bf16", g).cuda()

    def step():
        o, z = api.moe_linear_fwd(x, W, bias=b, act="silu", save_z=True)
        return (o, z) + tuple(api.moe_linear_bwd(d, x, W, act="silu", z=z))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in (1, 2, 3):
        x.copy_(_rand((M, K), "bf16", torch.Generator().manual_seed(seed)))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, w in zip(out, want):
            assert torch.equal(a, w)


def test_two_streams_at_once():
    M, K, N = 64, 2048, 256
    gs = [torch.Generator().manual_seed(s) for s in (1, 2)]
    xs = [_rand((M, K), "bf16", g).cuda() for g in gs]
    W = _rand((N, K), "bf16", gs[0], 0.02).cuda()
    want = [api.moe_linear_fwd(x, W) for x in xs]
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, st):
            s.wait_stream(torch.cuda.current_stream())
            got.append(api.moe_linear_fwd(x, W, stream=s))
        torch.cuda.synchronize()
        for a, w in zip(got, want):
            assert torch.equal(a, w)


@pytest.mark.parametrize("seed", range(16))
def test_sweep(seed):
    """Sizes around the rules that pick a kernel, both directions."""
    rng = np.random.default_rng(500 + seed)
    M = int(rng.choice([1, 3, 4, 5, 15, 16, 17, 63, 65, 120, 257, 400, 1100]))
    N = int(rng.choice([1, 8, 15, 16, 24, 64, 100, 128, 250, 256, 520, 1096]))
    K = int(rng.choice([1, 8, 30, 64, 72, 127, 192, 500, 1032, 2056]))
    dtype = ["bf16", "f32"][seed % 4 == 3]
    out = "f32" if dtype == "f32" or rng.random() < 0.4 else "bf16"
    act = ACTS[int(rng.integers(5))]
    _check_fwd(M, K, N, dtype, out, act=act, bias=bool(rng.integers(2)), residual=bool(rng.integers(2)), seed=seed)
    _check_bwd(M, K, N, dtype, out, act=act, seed=seed)


def _rows_close(got, x, W, rows):
    xf = x[rows].double().cpu().numpy()
    ref = xf @ W.double().cpu().numpy().T
    t = _sum_tol(xf, W.double().cpu().numpy().T, x.shape[1])
    ok = np.abs(host(got[rows]) - ref) <= t + U * np.abs(ref)
    assert ok.all()


def test_output_past_four_gigabytes():
    M, K, N = 66000, 64, 16384 + 8
    x = torch.randn((M, K), device="cuda").bfloat16()
    W = (torch.randn((N, K), device="cuda") * 0.1).bfloat16()
    o = api.moe_linear_fwd(x, W, out_dtype=torch.float32)
    assert o.numel() * 4 > 1 << 32
    _rows_close(o, x, W, [0, 1, 33000, M - 257, M - 1])


@pytest.mark.parametrize("N", [8, 72])
def test_input_past_two_gigabytes(N):
    """x of more than 2^31 bytes: streamed (N = 8) and staged (N = 72); and its backward,
    where it is the operand read across its rows."""
    M, K = 270000, 4096
    x = torch.empty((M, K), device="cuda", dtype=torch.bfloat16).normal_()
    assert x.numel() * 2 > 1 << 31
    W = (torch.randn((N, K), device="cuda") / 64).bfloat16()
    o = api.moe_linear_fwd(x, W, out_dtype=torch.float32)
    _rows_close(o, x, W, [0, 1000, M - 130, M - 1])
    d = torch.zeros((M, N), device="cuda", dtype=torch.bfloat16)
    d[-3:] = 1.0
    dX, dW, db = api.moe_linear_bwd(d, x, W)
    ref = x[-3:].double().sum(0)
    assert (dW.double() - ref).abs().max() <= V * ref.abs().max() + 1e-5
    assert bool((db == 3).all()) and not bool(dX[: M - 3].any())
    want = W.double().sum(0)
    assert (dX[-1].double() - want).abs().max() <= V * want.abs().max() + 1e-5


def _off(t):
    """The same values in a dense view that begins one element into its storage."""
    s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = s[1:].view(t.shape)
    v.copy_(t)
    return v


@pytest.mark.parametrize("M,K,N", [(300, 128, 264), (40, 1024, 128), (3, 256, 64), (9, 128, 96), (100, 64, 8)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_epilogue_operands_off_their_lines(M, K, N, dtype, out):
    """Bias, residual, z and out between 16-byte lines, with x and W on them."""
    x, W, b, r = (t.cuda() for t in _inputs(M, K, N, dtype, out, True, True, 5))
    kw = dict(act="gelu", out_dtype=DT[out])
    want, wz = api.moe_linear_fwd(x, W, bias=b, residual=r, save_z=True, **kw)
    got, gz = api.moe_linear_fwd(x, W, bias=_off(b), residual=_off(r), out=_off(want), z=_off(wz), **kw)
    assert torch.equal(got, want) and torch.equal(gz, wz)
    d = torch.randn((M, N), device="cuda").to(DT[out])
    for a, c in zip(api.moe_linear_bwd(d, x, W, act="gelu", z=wz), api.moe_linear_bwd(_off(d), x, W, act="gelu", z=_off(wz))):
        assert torch.equal(a, c)
