"""Every tile of the linear layer's bf16 products, dense random operands, every element against a
64-bit product formed on the device; calls repeat bit for bit.

Tolerances per element as for the linear layer's other tests, u = 2^-24, v = 2^-8: a sum of n products
8 u sqrt(n) S, S = sqrt(sum (a b)^2), and n u max|a b| min(1, 16 / n); an activation's slope is at most
1.13 and its value within 8 u (1 + |z|); the output is rounded once.  A bf16 d_out without an
activation is its own dz, so nothing else is rounded in the backward; with one, dz is rounded to bf16
(4 v sqrt(sum (dz b)^2) for independent errors of at most v |dz|) from a derivative within 16 u."""
import math

import pytest
import torch

from moe_variable_size_amd import api
from tests.gpu_util import log
from tests.linear_tiles import PIPELINED, STAGED

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["gelu", "silu", "none", "gelu_tanh", "relu"]


def _randn(shape, seed, std=1.0, dtype=BF16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _off(t):
    """The same values in a dense view that begins one element into its storage."""
    s = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
    v = s[1:].view(t.shape)
    v.copy_(t)
    return v


def _act(z, kind):
    if kind == "relu":
        return torch.relu(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if kind == "silu" else z


def _sum_tol(A, B):
    """Accumulation error of A @ B (64-bit operands)."""
    n = A.shape[1]
    S = torch.sqrt(A.square() @ B.square())
    return 8 * U * math.sqrt(n) * S + n * U * float(A.abs().max() * B.abs().max()) * min(1.0, 16.0 / n)


def _close(got, ref, tol, what):
    half = V if got.dtype == BF16 else U
    e = (got.double() - ref).abs()
    ok = e <= tol + half * (ref.abs() + tol)  # false for a NaN
    assert bool(ok.all()), (what, float(e.max()), int((~ok).sum()))


def _forward(M, K, N, act, out, off, seed):
    log(f"fwd {M} {K} {N} {act} {out} off={off}")
    x, W, b = _randn((M, K), seed), _randn((N, K), seed + 1, K ** -0.5), _randn((N,), seed + 2, 0.3)
    r = _randn((M, N), seed + 3, dtype=out)
    place = _off if off else (lambda t: t)
    outs = []
    for _ in range(3):
        o = place(torch.full((M, N), float("nan"), dtype=out, device="cuda"))
        z = place(torch.full((M, N), float("nan"), dtype=BF16, device="cuda"))
        api.moe_linear_fwd(x, W, bias=place(b), act=act, residual=place(r), out_dtype=out, out=o, z=z)
        outs.append((o, z))
    torch.cuda.synchronize()
    for o, z in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(z, outs[0][1])
    xd, Wd = x.double(), W.double().t().contiguous()
    rz = xd @ Wd + b.double()
    ro = _act(rz, act) + r.double()
    tz = _sum_tol(xd, Wd) + 2 * U * rz.abs()
    _close(outs[0][1], rz, tz, "z")
    _close(outs[0][0], ro, 1.13 * tz + 8 * U * (1 + rz.abs()) + 2 * U * ro.abs(), "out")


def _backward(product, M, K, N, act, out, seed):
    log(f"{product} {M} {K} {N} {act} {out}")
    x, W = _randn((M, K), seed), _randn((N, K), seed + 1, K ** -0.5)
    d, z = _randn((M, N), seed + 2, dtype=out), _randn((M, N), seed + 3, 1.5)
    want = 0 if product == "dX" else 1
    got = []
    for _ in range(3):
        r = api.moe_linear_bwd(d, x, W, act=act, z=None if act == "none" else z, dx=want == 0, dw=want == 1,
                               dbias=False)
        assert r[1 - want] is None and r[2] is None
        got.append(r[want])
    torch.cuda.synchronize()
    assert torch.equal(got[1], got[0]) and torch.equal(got[2], got[0])
    dz, ev = d.double(), None
    if act != "none":
        zd = z.double().requires_grad_()
        dz = torch.autograd.grad(_act(zd, act), zd, dz)[0]
        ev = 16 * U * 1.13 * d.double().abs()
    A, B, E = (dz, W.double(), ev) if want == 0 else \
        (dz.t().contiguous(), x.double(), None if ev is None else ev.t().contiguous())
    tol = _sum_tol(A, B)
    if act != "none" or out != BF16:
        tol = tol + 4 * V * torch.sqrt(A.square() @ B.square())
    if E is not None:
        tol = tol + E @ B.abs()
    _close(got[0], A @ B, tol, product)


@pytest.mark.parametrize("at", range(len(PIPELINED)), ids=lambda i: "-".join(map(str, PIPELINED[i])))
def test_pipelined_tiles(at):
    product, M, K, N, _, _ = PIPELINED[at]
    if product == "fwd":
        _forward(M, K, N, ACTS[at % 5], BF16, False, at)
        _forward(M, K, N, ACTS[(at + 1) % 5], F32, at % 2 == 1, 100 + at)
    else:
        _backward(product, M, K, N, "none", BF16, at)
        _backward(product, M, K, N, ["silu", "gelu", "relu"][at % 3], F32 if at % 2 else BF16, 100 + at)


@pytest.mark.parametrize("product,M,K,N,run", STAGED)
def test_wide_staged_tiles(product, M, K, N, run):
    if product == "fwd":
        _forward(M, K, N, "gelu", BF16, False, 7)
        _forward(M, K, N, "none", F32, True, 8)
    else:
        _backward(product, M, K, N, "none", BF16, 9)
        _backward(product, M, K, N, "silu", BF16, 10)


@pytest.mark.parametrize("act", ACTS)
def test_every_activation_in_the_large_tiles(act):
    """The two large tiles' epilogues with whole lines and, from views off their lines, element by element."""
    for M, K, N in ((2890, 264, 2968), (2437, 264, 2488)):
        _forward(M, K, N, act, BF16, False, 20)
        _forward(M, K, N, act, BF16, True, 21)


def test_large_training_backward_repeats():
    """A training batch's backward (256 x 256 tiles for dX, 256 x 128 for dW) again and again, with other
    work between: equal every time."""
    M, K, N = 8192, 4096, 2048
    x, W = _randn((M, K), 1), _randn((N, K), 2, K ** -0.5)
    d, z = _randn((M, N), 3), _randn((M, N), 4)
    first = api.moe_linear_bwd(d, x, W, act="silu", z=z)
    for i in range(12):
        api.moe_linear_fwd(x[: 64 + 501 * i], W, act="silu")
        for a, b in zip(api.moe_linear_bwd(d, x, W, act="silu", z=z), first):
            assert torch.equal(a, b)


@pytest.mark.parametrize("act", ["none", "relu"])
@pytest.mark.parametrize("M,K,N", [(2437, 2488, 328), (261, 2968, 2896), (300, 40, 48), (77, 33, 50)])
def test_dz_is_rounded_once_to_the_nearest(act, M, K, N):
    """With a derivative of 0 or 1 dz is d_out itself, so an fp32 d_out shows its one rounding to bf16: the
    two products are those of the rounded values, the bias gradient the sum of the unrounded ones."""
    log(f"dz {M} {K} {N} {act}")
    x, W = _randn((M, K), 31), _randn((N, K), 32, K ** -0.5)
    d, z = _randn((M, N), 33, dtype=F32), _randn((M, N), 34)
    dX, dW, db = api.moe_linear_bwd(d, x, W, act=act, z=None if act == "none" else z)
    torch.cuda.synchronize()
    exact = d * (z > 0) if act == "relu" else d
    dz = exact.bfloat16().double()
    for got, A, B, name in ((dX, dz, W.double(), "dX"), (dW, dz.t().contiguous(), x.double(), "dW")):
        _close(got, A @ B, _sum_tol(A, B), name)
    one = torch.ones((1, M), dtype=torch.float64, device="cuda")
    _close(db, exact.double().sum(0), _sum_tol(one, exact.double())[0], "db")
