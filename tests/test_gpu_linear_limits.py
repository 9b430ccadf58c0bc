"""Activations of the linear layer at infinite, NaN and far pre-activations, in every kernel's epilogue."""
import math

import pytest
import torch

from moe_variable_size_amd import api
from tests.gpu_util import log

pytestmark = pytest.mark.gpu

U, V = 2.0 ** -24, 2.0 ** -8
F32, BF16 = torch.float32, torch.bfloat16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
INF, NAN = float("inf"), float("nan")
# each as its formula gives it: z Phi(z), its tanh form and z sigmoid(z) are -inf * 0 at -inf
AT_PLUS_INF = dict.fromkeys(ACTS, INF)
AT_MINUS_INF = {"none": -INF, "relu": 0.0, "gelu": NAN, "gelu_tanh": NAN, "silu": NAN}


def _act(z, kind):
    if kind == "relu":
        return torch.relu(z)
    if kind == "gelu":
        return 0.5 * z * torch.erfc(-z * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    return z * torch.sigmoid(z) if kind == "silu" else z


# (M, K, N, type): a wave per column, streamed, 128 x 128 tiles as a ring of four stages, in ranges
# (joined), in a ring of two, 256 x 128 and 256 x 256 tiles; staged: bf16 off its lines, wide, and
# fp32, whole and in ranges
KERNELS = [(1, 64, 24, BF16), (4, 96, 40, BF16), (4, 96, 40, F32), (16, 200, 72, BF16), (300, 64, 12, BF16),
           (12, 64, 20, F32), (500, 64, 520, BF16), (64, 2048, 192, BF16), (100, 64, 38392, BF16),
           (2437, 64, 2488, BF16), (2890, 64, 2968, BF16), (90, 33, 50, BF16), (2890, 33, 2965, BF16),
           (90, 64, 50, F32), (40, 520, 50, F32)]


@pytest.mark.parametrize("M,K,N,dtype", KERNELS)
@pytest.mark.parametrize("act", ACTS)
def test_infinite_and_nan_pre_activations(M, K, N, dtype, act):
    log(f"limits {M} {K} {N} {dtype} {act}")
    g = torch.Generator(device="cuda").manual_seed(M + N)
    W = (torch.rand((N, K), generator=g, device="cuda") / K + 2.0 ** -12).to(dtype)   # positive
    base = torch.randn((M, K), generator=g, device="cuda").to(dtype)
    for bad, limit in ((INF, AT_PLUS_INF[act]), (-INF, AT_MINUS_INF[act]), (NAN, NAN)):
        x = base.clone()
        rows = sorted({0, M // 2, M - 1})
        x[rows, K // 3] = bad
        want = torch.full((len(rows), N), limit, device="cuda")
        for out in (F32,) if dtype == F32 else (BF16, F32):
            o, z = api.moe_linear_fwd(x, W, act=act, out_dtype=out, save_z=True)
            torch.cuda.synchronize()
            assert torch.allclose(o[rows].float(), want, rtol=0, atol=0, equal_nan=True), (bad, out)
            assert torch.allclose(z[rows].float(), torch.full_like(want, bad), rtol=0, atol=0, equal_nan=True)
            rest = torch.ones(M, dtype=torch.bool, device="cuda")
            rest[rows] = False
            assert bool(o[rest].isfinite().all()) and bool(z[rest].isfinite().all())


def test_gelu_keeps_its_relative_precision_below_zero():
    """gelu(z) = -x Q(x) at z = -x.  Q = exp(-x^2 / 2) G(t), t = 1 / (1 + 0.3 x).  In units of u: the
    exponent's constant and its two products are rounded, 3 x^2 / 2 in the exponential, whose own
    error is 2; t (one sum, a reciprocal of 2) has 3, which G multiplies by at most t G' / G = 2.7;
    G's fit is off by 1.2 and its eight steps' roundings, at most the sum of the partial results over
    G = 4.2; two products: 1.5 x^2 + 18."""
    x = torch.cat([torch.linspace(1e-3, 12.5, 200001, dtype=torch.float64), 10.0 ** torch.linspace(-30, -3, 500).double()])
    z = -x.float()
    o = api.moe_linear_fwd(torch.zeros((1, 1), device="cuda"), torch.zeros((z.numel(), 1), device="cuda"),
                           bias=z.cuda(), act="gelu")
    zd = z.double()
    ref = 0.5 * zd * torch.erfc(-zd * math.sqrt(0.5))
    bound = (1.5 * zd * zd + 18.0) * U
    e = (o[0].cpu().double() / ref - 1.0).abs()
    at = int((e / bound).argmax())
    assert bool((e <= bound).all()), (float(z[at]), float(e[at] / U), float(bound[at] / U))


def test_gelu_far_above_zero_is_its_argument():
    z = torch.tensor([8.0, 13.9, 14.0, 14.1, 14.5, 14.6, 20.0, 1e4, 1e30, 3.4e38], device="cuda")
    for dtype in (F32, BF16):
        b = z.to(dtype)
        o = api.moe_linear_fwd(torch.zeros((1, 1), device="cuda", dtype=dtype),
                               torch.zeros((z.numel(), 1), device="cuda", dtype=dtype), bias=b, act="gelu")
        assert torch.equal(o[0], b)
