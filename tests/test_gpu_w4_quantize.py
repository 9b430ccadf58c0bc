"""4-bit codes of weights whose range is past fp32's, and of weights that are codes' values already."""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from oracle import train_oracle as O
from tests.test_gpu_w4 import f64

pytestmark = pytest.mark.gpu

H16 = 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [3.3e38, 1.75e38, 1e38, 1e-36])
def test_values_near_the_types_ends(size, dtype, symmetric):
    """hi - lo is above fp32's largest number where both are above half of it."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    W = ((torch.rand((5, 264), generator=gen, device="cuda") * 2 - 1) * size).to(dtype)
    W[:, ::32], W[:, 1::32] = size, -size
    w = api.moe_w4_quantize(W, group=32, symmetric=symmetric)
    Wd = f64(W)
    q, s0, z0 = O.w4_quantize(Wd, 32, symmetric)
    g = np.arange(264) // 32
    s = f64(w.scales)[:, :5].T
    z = np.full(s.shape, 8.0) if symmetric else f64(w.zeros)[:, :5].T
    assert (s > 0).all() and (abs(s - s0) <= 2 * H16 * s0).all() and (abs(z - z0) <= 1).all()
    place = Wd / s[:, g] + z[:, g]
    codes = O.w4_codes(w.codes.cpu().numpy(), 264)
    assert (abs(np.clip(place, 0, 15) - codes) <= 0.5 + 1e-4).all()
    # (a value that stands above the largest number is that, rounded: infinity)
    back = f64(api.moe_w4_dequantize(w, F32))
    with np.errstate(over="ignore"):
        assert np.array_equal(back, ((codes - z[:, g]) * s[:, g]).astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("shape", [(33, 129), (7, 1000), (3, 20, 264), (2, 17, 515)])
def test_values_of_codes_are_quantised_to_themselves(shape, symmetric, group):
    """Of what the codes stand for, exact in fp32, a group whose scale and zero point come back has its codes again, and any
    group values within half a step of the new scale and what that scale's rounding to bf16 moves 15 steps by."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    W = torch.randn(shape, generator=gen, device="cuda") + 0.3
    w = api.moe_w4_quantize(W, group=group, symmetric=symmetric)
    first = api.moe_w4_dequantize(w, F32)
    again = api.moe_w4_quantize(first, group=group, symmetric=symmetric)
    N, K = shape[-2:]
    g = np.arange(K) // group

    def parts(v):
        s = np.swapaxes(f64(v.scales)[..., :N], -1, -2)
        z = np.full(s.shape, 8.0) if symmetric else np.swapaxes(f64(v.zeros)[..., :N], -1, -2)
        return O.w4_codes(v.codes.cpu().numpy(), K), s, z

    (q, s, z), (q2, s2, z2) = parts(w), parts(again)
    alike = (s == s2) & (z == z2)
    # the scale comes back where the range is whole, 15 steps of it (symmetric: 7 to one side) up to a rounding of bf16
    lo, hi = np.minimum.reduceat(q, np.arange(0, K, group), -1), np.maximum.reduceat(q, np.arange(0, K, group), -1)
    whole = (np.maximum(hi - z, z - lo) == 7) if symmetric else (np.maximum(hi, z) - np.minimum(lo, z) == 15)
    assert whole.mean() > 0.5 and alike[whole].all()
    assert np.array_equal(q[alike[..., g]], q2[alike[..., g]])
    back = (q2 - z2[..., g]) * s2[..., g]
    assert (abs(back - f64(first)) <= s2[..., g] * (0.5 + 16 * H16 + 0.5 * (not symmetric))).all()
