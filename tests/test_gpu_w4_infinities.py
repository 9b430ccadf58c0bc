"""Products with 4-bit weights of x that is infinite, or so large that it is with a code's 16 added: what the formula gives,
sum (q - z) s x, in every kernel; other rows are what they were, bit for bit.

Sums that are taken again are off by a half step (2^-24) per addition of |w x| at most, K of them, and 4 for w x and the
routing weight.  Those that stay finite with the 16s in them, of large x as of any, by what test_gpu_w4.py counts: products
(16 + q) x are exact, and each of a group's G + 8 additions and its zero point's product is off by a half step of at most
(31 + 15) |x| s (2e37 * 16 is finite, and (q - z) may be 0 there: |w x| does not bound it).
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from tests.test_gpu_w4 import f64, rows, routed, values, weight

pytestmark = pytest.mark.gpu

H32 = 2.0 ** -24
INF = float("inf")
F32, BF = torch.float32, torch.bfloat16


def spoil(x, used):
    """x with rows of several kinds among those at `used`."""
    K = x.shape[1]
    kinds = [((1, INF),), ((K - 1, -INF),), ((2, INF), (K // 2, INF)), ((0, INF), (K - 3, -INF)), ((5, float("nan")), (1, INF)),
             ((3, 3e38), (4, 1e38)), ((K - 2, -2e37), (7, 2e37))]
    x = x.clone()
    for i, m in enumerate(used):
        for k, v in kinds[i % len(kinds)]:
            x[m, k % K] = v
    return x


def product(x, W):
    with np.errstate(all="ignore"):
        return np.stack([(W * r[None, :]).sum(1) for r in x])


def same(got, want, room):
    """Equal where the exact value is not finite or past fp32's range; within room elsewhere."""
    with np.errstate(all="ignore"):
        f = want.astype(np.float32).astype(np.float64)
    special = ~np.isfinite(f)
    assert np.array_equal(got[special], f[special], equal_nan=True)
    assert np.isfinite(got[~special]).all() and (abs(got[~special] - want[~special]) <= room[~special]).all()
    return special


def magnitudes(x, W):
    with np.errstate(all="ignore"):
        return np.nan_to_num(abs(np.where(np.isfinite(x), x, 0.0)) @ abs(W).T)


def scales(w):
    """[.., N, K]"""
    s = np.swapaxes(f64(w.scales)[..., :w.N], -1, -2)
    return s[..., np.arange(w.K) // w.group]


def room(x, W, s, group):
    K = x.shape[1]
    return (K + 4) * H32 * magnitudes(x, W) + (group + 8) * 46 * H32 * magnitudes(x, s) + 1e-30


# (1, 2 and 4 rows, of both halves of an operand's; dense tiles of 16, of 32 rows and 32 and 64 columns)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("M,N,K", [(1, 48, 520), (2, 4100, 264), (4, 20, 1032), (3, 8200, 136), (16, 33, 72), (40, 100, 392), (70, 8200, 136)])
def test_dense(M, N, K, group, zeros):
    w, x = weight(N, K, group, zeros, seed=M), rows(M, K, seed=K)
    w.scales.mul_(0.01)
    clean = api.moe_linear_w4_fwd(x, w, out_dtype=F32)
    used = list(range(0, M, 2))[:14]
    for shift in range(0, 7, 3 if M > 2 else 1):
        bad = spoil(x, used) if shift == 0 else spoil(x.roll(shift, 0), used)
        got = api.moe_linear_w4_fwd(bad, w, out_dtype=F32)
        W, xx = values(w), f64(bad)
        special = same(f64(got), product(xx, W), room(xx, W, scales(w), group))
        assert special[used[0]].any()
        if shift == 0:
            keep = [m for m in range(M) if m not in used]
            assert torch.equal(got[keep], clean[keep])
        if M <= 2:  # every kind in turn in a row of its own
            x = x.clone()
            for i in range(7):
                one = x.clone()
                one[0] = spoil(x[:1].repeat(7, 1), range(7))[i]
                same(f64(api.moe_linear_w4_fwd(one, w, out_dtype=F32)), product(f64(one), W), room(f64(one), W, scales(w), group))


@pytest.mark.parametrize("act", ["relu", "silu", "gelu"])
def test_epilogue_of_infinities(act):
    w, x = weight(40, 136, 32, True, seed=1), rows(5, 136, seed=2)
    x[1, 3], x[3, 100] = INF, -INF
    bias = torch.randn(40, device="cuda").to(BF)
    z = api.moe_linear_w4_fwd(x, w, bias=bias, out_dtype=F32)
    got = api.moe_linear_w4_fwd(x, w, bias=bias, act=act, out_dtype=F32)
    assert torch.isinf(z[[1, 3]]).any()
    fn = {"relu": torch.nn.functional.relu, "silu": lambda v: v / (1 + torch.exp(-v)), "gelu": torch.nn.functional.gelu}[act]
    want = fn(z)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]) and torch.isfinite(got[[0, 2, 4]]).all()


# experts through a schedule in 16, 32 rows, without a split of the reduction, and single tokens
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (32, False)])
@pytest.mark.parametrize("T,k,E,N,K", [(6, 2, 4, 50, 264), (120, 2, 3, 40, 136), (150, 4, 32, 930, 264), (1, 8, 64, 64, 520)])
def test_experts(T, k, E, N, K, group, zeros):
    w, x = weight(N, K, group, zeros, E, seed=T), rows(T, K, seed=K)
    w.scales.mul_(0.01)
    ids, wt = routed(T, k, E, seed=T + K)
    wt += 0.1
    used = list(range(0, T, 3))[:14]
    W, idn, wn = values(w), ids.cpu().numpy(), f64(wt)
    clean = [api.moe_token_fwd_w4(x, w, ids, wt), api.moe_fused_fwd_w4(x, w, api.moe_build_schedule(ids, wt, E))]
    bad = spoil(x, used)
    xx = f64(bad)
    want, size, off, sc = np.zeros((T, N)), np.zeros((T, N)), np.zeros((T, N)), scales(w)
    for t in range(T):
        for j in range(k):
            if 0 <= idn[t, j] < E:
                with np.errstate(all="ignore"):
                    p = product(xx[t:t + 1], W[idn[t, j]])[0]
                    want[t] += wn[t, j] * p
                size[t] += wn[t, j] * magnitudes(xx[t:t + 1], W[idn[t, j]])[0]
                off[t] += wn[t, j] * room(xx[t:t + 1], W[idn[t, j]], sc[idn[t, j]], group)[0]
    # (a sum of assignments whose parts pass fp32's range: either may come first)
    mask = size < 3e38
    for got, was in zip((api.moe_token_fwd_w4(bad, w, ids, wt), api.moe_fused_fwd_w4(bad, w, api.moe_build_schedule(ids, wt, E))), clean):
        g = f64(got)
        same(np.where(mask, g, 0), np.where(mask, want, 0), off + 20 * H32 * size)
        if k <= 2:
            keep = [t for t in range(T) if t not in used]
            assert torch.equal(got[keep], was[keep])


def test_groups_of_scale_zero():
    """0 times what is large is 0, times what is infinite NaN."""
    w, x = weight(20, 264, 32, True, seed=3), rows(3, 264, seed=4)
    w.scales[0, :20] = 0
    x[0, 5] = 3e38
    x[1, 5] = INF
    got = f64(api.moe_linear_w4_fwd(x, w, out_dtype=F32))
    xx = f64(x)
    xx[0, :32] = 0
    W = values(w)
    assert (abs(got[0] - W @ xx[0]) <= 300 * H32 * (abs(W) @ abs(xx[0]))).all()
    assert np.isnan(got[1]).all() and np.isfinite(got[2]).all()
