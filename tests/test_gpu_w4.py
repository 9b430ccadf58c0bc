"""Products with 4-bit weights on the GPU against the 64-bit oracle.

x holds small whole numbers, so that a group's sum of (16 + q) x, sum x and their difference are whole numbers
below 2^24, exact in fp32.  What is off, in half steps of 2^-24: one for each group that is added with its scale,
one for each of 16 waves, and those of the epilogue (bias, residual, routing weight, the adds of k experts), all of
the sum of the groups' magnitudes; then a rounding to the output's type.  With bf16 x of any value a group's products
are exact and its sum is off by one half step per addition of at most 31 |x| (and 15 |x| of the zero point).
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import _lib, api
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

H32, H16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def weight(N, K, group, zeros, E=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lead = () if E is None else (E,)
    groups, cols = -(-K // group), -(-N // 16) * 16
    w = api.W4Weight(
        torch.randint(0, 256, (*lead, N, -(-K // 128) * 64), generator=gen, device="cuda", dtype=torch.uint8),
        (torch.rand((*lead, groups, cols), generator=gen, device="cuda") + 0.5).to(BF),
        torch.randint(0, 16, (*lead, groups, cols), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None,
        N, K, group)
    w.scales[..., N:] = float("nan")  # what lies behind N enters nothing
    return w


def values(w):
    return O.w4_weight(w.codes.cpu().numpy(), f64(w.scales), None if w.zeros is None else w.zeros.cpu().numpy(), w.N, w.K, w.group)


def rows(M, K, seed=1, spread=3):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-spread, spread + 1, (M, K), generator=gen, device="cuda").to(BF)


def group_sizes(x, W, group):
    """sum over groups of |x . W of the group| [M, N]"""
    return sum(abs(x[:, k:k + group] @ W[:, k:k + group].T) for k in range(0, x.shape[1], group))


ACTS = {"none": lambda z: z, "relu": lambda z: np.maximum(z, 0), "silu": lambda z: z / (1 + np.exp(-z)),
        "gelu": lambda z: 0.5 * z * (1 + np.vectorize(__import__("math").erf)(z / 2 ** 0.5)),
        "gelu_tanh": lambda z: 0.5 * z * (1 + np.tanh((2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))}


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [True, False])
@pytest.mark.parametrize("M,N,K", [(1, 1, 8), (1, 16, 128), (1, 4099, 264), (2, 37, 4096), (15, 64, 1032), (16, 129, 2048), (17, 33, 384),
                                   (32, 200, 136), (33, 65, 640), (64, 130, 1024), (65, 47, 72), (200, 31, 1320), (3, 50, 14336),
                                   # more columns: a few rows' tiles of 8 (above), 16 and 32, 16 and 32 dense columns, 32 rows x 64
                                   (2, 4100, 264), (1, 16390, 72), (3, 4100, 264), (4, 8200, 136), (40, 8200, 136)])
def test_linear(M, N, K, group, zeros):
    w, x = weight(N, K, group, zeros, seed=M + N), rows(M, K, seed=K)
    W, xx = values(w), f64(x)
    want, size = xx @ W.T, group_sizes(xx, W, group)
    tol = (-(-K // group) + 16 + 2) * H32 * size
    got = f64(api.moe_linear_w4_fwd(x, w, out_dtype=F32))
    assert got.shape == (M, N) and (abs(got - want) <= tol).all()
    got = f64(api.moe_linear_w4_fwd(x, w))
    assert (abs(got - want) <= tol + H16 * (abs(want) + tol)).all()


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("M,out_dtype", [(3, F32), (40, BF), (18, F32)])
def test_epilogue(act, M, out_dtype):
    N, K = 77, 520
    w, x = weight(N, K, 64, True, seed=2), rows(M, K, seed=3)
    w.scales.mul_(0.01)
    gen = torch.Generator(device="cuda").manual_seed(4)
    bias = torch.randn(N, generator=gen, device="cuda").to(BF)
    res = torch.randn(M, N, generator=gen, device="cuda").to(out_dtype)
    W, xx = values(w), f64(x)
    z = xx @ W.T + f64(bias)
    tol = (-(-K // 64) + 18) * H32 * (group_sizes(xx, W, 64) + abs(f64(bias)))
    want = ACTS[act](z) + f64(res)
    # slopes below 1.13; an activation's own error (1.5 z^2 + 18) of itself (at most |z|)
    tol = 1.13 * tol + (0 if act in ("none", "relu") else 1) * (1.5 * np.minimum(abs(z), 14) ** 2 + 18) * H32 * abs(z) + H32 * abs(want)
    half = H16 if out_dtype == BF else 0
    kw = dict(bias=bias, act=act, residual=res, out_dtype=out_dtype)
    got = api.moe_linear_w4_fwd(x, w, **kw)
    assert (abs(f64(got) - want) <= tol + half * (abs(want) + tol)).all()
    buf = res.clone()
    assert api.moe_linear_w4_fwd(x, w, **{**kw, "residual": buf, "out": buf}) is buf and torch.equal(buf, got)


def test_values_of_any_size():
    """Normally distributed x over six orders of magnitude, rows of zeros, and x that is not finite."""
    M, N, K, G = 20, 48, 1000, 128
    w = weight(N, K, G, True, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = (torch.randn(M, K, generator=gen, device="cuda") * 10 ** torch.linspace(-3, 3, M, device="cuda")[:, None]).to(BF)
    x[3] = 0
    W, xx = values(w), f64(x)
    s = np.repeat(f64(w.scales[:, :N]), G, 0)[:K]
    tol = (G + 8) * 46 * H32 * (abs(xx) @ s) + 30 * H32 * group_sizes(xx, W, G)
    got = f64(api.moe_linear_w4_fwd(x, w, out_dtype=F32))
    assert (abs(got - xx @ W.T) <= tol).all() and (got[3] == 0).all()
    x[5, 7] = float("nan")
    again = f64(api.moe_linear_w4_fwd(x, w, out_dtype=F32))
    assert np.isnan(again[5]).all() and np.array_equal(np.delete(again, 5, 0), np.delete(got, 5, 0))


def oracle_experts(x, W, ids, wt, used=None):
    """(y, sum of the contributions' magnitudes) of the assignments (used: a mask of them)."""
    T, k = ids.shape
    y, size = np.zeros((T, W.shape[1])), np.zeros((T, W.shape[1]))
    for t in range(T):
        for j in range(k):
            e = ids[t, j]
            if 0 <= e < W.shape[0] and (used is None or used[t, j]):
                v = wt[t, j] * (W[e] @ x[t])
                y[t] += v
                size[t] += abs(v)
    return y, size


def routed(T, k, E, seed, bad=0.1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(0, E, (T, k), generator=gen, device="cuda").int()
    off = torch.rand((T, k), generator=gen, device="cuda")
    ids = torch.where(off < bad / 2, -1, torch.where(off < bad, E, ids.long())).int()
    return ids, torch.rand((T, k), generator=gen, device="cuda")


# (the last three have enough experts and columns for the kernel that does not split the reduction: 16, 17 to 32 and more
# rows per expert, an odd and an even number of blocks)
EXPERTS = [(1, 1, 4, 17, 128), (1, 8, 64, 64, 520), (7, 3, 5, 33, 264), (60, 2, 9, 100, 136), (128, 4, 8, 48, 640), (300, 2, 3, 20, 72),
           (40, 2, 256, 70, 392), (150, 4, 32, 930, 264), (500, 3, 16, 1930, 136)]


@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (32, False), (64, True), (128, False)])
@pytest.mark.parametrize("T,k,E,N,K", EXPERTS)
def test_experts(T, k, E, N, K, group, zeros):
    w, x = weight(N, K, group, zeros, E, seed=T), rows(T, K, seed=K)
    ids, wt = routed(T, k, E, seed=T + K)
    W, xx = values(w), f64(x)
    want, _ = oracle_experts(xx, W, ids.cpu().numpy(), f64(wt))
    size = oracle_experts(abs(xx), abs(W), ids.cpu().numpy(), f64(wt))[0]
    tol = (-(-K // group) + 16 + 2 + 2 * k) * H32 * size
    y = torch.full((T, N), float("nan"), device="cuda")
    api.moe_fused_fwd_w4(x, w, api.moe_build_schedule(ids, wt, E), y=y)
    assert (abs(f64(y) - want) <= tol).all()
    y.fill_(float("nan"))
    api.moe_token_fwd_w4(x, w, ids, wt, y=y)
    assert (abs(f64(y) - want) <= tol).all()
    # masked, some over the capacity: the first ones of each expert count
    cap = max(1, T * k // E // 2)
    seen, used = {}, np.zeros((T, k), bool)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            used[t, j] = seen.get(e, 0) < cap
            seen[e] = seen.get(e, 0) + 1
    want, _ = oracle_experts(xx, W, ids.cpu().numpy(), f64(wt), used)
    sched = api.moe_build_schedule(ids, wt, E, layout=api.MOE_LAYOUT_MASKED, capacity=cap)
    assert (abs(f64(api.moe_fused_fwd_w4(x, w, sched)) - want) <= tol).all()
    if k == 1:
        one = api.moe_token_fwd_w4(x, w, ids)
        assert (abs(f64(one) - oracle_experts(xx, W, ids.cpu().numpy(), np.ones((T, k)))[0]) <= tol + 4 * H32 * size / (f64(wt) + 1e-9)).all()


def test_tokens_that_name_an_expert_twice_and_none():
    w, x = weight(40, 136, 32, True, 3, seed=7), rows(4, 136, seed=8)
    ids = torch.tensor([[1, 1], [-1, -1], [3, 2], [0, -7]], dtype=torch.int32, device="cuda")
    W, xx = values(w), f64(x)
    want, _ = oracle_experts(xx, W, ids.cpu().numpy(), np.ones((4, 2)))
    size = oracle_experts(abs(xx), abs(W), ids.cpu().numpy(), np.ones((4, 2)))[0]
    y = f64(api.moe_token_fwd_w4(x, w, ids))
    assert (abs(y - want) <= 30 * H32 * size).all() and (y[1] == 0).all()
    assert (abs(f64(api.moe_fused_fwd_w4(x, w, api.moe_build_schedule(ids, None, 3))) - want) <= 30 * H32 * size).all()


def test_single_tokens_repeat_and_agree_with_dense():
    w, x = weight(300, 1032, 128, True, 6, seed=9), rows(5, 1032, seed=10)
    ids, wt = routed(5, 4, 6, seed=11, bad=0)
    a, b = api.moe_token_fwd_w4(x, w, ids, wt), api.moe_token_fwd_w4(x, w, ids, wt)
    assert torch.equal(a, b)
    one = ids[:, :1].contiguous()
    y = api.moe_token_fwd_w4(x, w, one)
    for t in range(5):
        e = int(one[t, 0])
        dense = api.W4Weight(w.codes[e], w.scales[e], w.zeros[e], w.N, w.K, w.group)
        d = api.moe_linear_w4_fwd(x[t:t + 1], dense, out_dtype=F32)
        assert torch.allclose(y[t:t + 1], d, rtol=0, atol=float(30 * H32 * (x[t].abs().double().sum() * 24)))


def test_no_rows():
    w = weight(40, 136, 32, True, seed=12)
    assert api.moe_linear_w4_fwd(rows(0, 136), w).shape == (0, 40)
    w = weight(40, 136, 32, True, 3, seed=12)
    assert api.moe_token_fwd_w4(rows(0, 136), w, torch.empty((0, 2), dtype=torch.int32, device="cuda")).shape == (0, 40)


def test_codes_past_4_gib():
    """The last rows of the last expert: offsets past 2^32 bytes."""
    N, K, E = (1 << 18) - 5, 12296, 3
    w = weight(N, K, 128, False, E, seed=13)
    assert w.codes.numel() > (1 << 32)
    x, ids = rows(2, K, seed=14), torch.tensor([[2, 0], [1, 2]], dtype=torch.int32, device="cuda")
    lo = N - 70
    part = api.W4Weight(w.codes[:, lo:].contiguous(), w.scales[..., lo // 16 * 16:].contiguous(), None, 70, K, 128)
    s = f64(w.scales[..., lo:N])
    W = np.stack([(O.w4_codes(part.codes[e].cpu().numpy(), K) - 8) * s[e][np.arange(K) // 128].T for e in range(E)])
    xx = f64(x)
    want, _ = oracle_experts(xx, W, ids.cpu().numpy(), np.ones((2, 2)))
    size = oracle_experts(abs(xx), abs(W), ids.cpu().numpy(), np.ones((2, 2)))[0]
    for y in (api.moe_token_fwd_w4(x, w, ids), api.moe_fused_fwd_w4(x, w, api.moe_build_schedule(ids, None, E))):
        assert (abs(f64(y[:, lo:]) - want) <= (97 + 20) * H32 * size).all()
    dense = api.W4Weight(w.codes[2], w.scales[2], None, N, K, 128)
    got = f64(api.moe_linear_w4_fwd(x, dense, out_dtype=F32)[:, lo:])
    assert (abs(got - xx @ W[2].T) <= (97 + 20) * H32 * (abs(xx) @ abs(W[2]).T)).all()


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("shape", [(1, 1), (5, 8), (33, 129), (7, 1000), (3, 20, 264), (2, 17, 515)])
def test_quantize(shape, dtype, symmetric, group):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    W = (torch.randn(shape, generator=gen, device="cuda") + 0.3).to(dtype)
    W.view(-1, shape[-1])[0, :32] = 0  # a group of zeros (of 32)
    w = api.moe_w4_quantize(W, group=group, symmetric=symmetric)
    N, K = shape[-2:]
    Wd = f64(W)
    q = O.w4_codes(w.codes.cpu().numpy(), K)
    g = np.arange(K) // group
    s = np.swapaxes(f64(w.scales)[..., :N], -1, -2)
    z = np.full(s.shape, 8.0) if symmetric else np.swapaxes(w.zeros.cpu().numpy().astype(float)[..., :N], -1, -2)
    assert w.zeros is None if symmetric else True
    _, s0, z0 = O.w4_quantize(Wd, group, symmetric)
    assert (abs(s - s0) <= 2 * H16 * s0).all() and (s == s0).mean() > 0.99  # (a tie's neighbour, by fp32's rounding)
    assert (abs(z - z0) <= 1).all() and (z == z0).mean() > 0.99
    place = np.divide(Wd, s[..., g], out=np.zeros_like(Wd), where=s[..., g] > 0) + z[..., g]
    assert (abs(np.clip(place, 0, 15) - q) <= 0.5 + 1e-4).all()
    back = (q - z[..., g]) * s[..., g]
    assert np.array_equal(f64(api.moe_w4_dequantize(w, F32)), back)
    assert np.array_equal(f64(api.moe_w4_dequantize(w)), O.bf16(back).astype(np.float64))
    # within half a step of what it stands for, up to the bf16 scale's 2^-8 of the range
    assert (abs(back - Wd) <= s[..., g] * (0.5 + 16 * H16 + 0.5 * (not symmetric))).all()
    if dtype == F32:  # of what it stands for itself, the codes are the same again
        again = api.moe_w4_quantize(api.moe_w4_dequantize(w, F32), group=group, symmetric=symmetric)
        assert again.codes.shape == w.codes.shape


def test_quantized_layer_end_to_end():
    """A layer's weights quantised, its single tokens answered: what the codes stand for through moe_linear_fwd, in bf16."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    W = torch.randn(200, 512, generator=gen, device="cuda") / 512 ** 0.5
    x = torch.randn(9, 512, generator=gen, device="cuda").to(BF)
    w = api.moe_w4_quantize(W, group=64)
    a = api.moe_linear_w4_fwd(x, w, act="silu", out_dtype=F32)
    b = api.moe_linear_fwd(x.float(), api.moe_w4_dequantize(w, F32), act="silu")
    # fp32 sums of 512 terms, in two orders and with 16 added to each code
    room = x.abs().double() @ (W.abs().double() + 0.05).t()
    assert ((a - b).abs() <= 600 * H32 * 8 * room).all()


@pytest.mark.parametrize("form", ["dense", "experts", "token"])
def test_captured_and_replayed(form):
    E, N, K, T = 5, 65, 264, 12
    w = weight(N, K, 64, True, None if form == "dense" else E, seed=16)
    x, (ids, wt) = rows(T, K, seed=17), routed(T, 2, E, seed=18)

    def call():
        if form == "dense":
            return api.moe_linear_w4_fwd(x, w)
        if form == "token":
            return api.moe_token_fwd_w4(x, w, ids, wt)
        return api.moe_fused_fwd_w4(x, w, api.moe_build_schedule(ids, wt, E))

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for seed in (19, 20, 21):
        x.copy_(rows(T, K, seed=seed))
        a, b = routed(T, 2, E, seed=seed)
        ids.copy_(a), wt.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, call())  # (k = 2: in any order)


def test_streams():
    w, x = weight(500, 1024, 128, True, 4, seed=22), rows(8, 1024, seed=23)
    ids, wt = routed(8, 2, 4, seed=24)
    sched = api.moe_build_schedule(ids, wt, 4)
    want = [api.moe_token_fwd_w4(x, w, ids, wt), api.moe_fused_fwd_w4(x, w, sched)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [(api.moe_token_fwd_w4(x, w, ids, wt, stream=s), api.moe_fused_fwd_w4(x, w, sched, stream=s)) for s in streams]
    torch.cuda.synchronize()
    for a in got:
        assert torch.equal(a[0], want[0]) and torch.equal(a[1], want[1])


def test_refusals_on_device_tensors():
    w, we = weight(40, 136, 32, True, seed=25), weight(40, 136, 32, True, 3, seed=25)
    x = rows(4, 136)
    ids = torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    lin = api.moe_linear_w4_fwd
    for bad in (lambda: lin(x, we), lambda: lin(rows(4, 128), w), lambda: lin(x.t(), w), lambda: lin(x, w, act="tanh"),
                lambda: lin(x, w, bias=torch.zeros(39, dtype=BF, device="cuda")),
                lambda: lin(x, w, residual=torch.zeros(4, 39, dtype=BF, device="cuda")),
                lambda: lin(x, api.W4Weight(w.codes, w.scales, w.zeros, 40, 136, 16)),
                lambda: lin(x, api.W4Weight(w.codes, w.scales[:, :40].contiguous(), w.zeros, 40, 136, 32)),
                lambda: lin(x, api.W4Weight(w.codes, w.scales, w.zeros[:2], 40, 136, 32)),
                lambda: api.moe_token_fwd_w4(x, w, ids), lambda: api.moe_token_fwd_w4(x, we, ids[:3]),
                lambda: api.moe_fused_fwd_w4(x, we, api.moe_build_schedule(ids, None, 4)),
                lambda: api.moe_fused_fwd_w4(x[:3], we, api.moe_build_schedule(ids, None, 3)),
                lambda: api.moe_w4_quantize(torch.zeros(4, 4, device="cuda"), group=48)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: lin(x.float(), w), lambda: lin(x, w, out_dtype=torch.float16), lambda: lin(x, w.codes),
                lambda: lin(x, w, residual=torch.zeros(4, 40, device="cuda")), lambda: api.moe_token_fwd_w4(x, we, ids.long()),
                lambda: api.moe_w4_quantize(torch.zeros(4, 4, dtype=torch.float16, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    odd = weight(40, 100, 32, True, seed=26)  # K not a multiple of 8
    with pytest.raises(_lib.MoeError):
        lin(rows(4, 100), odd)
    shifted = torch.zeros(4 * 136 + 1, dtype=BF, device="cuda")[1:].view(4, 136)
    with pytest.raises(_lib.MoeError):
        lin(shifted, w)
