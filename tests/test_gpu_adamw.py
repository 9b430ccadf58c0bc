"""AdamW step on the GPU against the 64-bit oracle, element by element.

Tolerances count roundings of half a step (2^-24 in fp32, 2^-8 in bf16).  m: the two coefficients, the
scaled gradient, its product and the sum, at most 5 of |b1 m| + |a1 g|; v: 7 of v; the parameter: 3 of itself
(the decay and the sum) and of the step 3 (rate), 1 (product), 5 (m), 5.5 (v, and 2 for a root off by a whole step),
2.5 (root of the correction), 2 (eps, sum), 3 (a reciprocal off by a whole step, the product): 22 of the step taken with
|b1 m| + |a1 g|.  8-bit states add one rounding of their values (two of v): 24.
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import _lib, api
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

H32 = 2.0 ** -24
F8 = torch.float8_e4m3fn
OPTS = dict(lr=1e-2, betas=(0.9, 0.99), eps=1e-8, weight_decay=0.1)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Set:
    """Tensors of these sizes, `off` elements behind a 16-byte line."""

    def __init__(self, sizes, dtype=torch.float32, gdtype=torch.float32, bits=32, master=False, off=0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(n, std):
            return torch.randn(n + off, generator=gen, device="cuda")[off:] * std

        def place(a, dtype):
            out = torch.empty(a.numel() + off, dtype=dtype if dtype != F8 else torch.uint8, device="cuda")
            out = (out.view(F8) if dtype == F8 else out)[off:]
            (out.view(torch.uint8) if dtype == F8 else out).copy_(a.view(torch.uint8) if dtype == F8 else a)
            return out

        self.bits, self.sizes = bits, sizes
        self.w0 = [rnd(n, 0.5) for n in sizes]
        self.p = [place(w, dtype) for w in self.w0]
        self.master = [place(w, torch.float32) for w in self.w0] if master else None
        self.g = [place(rnd(n, 0.1), gdtype) for n in sizes]
        self.ms = self.vs = None
        m, v = [rnd(n, 0.03) for n in sizes], [rnd(n, 0.1) ** 2 for n in sizes]
        if bits == 32:
            self.m, self.v = [place(a, torch.float32) for a in m], [place(a, torch.float32) for a in v]
        else:
            def codes(n, high):
                c = torch.randint(0, 127, (n,), generator=gen, device="cuda", dtype=torch.uint8)
                return place((c if not high else c ^ (torch.randint(0, 2, (n,), generator=gen, device="cuda") << 7).to(torch.uint8)).view(F8), F8)

            self.m, self.v = [codes(n, True) for n in sizes], [codes(n, False) for n in sizes]
            blocks = [-(-n // 256) for n in sizes]
            self.ms = [rnd(b, 1e-4).abs() for b in blocks]
            self.vs = [rnd(b, 3e-4).abs() for b in blocks]

    def before(self):
        w = self.master or self.p
        out = [[f64(t) for t in w], [f64(t) for t in self.g]]
        if self.bits == 32:
            return out + [[f64(t) for t in self.m], [f64(t) for t in self.v]]
        c = [[t.view(torch.uint8).cpu().numpy() for t in x] for x in (self.m, self.v)]
        return out + [[O.unpack8(a, f64(s)) for a, s in zip(c[0], self.ms)],
                      [O.unpack8(a, f64(s)) ** 2 for a, s in zip(c[1], self.vs)]]

    def step(self, t, **k):
        api.moe_adamw_step(self.p, self.g, self.m, self.v, step=t, masters=self.master, m_scales=self.ms,
                           v_scales=self.vs, **{**OPTS, **k})

    def check(self, before, t, s=1.0, seed=0, opts=OPTS, numbers=None):
        b1, b2 = opts["betas"]
        for i, n in enumerate(self.sizes):
            if not n:
                continue
            w0, g, m0, v0 = (a[i] for a in before)
            w, m, v = O.adamw(w0, g, m0, v0, t, opts["lr"], opts["betas"], opts["eps"], opts["weight_decay"], s)
            room = abs(b1 * m0) + abs((1 - b1) * g * s)
            stepped = opts["lr"] / (1 - b1 ** t) * room / (np.sqrt(v / (1 - b2 ** t)) + opts["eps"])
            tol = H32 * (3 * abs(w) + 3 * abs(w0) + 24 * stepped)
            if self.master:
                got = f64(self.master[i])
                assert (abs(got - w) <= tol).all()
                assert torch.equal(self.p[i], self.master[i].to(self.p[i].dtype))
            else:
                half = 2.0 ** -8 if self.p[i].dtype == torch.bfloat16 else 0.0
                assert (abs(f64(self.p[i]) - w) <= tol + half * (abs(w) + tol)).all(), (i, n)
            if self.bits == 32:
                assert (abs(f64(self.m[i]) - m) <= 5 * H32 * room).all()
                assert (abs(f64(self.v[i]) - v) <= 7 * H32 * v).all()
                continue
            u = O.dither(np.arange(n), i if numbers is None else numbers[i], seed, t)
            for a, uu, codes, scales in ((m, u[0], self.m[i], self.ms[i]), (np.sqrt(v), u[1], self.v[i], self.vs[i])):
                q, sc, near, d = O.pack8(a, uu)
                got = O.e4m3(codes.view(torch.uint8).cpu().numpy())
                assert np.allclose(f64(scales), sc, rtol=16 * H32, atol=0)
                # y / d + u <= 17 is off by at most 20 roundings of 16: only so near a whole number may it differ
                # (m: of the block's largest |b1 m| + |a1 g|, m itself being smaller by at most what 'room' says)
                slack = 20 * H32 * 16 * (1 + np.where(a != 0, room / np.maximum(abs(a), 1e-300), 1))
                sure = near > slack
                assert (got[sure] == q[sure]).all(), (i, n)
                assert (abs(got - q) <= d * 1.001).all()


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 4096, 0, 100003]


@pytest.mark.parametrize("off", [0, 1, 8])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gdtype,master", [
    (torch.float32, torch.float32, False), (torch.float32, torch.bfloat16, False),
    (torch.bfloat16, torch.bfloat16, False), (torch.bfloat16, torch.float32, False),
    (torch.bfloat16, torch.float32, True), (torch.bfloat16, torch.bfloat16, True)])
def test_step(dtype, gdtype, master, bits, off):
    a = Set(SIZES, dtype, gdtype, bits, master, off, seed=3)
    before = a.before()
    a.step(5, seed=11)
    a.check(before, 5, seed=11)


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch(bits):
    a = Set([(37 * i) % 1500 for i in range(131)], torch.bfloat16, torch.float32, bits, True, seed=4)
    before = a.before()
    a.step(1, grad_scale=torch.tensor([0.3], device="cuda"))
    a.check(before, 1, s=float(np.float32(0.3)))


def test_step_and_rate_on_the_device():
    a, b = (Set([3000, 17], torch.float32, torch.float32, 8, seed=5) for _ in range(2))
    before = a.before()
    a.step(1000, seed=2)
    b.step(torch.tensor([1000], dtype=torch.int32, device="cuda"), lr=torch.tensor([1e-2], device="cuda"), seed=2)
    b.check(before, 1000, seed=2)
    for x, y in zip(a.m + a.v, b.m + b.v):  # the rounding's numbers are the same ones
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("t", [1, 2, 1000000])
def test_corrections_on_the_device(t):
    opts = dict(lr=1e-2, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0)
    a = Set([5000], seed=6)
    before = a.before()
    a.step(torch.tensor([t], dtype=torch.int32, device="cuda"), **opts)
    a.check(before, t, opts=opts)


@pytest.mark.parametrize("s", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_that_is_not_finite_changes_nothing(s, bits):
    a = Set([3000, 5], torch.bfloat16, torch.float32, bits, True, seed=7)
    keep = [t.clone() for t in a.p + a.master + a.m + a.v + (a.ms or []) + (a.vs or [])]
    a.step(3, grad_scale=torch.tensor([s], device="cuda"))
    for x, y in zip(a.p + a.master + a.m + a.v + (a.ms or []) + (a.vs or []), keep):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_zeros_and_tiny_blocks():
    """A block of zeros keeps scale 0; one below 2^-100 becomes one; zeros stay zeros at eps = 0 only with NaN."""
    n = 1024
    a = Set([n], bits=8, seed=8)
    a.g[0].zero_()
    for x in (a.m, a.v, a.ms, a.vs):
        x[0].view(torch.uint8).zero_()
    a.g[0][256:512] = 2.0 ** -110
    a.g[0][600] = 1.0
    p = a.p[0].clone()
    a.step(1, weight_decay=0.0, betas=(0.5, 0.5))
    ms, vs = f64(a.ms[0]), f64(a.vs[0])
    assert ms[0] == ms[1] == ms[3] == 0 and vs[0] == vs[1] == vs[3] == 0
    assert ms[2] == np.float32(0.5 / 448) and abs(vs[2] * 448 - 0.5 ** 0.5) < 1e-7
    m = a.m[0].float().cpu()
    assert m[600] == 448 and (m[:600] == 0).all() and (m[601:] == 0).all()
    moved = (a.p[0] != p).nonzero()[:, 0].tolist()
    assert moved == [600]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_are_not_finite_reach_their_block_only(bad):
    a = Set([1024], bits=8, seed=9)
    a.g[0][300] = bad
    a.step(1)
    m = a.m[0].float().cpu().numpy() * np.repeat(f64(a.ms[0]), 256)
    v = a.v[0].float().cpu().numpy() * np.repeat(f64(a.vs[0]), 256)
    assert np.isnan(m[256:512]).all() and np.isnan(v[256:512]).all()
    assert np.isfinite(np.delete(m, range(256, 512))).all() and np.isfinite(np.delete(v, range(256, 512))).all()
    assert torch.isfinite(a.p[0]).sum() >= 1023


def test_rounding_is_right_on_average():
    """States that move by much less than a code's distance per step follow their formulas."""
    n = 1 << 16
    a = Set([n], bits=8, seed=10)
    for x in (a.m, a.v):
        x[0].view(torch.uint8).zero_()
    a.ms[0].zero_(), a.vs[0].zero_()
    a.g[0].fill_(0.37)  # 165.76 of the block's 448: between the codes of 160 and 176
    a.g[0][::256] = 1.0
    m = v = 0.0
    for t in range(1, 201):
        a.step(t, betas=(0.99, 0.99), lr=0.0)
        m, v = 0.99 * m + 0.01 * 0.37, 0.99 * v + 0.01 * 0.37 ** 2
    keep = np.arange(n) % 256 != 0
    m8 = (a.m[0].float().cpu().numpy())[keep]
    r8 = (a.v[0].float().cpu().numpy())[keep]
    # each new value is a mean of one of the two codes (squared, for v) and the true one, so it stays between them
    assert set(np.unique(m8)) == set(np.unique(r8)) == {160.0, 176.0}
    # a rounding's standard deviation is at most half the distance, 8 / 165.76 of the value; that of i steps ago counts 0.99^i
    sigma = 8 / 165.76 / np.sqrt(1 - 0.99 ** 2) / np.sqrt(keep.sum())
    got = m8 * np.repeat(f64(a.ms[0]), 256)[keep]
    assert abs(got.mean() / m - 1) < 6 * sigma
    # the root's mean lies between the codes as the value does, up to what rounding adds to its square:
    # at most the distance times the move towards 165.76, 0.01 / 2 of 13 % per step, over 0.01
    got = r8 * np.repeat(f64(a.vs[0]), 256)[keep]
    assert abs((got ** 2).mean() / v - 1) < 0.13 / 2 * 16 / 165.76 + 12 * sigma


def test_past_four_billion_elements():
    n = (1 << 32) + 700
    gen = torch.Generator(device="cuda").manual_seed(12)
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    lo = (1 << 32) - 512
    p[lo:] = torch.randn(n - lo, generator=gen, device="cuda").bfloat16()
    g[lo:] = torch.randn(n - lo, generator=gen, device="cuda").bfloat16()
    w0, gg = f64(p[lo:]), f64(g[lo:])
    api.moe_adamw_step([p], [g], [m], [v], step=1, m_scales=[ms], v_scales=[vs], seed=3, **OPTS)
    w, mm, vv = O.adamw(w0, gg, 0 * gg, 0 * gg, 1, *OPTS.values())
    assert (abs(f64(p[lo:]) - w) <= 2.0 ** -8 * abs(w) + 1e-6).all()
    u = O.dither(np.arange(lo, n), 0, 3, 1)
    for a, uu, c, s in ((mm, u[0], m, ms), (np.sqrt(vv), u[1], v, vs)):
        q, sc, near, d = O.pack8(a, uu)
        got = O.e4m3(c.view(torch.uint8)[lo:].cpu().numpy())
        assert np.allclose(f64(s[lo // 256:]), sc, rtol=16 * H32, atol=0)
        assert (got[near > 1e-3] == q[near > 1e-3]).all() and (abs(got - q) <= d * 1.001).all()
    assert not p[:lo].any() and not m.view(torch.uint8)[:lo].any() and not ms[:lo // 256].any()


def test_other_stream_and_repeats():
    a, b = (Set([70000, 300], torch.bfloat16, torch.bfloat16, 8, seed=13) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for t in range(1, 4):
        a.step(t, seed=1)
        b.step(t, seed=1, stream=s)
    torch.cuda.synchronize()
    for x, y in zip(a.p + a.m + a.v + a.ms + a.vs, b.p + b.m + b.v + b.ms + b.vs):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_class_captured_and_replayed(bits):
    """Replays of one captured step, with the rate changed between, equal eager steps."""
    def make(capturable):
        gen = torch.Generator(device="cuda").manual_seed(14)
        ps = [torch.randn(sh, generator=gen, device="cuda").to(dt).requires_grad_()
              for sh, dt in (((64, 48), torch.bfloat16), ((7,), torch.float32), ((3, 5, 11), torch.bfloat16))]
        opt = api.AdamW(ps, lr=1e-2, state_bits=bits, master=True, capturable=capturable, seed=9)
        for p in ps:
            p.grad = torch.zeros_like(p)
        return ps, opt

    (pe, eager), (pc, cap) = make(False), make(True)
    graph = None
    for t in range(5):
        if t == 3:
            eager.set_lr(3e-3), cap.set_lr(3e-3)
        for a, b in zip(pe, pc):
            gen = torch.Generator(device="cuda").manual_seed(20 + t)
            a.grad.copy_(torch.randn(a.shape, generator=gen, device="cuda"))
            b.grad.copy_(a.grad)
        eager.step()
        if t == 0:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                cap.step()
            torch.cuda.current_stream().wait_stream(s)
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    cap.step()
            graph.replay()
        torch.cuda.synchronize()
        for a, b, x, y in zip(pe, pc, eager.m, cap.m):
            # the corrections come from the host's double or the device's float: 4 roundings of the step
            assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-6)
            assert torch.allclose(x.float(), y.float(), rtol=0, atol=0)
    assert int(cap.t) == 5 == eager.t


def test_class_saves_loads_and_skips_missing_gradients():
    ps = [torch.randn(300, device="cuda").bfloat16().requires_grad_() for _ in range(3)]
    a = api.AdamW(ps, state_bits=8, master=True, seed=5)
    (ps[0].float().sum() + (ps[2].float() ** 2).sum()).backward()
    keep = ps[1].detach().clone()
    version = ps[0]._version
    a.step()
    assert torch.equal(ps[1].detach(), keep) and not a.m[1].view(torch.uint8).any()
    assert ps[0]._version > version  # a graph that saved it notices
    qs = [p.detach().clone().requires_grad_() for p in ps]
    b = api.AdamW(qs, state_bits=8, master=True)
    b.load_state_dict(a.state_dict())
    for p, q in zip(ps, qs):
        p.grad = torch.ones_like(p).t()
        q.grad = torch.ones_like(q)
    a.step(), b.step()
    for p, q in zip(ps + a.m + a.v, qs + b.m + b.v):
        assert torch.equal(p.detach().view(torch.uint8), q.detach().view(torch.uint8))
    with pytest.raises(ValueError):
        api.AdamW(qs, state_bits=32).load_state_dict(a.state_dict())


def test_refusals_on_device_tensors():
    def t(n, dt=torch.float32):
        return torch.zeros(n, dtype=dt, device="cuda")

    p, ok = [t(8), t(5)], dict(step=1, lr=1e-3)
    call = api.moe_adamw_step
    with pytest.raises(ValueError):
        call(p, [t(8)], [t(8), t(5)], [t(8), t(5)], **ok)
    with pytest.raises(ValueError):
        call(p, [t(8), t(6)], [t(8), t(5)], [t(8), t(5)], **ok)
    with pytest.raises(ValueError):
        call([p[0], p[0]], [t(8), t(8)], [t(8), t(8)], [t(8), t(8)], **ok)
    with pytest.raises(TypeError):
        call(p, [t(8), t(5, torch.bfloat16)], [t(8), t(5)], [t(8), t(5)], **ok)
    with pytest.raises(TypeError):
        call(p, [t(8), t(5)], [t(8), t(5)], [t(8), t(5, torch.float64)], **ok)
    with pytest.raises(TypeError):
        call(p, [t(8), t(5)], [t(8), t(5)], [t(8), t(5)], masters=[t(8), t(5)], **ok)
    with pytest.raises(ValueError):
        call([t((4, 4)).t()[:2].t()], [t((4, 2))], [t((4, 2))], [t((4, 2))], **ok)
    m8 = [t(8, torch.uint8).view(F8), t(5, torch.uint8).view(F8)]
    with pytest.raises(ValueError):
        call(p, [t(8), t(5)], m8, [x.clone() for x in m8], **ok)
    with pytest.raises(ValueError):
        call(p, [t(8), t(5)], m8, [x.clone() for x in m8], m_scales=[t(1), t(2)], v_scales=[t(1), t(1)], **ok)
    with pytest.raises(ValueError):
        call(p, [t(8), t(5)], [t(8), t(5)], [t(8), t(5)], step=t(2, torch.int32), lr=1e-3)
    with pytest.raises(ValueError):
        call(p, [t(8), t(5)], [t(8), torch.zeros(5)], [t(8), t(5)], **ok)
    with pytest.raises(_lib.MoeError):
        call(p, [t(8), t(5)], [t(8), t(5)], [t(8), t(5)], step=0, lr=1e-3)
    with pytest.raises(_lib.MoeError):
        call(p, [t(8), t(5)], [t(8), t(5)], [t(8), t(5)], step=1, lr=float("nan"))
    call([], [], [], [], **ok)


def test_states_in_8_bits_are_those_of_single_roundings():
    """Codes and scales are, bit for bit, what fp32 operations give one by one, over steps that build on each other."""
    f = np.float32
    s = Set([70001, 256, 3], bits=8, seed=77)
    b1, b2, one = f(0.9), f(0.99), f(1.0)
    a1, a2 = f(1.0 - 0.9), f(1.0 - 0.99)
    for t in range(1, 5):
        want = []
        for i, n in enumerate(s.sizes):
            g = s.g[i].cpu().numpy().astype(f)
            rep = lambda a: np.repeat(a.cpu().numpy(), 256)[:n]  # noqa: E731
            m = O.e4m3(s.m[i].view(torch.uint8).cpu().numpy()).astype(f) * rep(s.ms[i])
            r = O.e4m3(s.v[i].view(torch.uint8).cpu().numpy()).astype(f) * rep(s.vs[i])
            m = b1 * m + a1 * g
            r = np.sqrt(b2 * (r * r) + a2 * g * g)
            u = O.dither(np.arange(n), i, 5, t)
            for a, uu in ((m, u[0]), (r, u[1])):
                b = np.zeros(-(-n // 256) * 256, f)
                b[:n] = a
                top = np.abs(b.reshape(-1, 256)).max(1)
                inv = np.repeat(one / top * f(448.0), 256)[:n]
                y = np.abs(a) * inv
                assert y.dtype == f
                d = 2.0 ** (np.maximum(np.frexp(y.astype(np.float64))[1] - 1, -6) - 3)
                want.append((np.sign(a) * np.minimum(np.floor(y / d + uu) * d, 448.0), top * (one / f(448.0))))
        api.moe_adamw_step(s.p, s.g, s.m, s.v, step=t, lr=1e-3, betas=(0.9, 0.99), m_scales=s.ms, v_scales=s.vs, seed=5)
        for i in range(len(s.sizes)):
            for (q, scale), (codes, scales) in zip(want[2 * i:2 * i + 2], ((s.m[i], s.ms[i]), (s.v[i], s.vs[i]))):
                assert np.array_equal(scales.cpu().numpy(), scale)
                assert np.array_equal(O.e4m3(codes.view(torch.uint8).cpu().numpy()), q)
