"""AdamW's counts of steps: each parameter has its own.  Tolerances as in test_gpu_adamw.py, at a parameter's own t."""
import copy

import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

H32 = 2.0 ** -24
BETAS, LR, WD = (0.9, 0.99), 1e-2, 0.1
SHAPES = [(300,), (17, 5), (1000,), (3,)]


def params(dtype=torch.float32, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(s, generator=gen, device="cuda").to(dtype).requires_grad_() for s in SHAPES]


def gradients(step, seed=100):
    gen = torch.Generator(device="cuda").manual_seed(seed + step)
    return [torch.randn(s, generator=gen, device="cuda") * 0.1 for s in SHAPES]


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64).reshape(-1)


# parameter 1 has no gradient until step 6, 2 has one every other step, 3 none at the end
def has(i, step):
    return (True, step >= 6, step % 2 == 0, step < 8)[i]


def follow(opt, ps, run, steps=10):
    """Takes steps with `run` and checks every parameter against 64 bits at its own count."""
    t = [0] * len(ps)
    for step in range(1, steps + 1):
        before = [(f64(p), f64(m), f64(v)) for p, m, v in zip(ps, opt.m, opt.v)]
        gs = gradients(step)
        run(step, gs)
        for i, (p, m, v) in enumerate(zip(ps, opt.m, opt.v)):
            w0, m0, v0 = before[i]
            if not has(i, step):
                assert (f64(p) == w0).all() and (f64(m) == m0).all() and (f64(v) == v0).all()
                continue
            t[i] += 1
            g = f64(gs[i])
            w, m1, v1 = O.adamw(w0, g, m0, v0, t[i], LR, BETAS, 1e-8, WD)
            room = abs(BETAS[0] * m0) + abs((1 - BETAS[0]) * g)
            stepped = LR / (1 - BETAS[0] ** t[i]) * room / (np.sqrt(v1 / (1 - BETAS[1] ** t[i])) + 1e-8)
            # (the corrections of a count on the device: 4 more roundings of the step)
            assert (abs(f64(p) - w) <= H32 * (3 * abs(w) + 3 * abs(w0) + 28 * stepped)).all(), (step, i)
    assert opt.state_dict()["steps"] == t and int(opt.t) == max(t)


def make(**k):
    ps = params()
    return ps, api.AdamW(ps, lr=LR, betas=BETAS, weight_decay=WD, **k)


@pytest.mark.parametrize("capturable", [False, True])
def test_late_and_rare_gradients(capturable):
    ps, opt = make(capturable=capturable)

    def run(step, gs):
        for i, (p, g) in enumerate(zip(ps, gs)):
            p.grad = g if has(i, step) else None
        opt.step()

    follow(opt, ps, run)


def test_first_gradient_after_many_steps_moves_by_the_rate():
    """m / (1 - beta1) over the root of v / (1 - beta2) is 1 at a parameter's first step, whenever that is."""
    ps, opt = make()
    opt.weight_decay = 0.0
    for step in range(300):
        ps[0].grad = torch.ones_like(ps[0])
        opt.step()
    before = ps[1].detach().clone()
    ps[1].grad = torch.full_like(ps[1], 0.3)
    opt.step()
    assert torch.allclose(before - ps[1].detach(), torch.full_like(before, LR), rtol=1e-4, atol=1e-7)


def test_captured_steps_of_some_parameters():
    """A graph of a step that some have a gradient in, one of a step that all have, and eager steps, in turn."""
    ps, opt = make(capturable=True)
    bufs = [torch.zeros(s, device="cuda") for s in SHAPES]
    graphs = {}

    def run(step, gs):
        for b, g in zip(bufs, gs):
            b.copy_(g)
        live = tuple(has(i, step) for i in range(len(ps)))
        for p, b, on in zip(ps, bufs, live):
            p.grad = b if on else None
        if step <= 3:
            opt.step()
            return
        if live not in graphs:
            torch.cuda.synchronize()
            graphs[live] = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graphs[live]):
                opt.step()
        graphs[live].replay()
        torch.cuda.synchronize()

    follow(opt, ps, run, steps=12)
    assert len(graphs) > 2


def test_a_graph_replayed_after_some_went_ahead():
    """All parameters in one graph; eager steps of some of them between its replays."""
    ps, opt = make(capturable=True)
    bufs = [torch.zeros(s, device="cuda") for s in SHAPES]
    for p, b in zip(ps, bufs):
        p.grad = b
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        opt.step()
    t = [0] * len(ps)
    for step in range(1, 9):
        some = step % 3 == 0
        before = [(f64(p), f64(m), f64(v)) for p, m, v in zip(ps, opt.m, opt.v)]
        gs = gradients(step)
        if some:
            for i, (p, g) in enumerate(zip(ps, gs)):
                p.grad = g if i in (0, 2) else None
            opt.step()
        else:
            for b, g in zip(bufs, gs):
                b.copy_(g)
            graph.replay()
        torch.cuda.synchronize()
        for i, p in enumerate(ps):
            w0, m0, v0 = before[i]
            if some and i not in (0, 2):
                assert (f64(p) == w0).all()
                continue
            t[i] += 1
            g = f64(gs[i])
            w, m1, v1 = O.adamw(w0, g, m0, v0, t[i], LR, BETAS, 1e-8, WD)
            room = abs(BETAS[0] * m0) + abs((1 - BETAS[0]) * g)
            stepped = LR / (1 - BETAS[0] ** t[i]) * room / (np.sqrt(v1 / (1 - BETAS[1] ** t[i])) + 1e-8)
            assert (abs(f64(p) - w) <= H32 * (3 * abs(w) + 3 * abs(w0) + 28 * stepped)).all(), (step, i)
    assert opt.state_dict()["steps"] == t


def test_counts_by_number_of_more_tensors_than_a_launch():
    n = 70
    t = torch.arange(1, 2 * n + 1, dtype=torch.int32, device="cuda")
    taken = t.clone()
    numbers = [2 * i + 1 for i in range(n)]
    for bits in (32, 8):
        kind = torch.float32 if bits == 32 else torch.float8_e4m3fn

        def zeros(k, dt=torch.float32):
            return torch.zeros(k, dtype=torch.uint8 if dt != torch.float32 else dt, device="cuda").view(dt)

        def build():
            return ([torch.ones(300 + i, device="cuda") for i in range(n)], [torch.full((300 + i,), 0.1, device="cuda") for i in range(n)],
                    [zeros(300 + i, kind) for i in range(n)], [zeros(300 + i, kind) for i in range(n)],
                    [zeros(2) for _ in range(n)] if bits == 8 else None, [zeros(2) for _ in range(n)] if bits == 8 else None)

        a, b = build(), build()
        opts = dict(lr=LR, betas=BETAS, weight_decay=WD, seed=7)
        counts = t - 1
        api.moe_adamw_step(*a[:4], step=1, counts=counts, numbers=numbers, m_scales=a[4], v_scales=a[5], **opts)
        want = t - 1
        want[1::2] += 1
        assert torch.equal(counts, want) and torch.equal(t, taken)
        for i in range(n):
            each = [x[i:i + 1] if x is not None else None for x in b]
            api.moe_adamw_step(*each[:4], step=t[numbers[i]:numbers[i] + 1], numbers=[numbers[i]], m_scales=each[4],
                               v_scales=each[5], **opts)
        for x, y in zip(a, b):
            for u, v in zip(x or (), y or ()):
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    p, m, v = (torch.zeros(8, device="cuda") for _ in range(3))
    for bad in (dict(numbers=[2 * n]), dict(numbers=[-1])):
        with pytest.raises(Exception):
            api.moe_adamw_step([p], [p.clone()], [m], [v], step=1, lr=LR, counts=t, **bad)
    with pytest.raises(TypeError):
        api.moe_adamw_step([p], [p.clone()], [m], [v], step=1, lr=LR, counts=t.long())
    with pytest.raises(ValueError):
        api.moe_adamw_step([p], [p.clone()], [m], [v], step=1, lr=LR, counts=t.cpu())


@pytest.mark.parametrize("bits", [32, 8])
def test_saved_and_loaded_counts(bits):
    def build(seed=0):
        ps = params(torch.bfloat16, seed)
        return ps, api.AdamW(ps, lr=LR, state_bits=bits, master=True, seed=3)

    def run(ps, opt, step):
        for i, (p, g) in enumerate(zip(ps, gradients(step))):
            p.grad = g.to(p.dtype) if has(i, step) else None
        opt.step()

    ps, a = build()
    for step in range(1, 6):
        run(ps, a, step)
    state = copy.deepcopy(a.state_dict())
    assert state["steps"] == [5, 0, 2, 5] and state["t"] == 5
    for capturable in (False, True):
        qs = [p.detach().clone().requires_grad_() for p in ps]
        b = api.AdamW(qs, state_bits=bits, master=True, capturable=capturable)
        b.load_state_dict(state)
        c_ps = [p.detach().clone().requires_grad_() for p in ps]
        c = api.AdamW(c_ps, state_bits=bits, master=True)
        c.load_state_dict(state)
        for step in range(6, 9):
            run(qs, b, step), run(c_ps, c, step)
        assert b.state_dict()["steps"] == c.state_dict()["steps"] == [8, 3, 4, 7]
        for p, q in zip(qs, c_ps):
            # equal but for the corrections' arithmetic (and a rounding to bf16)
            assert torch.allclose(p.detach().float(), q.detach().float(), rtol=2.0 ** -7, atol=1e-5)
    # a state with one number for all
    old = {k: v for k, v in state.items() if k != "steps"}
    b = api.AdamW(params(torch.bfloat16), state_bits=bits, master=True)
    b.load_state_dict(old)
    assert b.state_dict()["steps"] == [5] * 4
    with pytest.raises(ValueError):
        b.load_state_dict({**state, "steps": [1, 2]})


@pytest.mark.parametrize("capturable", [False, True])
def test_a_refused_step_is_not_counted(capturable):
    ps, opt = make(capturable=capturable)
    ps[0].grad = torch.ones_like(ps[0])
    opt.step()
    ps[1].grad = torch.ones_like(ps[1])
    opt.betas = (1.0, 0.9)
    with pytest.raises(Exception):
        opt.step()
    assert opt.state_dict()["steps"] == [1, 0, 0, 0]
    opt.betas = BETAS
    for p in ps:
        p.grad = None
    opt.step()
    assert opt.state_dict()["steps"] == [1, 0, 0, 0]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("capturable", [False, True])
@pytest.mark.parametrize("some", [False, True])
def test_steps_left_out_are_not_counted(bits, capturable, some):
    """A run in which some steps' scales are not finite equals, bit for bit, the run of the others alone."""
    def run(scales):
        ps = params(torch.bfloat16)
        opt = api.AdamW(ps, lr=LR, betas=BETAS, state_bits=bits, master=True, capturable=capturable, seed=5)
        n = 0
        for s in scales:
            for i, (p, g) in enumerate(zip(ps, gradients(n))):
                p.grad = g.to(p.dtype) if not some or has(i, n) else None
            opt.step(grad_scale=torch.tensor([s], device="cuda"))
            n += bool(np.isfinite(s))
        return ps, opt

    inf, nan = float("inf"), float("nan")
    ps, a = run([inf, 0.5, nan, -inf, 0.25, 1.0, inf, 2.0])
    qs, b = run([0.5, 0.25, 1.0, 2.0])
    assert a.state_dict()["steps"] == b.state_dict()["steps"] and int(a.t) == 4
    for x, y in zip(ps + a.m + a.v + a.masters + (a.m_scale or []) + (a.v_scale or []),
                    qs + b.m + b.v + b.masters + (b.m_scale or []) + (b.v_scale or [])):
        assert torch.equal(x.detach().view(torch.uint8), y.detach().view(torch.uint8))


def test_steps_with_and_without_a_scale():
    """Counts go on through both; tolerances as above (the formulas at the counts)."""
    ps, opt = make()
    count = 0
    for step, s in enumerate([None, None, float("inf"), 0.5, None, float("nan"), 2.0]):
        before = [(f64(p), f64(m), f64(v)) for p, m, v in zip(ps, opt.m, opt.v)]
        gs = gradients(step)
        for p, g in zip(ps, gs):
            p.grad = g
        opt.step() if s is None else opt.step(grad_scale=torch.tensor([s], device="cuda"))
        left_out = s is not None and not np.isfinite(s)
        count += not left_out
        assert opt.t == count and isinstance(opt.t, int)
        for i, p in enumerate(ps):
            w0, m0, v0 = before[i]
            if left_out:
                assert (f64(p) == w0).all()
                continue
            g = f64(gs[i]) * (1.0 if s is None else s)
            w, m1, v1 = O.adamw(w0, g, m0, v0, count, LR, BETAS, 1e-8, WD)
            room = abs(BETAS[0] * m0) + abs((1 - BETAS[0]) * g)
            stepped = LR / (1 - BETAS[0] ** count) * room / (np.sqrt(v1 / (1 - BETAS[1] ** count)) + 1e-8)
            assert (abs(f64(p) - w) <= H32 * (3 * abs(w) + 3 * abs(w0) + 28 * stepped)).all(), (step, i)
    for bad in (torch.ones(2, device="cuda"), torch.ones(1)):
        with pytest.raises(ValueError):
            opt.step(grad_scale=bad)
    with pytest.raises(TypeError):
        opt.step(grad_scale=torch.ones(1, dtype=torch.float64, device="cuda"))
    assert opt.t == count


def test_captured_steps_left_out():
    ps, a = make(capturable=True)
    qs, b = make(capturable=True)
    scale = torch.ones(1, device="cuda")
    bufs = [torch.zeros(s, device="cuda") for s in SHAPES]
    for p, q, g in zip(ps, qs, bufs):
        p.grad = q.grad = g
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.step(grad_scale=scale)
    for step, s in enumerate([0.5, float("inf"), 1.0, float("nan"), 2.0, 0.25]):
        for x, g in zip(bufs, gradients(step)):
            x.copy_(g)
        scale.fill_(s)
        graph.replay()
        torch.cuda.synchronize()
        if np.isfinite(s):
            b.step(grad_scale=scale)
    assert a.state_dict()["steps"] == b.state_dict()["steps"] == [4] * 4
    for x, y in zip(ps + a.m + a.v, qs + b.m + b.v):
        assert torch.equal(x.detach(), y.detach())
