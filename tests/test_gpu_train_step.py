"""A small routed model trained with the linear cross entropy and AdamW, then served from its 4-bit weights.

    a = silu(x Wa^T),  h = a + sum_j w_j E[id_j] a,  loss = cross entropy of h Wo^T + balance loss of the router

Gradients in fp32 are compared with autograd in 64 bits of the same formulas, at the library's weights and choice of experts,
in norm: a sum of n products is off by n half steps (2^-24) of their magnitudes at most, and from its norm that differs
by sqrt n where signs are mixed, which the sum of n errors of mixed signs gains; the longest chain of sums has
K + H + E + V + T terms and some 50 roundings of exponentials, weights and products.
"""
import numpy as np
import pytest
import torch

from moe_variable_size_amd import api
from oracle import train_oracle as O

pytestmark = pytest.mark.gpu

H32, H16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32
T, K, H, E, TOP, V = 57, 40, 72, 6, 2, 331
G = 32  # of 4-bit weights: a group's sum is off by a half step per addition of at most 46 |x| scale


def parameters(dtype, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5).to(dtype).requires_grad_()
            for s in ((H, K), (E, H), (E, H, H), (V, H))]


def batch(dtype, seed):
    gen = torch.Generator(device="cuda").manual_seed(100 + seed)
    x = torch.randn((T, K), generator=gen, device="cuda").to(dtype)
    t = torch.randint(0, V, (T,), generator=gen, device="cuda")
    return x, torch.where(torch.arange(T, device="cuda") % 7 == 3, torch.full_like(t, -100), t)  # prompt tokens


def loss_of(p, x, t):
    Wa, Wr, We, Wo = p
    a = api.linear(x, Wa, act="silu")
    logits = api.linear(a, Wr, out_dtype=F32)
    ids, w = api.route(logits, TOP)
    h = a + api.moe(a, We, ids, w).to(a.dtype)
    return api.linear_cross_entropy(h, Wo, t, z_weight=1e-3) + 0.01 * api.router_loss(logits, ids)[0], ids


def exact_gradients(p, x, t, ids):
    """(loss, gradients) in 64 bits"""
    Wa, Wr, We, Wo = q = [a.detach().double().cpu().requires_grad_() for a in p]
    x, t, ids = x.double().cpu(), t.cpu(), ids.long().cpu()
    a = torch.nn.functional.silu(x @ Wa.t())
    logits = a @ Wr.t()
    s = torch.softmax(logits, 1)
    w = s.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    h = a + sum(w[:, j:j + 1] * torch.stack([We[ids[i, j]] @ a[i] for i in range(T)]) for j in range(TOP))
    l = h @ Wo.t()
    lse = torch.logsumexp(l, 1)
    ok = t >= 0
    ce = lse - l.gather(1, t.clamp(min=0)[:, None])[:, 0] + 1e-3 * lse ** 2
    counts = torch.bincount(ids.reshape(-1), minlength=E).double()
    loss = ce[ok].mean() + 0.01 * E * (counts / (T * TOP) * s.mean(0)).sum()
    return loss, torch.autograd.grad(loss, q)


def test_steps_in_fp32():
    p = parameters(F32)
    opt = api.AdamW(p, lr=1e-2, weight_decay=0.1)
    limit = (K + H + E + V + T + 50) * H32
    for step in range(1, 4):
        x, t = batch(F32, step)
        before = [a.detach().clone() for a in p]
        states = [(m.clone(), v.clone()) for m, v in zip(opt.m, opt.v)]
        opt.zero_grad()
        loss, ids = loss_of(p, x, t)
        loss.backward()
        want, grads = exact_gradients(before, x, t, ids)
        assert abs(float(loss.detach()) - float(want.detach())) <= limit * float(want.detach())
        for a, g in zip(p, grads):
            assert float((a.grad.double().cpu() - g).norm()) <= limit * float(g.norm())
        opt.step()
        for a, b, (m, v) in zip(p, before, states):
            w, _, _ = O.adamw(*(z.cpu().numpy().reshape(-1) for z in (b, a.grad, m, v)), step, 1e-2, (0.9, 0.999), 1e-8, 0.1)
            # 4 roundings of w, and 16 of what its change is made of (hardware's root and quotient among them): lr times
            # the corrected mean of the t gradients' magnitudes over the root of that of their squares, below sqrt t
            b = b.cpu().numpy().reshape(-1).astype(np.float64)
            tol = 4 * H32 * (abs(w) + abs(b)) + 16 * H32 * 1e-2 * 2
            assert (abs(a.detach().cpu().numpy().reshape(-1) - w) <= tol).all()


def test_gradients_against_differences():
    """Along one direction of the experts and the output layer (where the layers before the router move, the choice of experts
    does, and the loss jumps: those gradients are compared above), in fp32: a central difference of step e is off by e^2 / 6 times a third derivative of
    order 10 and by two roundings of the loss, (number of its terms' sums) half steps each, over 2 e."""
    p, (x, t) = parameters(F32, 3), batch(F32, 9)
    loss, ids = loss_of(p, x, t)
    loss.backward()
    gen = torch.Generator(device="cuda").manual_seed(5)
    d = [torch.randn(a.shape, generator=gen, device="cuda") / a.numel() ** 0.5 for a in p]
    d[0].zero_(), d[1].zero_()
    slope = sum(float((a.grad.double() * b.double()).sum()) for a, b in zip(p, d))
    e = 2.0 ** -6
    ends = []
    for s in (e, -e):
        q = [(a.detach() + s * b) for a, b in zip(p, d)]
        l, other = loss_of(q, x, t)
        assert torch.equal(ids, other)
        ends.append(float(l.detach()))
    assert abs((ends[0] - ends[1]) / (2 * e) - slope) <= 10 * e * e / 6 + (K + H + E + V + T + 50) * H32 * float(loss.detach()) / e


@pytest.mark.parametrize("bits", [32, 8])
def test_trained_in_bf16_and_served_from_4_bits(bits):
    p = parameters(BF, 1)
    opt = api.AdamW(p, lr=1e-3, state_bits=bits, master=True, seed=3)
    for step in range(1, 4):
        x, t = batch(BF, step)
        opt.zero_grad()
        loss, _ = loss_of(p, x, t)
        loss.backward()
        assert torch.isfinite(loss) and all(torch.isfinite(a.grad).all() for a in p)
        opt.step()
        for a, w in zip(p, opt.masters):
            assert torch.equal(a.detach().reshape(-1), w.to(BF).reshape(-1))
    Wa, Wr, We, Wo = (a.detach() for a in p)
    qa, qe, qo = (api.moe_w4_quantize(a, group=G) for a in (Wa, We, Wo))
    # each stage against 64 bits at its own inputs, with the values that the codes stand for (exact in fp32)
    da, de, do = (api.moe_w4_dequantize(q, F32).double() for q in (qa, qe, qo))
    for rows in (1, 4, T):
        x = batch(BF, 20)[0][:rows].contiguous()
        a = api.moe_linear_w4_fwd(x, qa, act="silu")
        z = x.double() @ da.t()
        off = 100 * H32 * (x.double().abs() @ da.abs().t()) + (G + 8) * 46 * H32 * (x.double().abs() @ scale_of(qa))
        want = torch.nn.functional.silu(z)
        assert ((a.double() - want).abs() <= H16 * want.abs() * 1.01 + 1.1 * off + 8 * H32 * want.abs()).all()
        ids, w = api.moe_route_fwd(api.moe_linear_fwd(a, Wr, out_dtype=F32), TOP)
        token = api.moe_token_fwd_w4(a, qe, ids, w)
        routed = api.moe_fused_fwd_w4(a, qe, api.moe_build_schedule(ids, w, E))
        want, size, fine = torch.zeros_like(token, dtype=torch.double), 0, 0
        for j in range(TOP):
            wj, M = w[:, j:j + 1].double(), de[ids[:, j].long()]
            want = want + wj * torch.bmm(M, a.double()[:, :, None])[:, :, 0]
            size = size + wj * torch.bmm(M.abs(), a.double().abs()[:, :, None])[:, :, 0]
            fine = fine + wj * torch.bmm(scale_of(qe).transpose(1, 2).contiguous()[ids[:, j].long()], a.double().abs()[:, :, None])[:, :, 0]
        off = 100 * H32 * size + (G + 8) * 46 * H32 * fine
        assert ((token.double() - want).abs() <= off).all() and ((routed.double() - want).abs() <= off).all()
        h = (a.float() + token).to(BF)
        logits = api.moe_linear_w4_fwd(h, qo, out_dtype=F32)
        want, size = h.double() @ do.t(), h.double().abs() @ do.abs().t()
        assert ((logits.double() - want).abs() <= 100 * H32 * size + (G + 8) * 46 * H32 * (h.double().abs() @ scale_of(qo))).all()
        # the loss of the same answers, by the layer that keeps no logits
        t = torch.arange(rows, device="cuda") % V
        loss, _ = api.moe_linear_ce_fwd(h, do.to(BF), t)
        l = h.double() @ do.to(BF).double().t()
        want = torch.logsumexp(l, 1) - l.gather(1, t[:, None])[:, 0]
        assert ((loss.double() - want).abs() <= (2 * H + 90 + 2 * 40) * H32 * (1 + l.abs().amax(1)) * (1 + h.double().abs().sum(1))).all()


def scale_of(q):
    """the scales [.., K, N] of every weight, transposed"""
    s = q.scales[..., :q.N].double()
    return s.repeat_interleave(q.group, -2)[..., :q.K, :].contiguous()


def test_whole_step_captured_and_replayed():
    """Layer, loss, gradients and update in one graph; replays with new data in between equal eager steps."""
    def build():
        gen = torch.Generator(device="cuda").manual_seed(7)
        W = [(torch.randn(s, generator=gen, device="cuda") * 0.1).to(BF) for s in ((H, K), (V, H))]
        m = [torch.zeros(a.numel(), device="cuda") for a in W]
        v = [torch.zeros(a.numel(), device="cuda") for a in W]
        return W, m, v, torch.zeros(1, dtype=torch.int32, device="cuda")

    lr, one = torch.full((1,), 1e-2, device="cuda"), torch.ones(1, device="cuda")

    def step(W, m, v, count, x, t):
        a, z = api.moe_linear_fwd(x, W[0], act="silu", save_z=True)
        total = torch.empty(3, device="cuda")
        loss, lse = api.moe_linear_ce_fwd(a, W[1], t, total=total)
        da, dWo = api.moe_linear_ce_bwd(one, a, W[1], t, lse, reduction="mean", total=total)
        _, dWa, _ = api.moe_linear_bwd(da, x, W[0], act="silu", z=z, dx=False, dbias=False)
        count += 1
        api.moe_adamw_step(W, [dWa, dWo], m, v, step=count, lr=lr)
        return loss, total

    x, t = batch(BF, 0)
    eager, graphed = build(), build()
    step(*eager, x, t)
    step(*graphed, x, t)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*graphed, x, t)
    for seed in range(1, 5):
        for a, b in zip((x, t), batch(BF, seed)):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        for a, b in zip(got, step(*eager, x, t)):
            assert torch.equal(a, b)
        for a, b in zip(eager[0] + eager[1] + eager[2], graphed[0] + graphed[1] + graphed[2]):
            assert torch.equal(a, b)
