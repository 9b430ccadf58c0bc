"""Timed cases of the router, the router losses and the dense linear layer.

Each case is one call (or one forward + backward pair) of an operator as a
program that trains or serves an MoE layer makes it.  run() computes it in
plain torch, or, with ``own`` set, through the library.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a decode batch's routing: 128 tokens, 64 experts, 8 of them per token
        {"name": "route decode", "op": "route", "T": 128, "E": 64, "k": 8, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "renorm": True, "dtype": "f32"},
        # a prefill batch, bf16 logits, weights left as probabilities
        {"name": "route prefill bf16", "op": "route", "T": 8192, "E": 60, "k": 4, "score": "softmax",
         "bias": False, "groups": 1, "topk_groups": 1, "renorm": False, "dtype": "bf16"},
        # a large training batch: sigmoid scores, a balance bias, 4 of 8 groups
        {"name": "route grouped", "op": "route", "T": 65536, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "topk_groups": 4, "renorm": True, "dtype": "f32"},
        # the gradient of a training batch's routing weights, back to every logit
        {"name": "route backward", "op": "route_bwd", "T": 65536, "E": 128, "k": 8,
         "score": "softmax", "renorm": False, "dtype": "f32"},
        # the balance and z losses of a training batch, forward and backward
        {"name": "losses", "op": "loss", "T": 65536, "E": 128, "k": 8, "score": "softmax",
         "dtype": "f32"},
        # the losses of a short odd batch with sigmoid scores and bf16 logits
        {"name": "losses small", "op": "loss", "T": 777, "E": 60, "k": 6, "score": "sigmoid",
         "dtype": "bf16"},
        # one token through a dense projection
        {"name": "linear 1 token", "op": "linear", "M": 1, "K": 4096, "N": 2048, "act": "silu",
         "bias": True, "residual": False, "save": False, "dtype": "bf16", "out": "bf16"},
        # a decode batch through a shared expert's projection, added to the routed output
        {"name": "linear decode", "op": "linear", "M": 128, "K": 7168, "N": 2048, "act": "none",
         "bias": False, "residual": True, "save": False, "dtype": "bf16", "out": "f32"},
        # the router's logits
        {"name": "linear router", "op": "linear", "M": 8192, "K": 4096, "N": 64, "act": "none",
         "bias": True, "residual": False, "save": False, "dtype": "bf16", "out": "f32"},
        # a training batch through a dense layer, pre-activations kept
        {"name": "linear train", "op": "linear", "M": 8192, "K": 4096, "N": 4096, "act": "gelu",
         "bias": True, "residual": True, "save": True, "dtype": "bf16", "out": "bf16"},
        # a training batch's backward
        {"name": "linear backward", "op": "linear_bwd", "M": 8192, "K": 4096, "N": 2048,
         "act": "silu", "bias": True, "dtype": "bf16", "out": "bf16"},
        # a small fp32 layer with every size odd
        {"name": "linear backward f32 odd", "op": "linear_bwd", "M": 1237, "K": 1001, "N": 499,
         "act": "relu", "bias": True, "dtype": "f32", "out": "f32"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "loss", "linear", "linear", "linear_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("route", "route_bwd", "loss"):
        E = _log_int(rng, 4, 512)
        T = _log_int(rng, 1, min(65536, (1 << 24) // E))
        k = rng.randint(1, min(16, E))
        c = {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(["softmax", "sigmoid"]),
             "dtype": dtype}
        if op != "loss":
            c["renorm"] = rng.random() < 0.5
        if op == "route":
            c.update(bias=rng.random() < 0.5, groups=1, topk_groups=1)
            if rng.random() < 0.4:
                g = rng.choice([2, 4, 8])
                c["E"] = E = max(2, E // g) * g
                c.update(groups=g, topk_groups=rng.randint(1, g))
                c["k"] = min(k, c["topk_groups"] * (E // g))
        return c
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    out = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
    K = _log_int(rng, 64, 8192)
    N = _log_int(rng, 8, 8192)
    if rng.random() < 0.6:  # most layers' widths are multiples of 8
        K, N = (K + 7) // 8 * 8, (N + 7) // 8 * 8
    most = (1 << 37) if op == "linear" else (1 << 36)
    M = _log_int(rng, 1, max(1, min(8192, most // (K * N))))
    c = {"op": op, "M": M, "K": K, "N": N, "act": act, "bias": rng.random() < 0.6, "dtype": dtype,
         "out": out}
    if op == "linear":
        c.update(residual=rng.random() < 0.4, save=rng.random() < 0.4)
    return c


# ---- the plain forms ---------------------------------------------------------------------------

def _scores(l, score):
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True)
    return 1.0 / (1.0 + torch.exp(-l))


def _route(logits, bias, k, c):
    """With a bias the choice goes by computed values, which may lie next to each other: 64 bits."""
    T, E = logits.shape
    l = logits.float() if bias is None else logits.double()
    s = _scores(l, c["score"])
    G = c.get("groups", 1)
    v = l if bias is None else s + bias.double()
    if G > 1:
        if bias is None:
            grp = v.view(T, G, E // G).amax(2)
        else:
            grp = torch.sort(v.view(T, G, E // G), dim=2, descending=True)[0][:, :, :2].sum(2)
        best = torch.sort(grp, dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
        kept = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, best, True)
        v = torch.where(kept.repeat_interleave(E // G, 1), v, -math.inf)
    ids = torch.sort(v, dim=1, descending=True, stable=True)[1][:, :k]
    w = torch.gather(s, 1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return ids.int(), w.float()


def _route_bwd(g, logits, ids, w, c):
    l = logits.float()
    idx = ids.long()
    d = torch.zeros_like(l)
    if c["renorm"]:
        t = w * (g - (g * w).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            t = t * (1.0 - _scores(torch.gather(l, 1, idx), "sigmoid"))
        d.scatter_(1, idx, t)
    elif c["score"] == "softmax":
        p = _scores(l, "softmax")
        d.scatter_(1, idx, g)
        d = p * (d - (d * p).sum(1, keepdim=True))
    else:
        s = _scores(torch.gather(l, 1, idx), "sigmoid")
        d.scatter_(1, idx, g * s * (1.0 - s))
    return d.to(logits.dtype)


def _loss(g, logits, ids, c):
    l = logits.float()
    T, E = l.shape
    f = torch.bincount(ids.reshape(-1).long(), minlength=E).float() * (E / ids.numel())
    m = l.amax(1, keepdim=True)
    e = torch.exp(l - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    p = e / total
    if c["score"] == "softmax":
        q = p
    else:
        s = _scores(l, "sigmoid")
        q = s / s.sum(1, keepdim=True)
    losses = torch.stack([(f * q.mean(0)).sum(), (lse * lse).mean()])
    gb, gz = g[0] / T, g[1] / T
    d = gb * q * (f - (f * q).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1.0 - s)
    d = d + gz * 2.0 * lse * p
    return losses, d.to(logits.dtype)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        u = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)
        t = torch.tanh(u)
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _linear(s, c):
    z = s["x"].float() @ s["W"].float().t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    out = _act(z, c["act"])
    if s["residual"] is not None:
        out = out + s["residual"].float()
    out = out.to(DTYPES[c["out"]])
    return (out, z.to(s["x"].dtype)) if c["save"] else (out,)


def _linear_bwd(s, c):
    dt = s["x"].dtype
    dz = s["d_out"].float()
    if s["z"] is not None:
        dz = dz * _act_grad(s["z"].float(), c["act"])
    dx = (dz @ s["W"].float()).to(dt)
    dw = (dz.t() @ s["x"].float()).to(dt)
    return (dx, dw, dz.sum(0).to(dt)) if c["bias"] else (dx, dw)


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)

    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("route", "route_bwd", "loss"):
        T, E, k = c["T"], c["E"], c["k"]
        # a router's logits: some experts liked by most tokens, others by few
        s["logits"] = (randn(T, E, std=1.5) + randn(E, std=0.5)).to(dt)
        s["bias"] = randn(E, std=0.1) if c.get("bias") else None
        if c["op"] != "route":
            s["ids"], s["w"] = _route(s["logits"], None, k, {"score": c["score"], "renorm": c.get("renorm", True)})
        if c["op"] == "route_bwd":
            s["g"] = randn(T, k)
        if c["op"] == "loss":
            s["g"] = torch.tensor([1e-2, 1e-3], device=dev) * T
        return s
    M, K, N = c["M"], c["K"], c["N"]
    s["x"] = randn(M, K, dtype=dt)
    s["W"] = randn(N, K, std=1.0 / math.sqrt(K), dtype=dt)
    s["bias"] = randn(N, std=0.2, dtype=dt) if c["bias"] else None
    if c["op"] == "linear":
        s["residual"] = randn(M, N, dtype=DTYPES[c["out"]]) if c["residual"] else None
    else:
        s["d_out"] = randn(M, N, dtype=DTYPES[c["out"]])
        s["z"] = randn(M, N, dtype=dt) if c["act"] != "none" else None
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    if c["op"] == "route":
        return _route(state["logits"], state["bias"], c["k"], c)
    if c["op"] == "route_bwd":
        return _route_bwd(state["g"], state["logits"], state["ids"], state["w"], c)
    if c["op"] == "loss":
        return _loss(state["g"], state["logits"], state["ids"], c)
    return _linear(state, c) if c["op"] == "linear" else _linear_bwd(state, c)


def _run_own(s, c):
    from moe_variable_size_amd import api
    if c["op"] == "route":
        return api.moe_route_fwd(s["logits"], c["k"], score=c["score"], bias=s["bias"],
                                 groups=c["groups"], topk_groups=c["topk_groups"],
                                 group_score="max" if s["bias"] is None else "top2",
                                 renormalize=c["renorm"])
    if c["op"] == "route_bwd":
        return api.moe_route_bwd(s["g"], s["logits"], s["ids"], s["w"], score=c["score"],
                                 renormalize=c["renorm"])
    if c["op"] == "loss":
        losses, stats = api.moe_router_loss_fwd(s["logits"], s["ids"], score=c["score"])
        return losses, api.moe_router_loss_bwd(s["g"], s["logits"], stats, score=c["score"])
    if c["op"] == "linear":
        r = api.moe_linear_fwd(s["x"], s["W"], bias=s["bias"], act=c["act"], residual=s["residual"],
                               out_dtype=DTYPES[c["out"]], save_z=c["save"])
        return r if c["save"] else (r,)
    dx, dw, db = api.moe_linear_bwd(s["d_out"], s["x"], s["W"], act=c["act"], z=s["z"],
                                    dbias=c["bias"])
    return (dx, dw, db) if c["bias"] else (dx, dw)


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    c = case
    es = 4 if c["dtype"] == "f32" else 2
    if c["op"] in ("route", "route_bwd", "loss"):
        T, E, k = c["T"], c["E"], c["k"]
        if c["op"] == "route":
            return {"bytes": T * E * es + T * k * 8 + (4 * E if c["bias"] else 0), "flops": 4 * T * E}
        if c["op"] == "route_bwd":
            # the renormalised softmax needs no logits, the sigmoid only the chosen ones
            read = T * E if (c["score"] == "softmax" and not c["renorm"]) else \
                T * k if c["score"] == "sigmoid" else 0
            return {"bytes": (T * E + read) * es + T * k * 12, "flops": 6 * T * E}
        return {"bytes": 2 * T * E * es + T * k * 4, "flops": 16 * T * E}
    M, K, N = c["M"], c["K"], c["N"]
    os_ = 4 if c["out"] == "f32" else 2
    b = (M * K + N * K) * es + (N * es if c["bias"] else 0)
    if c["op"] == "linear":
        b += M * N * (os_ * (2 if c["residual"] else 1) + (es if c["save"] else 0))
        return {"bytes": b, "flops": 2 * M * N * K}
    b += (M * K + N * K) * es + M * N * (os_ + (es if c["act"] != "none" else 0))
    return {"bytes": b, "flops": 4 * M * N * K}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "route":
        l = s["logits"].double()
        prob = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
        # one row of comparison values per token; every expert outside the kept groups is out
        val = l.clone() if s["bias"] is None else prob + s["bias"].double()
        G = c["groups"]
        if G > 1:
            per = val.unflatten(1, (G, -1))
            gv = per.topk(2, dim=2).values.sum(2) if s["bias"] is not None else per.max(2).values
            rank = torch.argsort(torch.argsort(gv, dim=1, descending=True, stable=True), dim=1)
            per.masked_fill_((rank >= c["topk_groups"]).unsqueeze(2), -math.inf)
        # equal values: the lowest index first
        order = torch.argsort(val, dim=1, descending=True, stable=True)
        top = order[:, :c["k"]]
        w = prob.gather(1, top)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return None, w
    if c["op"] == "route_bwd":
        with torch.enable_grad():
            l = s["logits"].double().requires_grad_()
            prob = torch.softmax(l, 1) if c["score"] == "softmax" else torch.sigmoid(l)
            w = prob.gather(1, s["ids"].long())
            if c["renorm"]:
                w = w / w.sum(1, keepdim=True)
            return torch.autograd.grad((w * s["g"].double()).sum(), l)[0]
    if c["op"] == "loss":
        with torch.enable_grad():
            l = s["logits"].double().requires_grad_()
            E = c["E"]
            share = torch.zeros(E, dtype=torch.float64, device=l.device)
            share.index_add_(0, s["ids"].flatten().long(),
                             torch.ones(s["ids"].numel(), dtype=torch.float64, device=l.device))
            share = share / share.sum()
            if c["score"] == "softmax":
                q = torch.softmax(l, 1)
            else:
                q = torch.nn.functional.normalize(torch.sigmoid(l), p=1.0, dim=1)
            balance = E * torch.dot(share, q.mean(0))
            zloss = torch.logsumexp(l, 1).pow(2).mean()
            g = s["g"].double()
            d = torch.autograd.grad(g[0] * balance + g[1] * zloss, l)[0]
            return torch.stack([balance, zloss]).detach(), d
    F = torch.nn.functional
    acts = {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
            "gelu_tanh": lambda v: F.gelu(v, approximate="tanh")}
    x, W = s["x"].double(), s["W"].double()
    if c["op"] == "linear":
        z = F.linear(x, W, s["bias"].double() if s["bias"] is not None else None)
        out = acts[c["act"]](z)
        if s["residual"] is not None:
            out = out + s["residual"].double()
        return (out, z) if c["save"] else (out,)
    dz = s["d_out"].double()
    if s["z"] is not None:
        with torch.enable_grad():
            z = s["z"].double().requires_grad_()
            dz = torch.autograd.grad(acts[c["act"]](z), z, dz)[0]
    r = (torch.mm(dz, W), torch.mm(dz.t(), x))
    return r + (dz.sum(0),) if c["bias"] else r
