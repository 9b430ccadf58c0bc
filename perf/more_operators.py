"""Timed cases of the linear cross entropy, the AdamW step and the products with 4-bit weights.

Each case is one call (or a loss with its gradients) as a program that trains
or serves a model makes it.  run() computes it in plain torch, or, with ``own``
set, through the library.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 256  # elements that share one scale of an 8-bit state
LEAST = 2.0 ** -100  # a block whose largest value is below holds zeros


def listed():
    return [
        # the score of one token over the vocabulary
        {"name": "ce 1 token", "op": "ce", "M": 1, "K": 4096, "V": 32000, "z": 0.0, "grad": False,
         "dtype": "bf16"},
        # an evaluation batch, a vocabulary of odd size
        {"name": "ce eval", "op": "ce", "M": 2048, "K": 4096, "V": 50257, "z": 0.0, "grad": False,
         "dtype": "bf16"},
        # the loss of a training batch and its gradients, with a z term
        {"name": "ce train", "op": "ce", "M": 8192, "K": 4096, "V": 65536, "z": 1e-4, "grad": True,
         "dtype": "bf16"},
        # a small fp32 model, every size odd
        {"name": "ce train f32 odd", "op": "ce", "M": 777, "K": 1001, "V": 5003, "z": 0.0, "grad": True,
         "dtype": "f32"},
        # a router's and a few small layers' weights
        {"name": "adamw small", "op": "adamw", "sizes": "131072,64,131072,64,65536,256,65536,256,1000,1,77,4097",
         "dtype": "f32", "gdtype": "f32", "master": False, "bits": 32, "wd": 0.1},
        # a model's many tensors in bf16 with fp32 master weights, gradients in fp32
        {"name": "adamw many", "op": "adamw", "sizes": ",".join(["1048576,1024,524288,2048,1441793,4096,262145,7"] * 12),
         "dtype": "bf16", "gdtype": "f32", "master": True, "bits": 32, "wd": 0.1},
        # the weights of 64 gated experts, bf16, states in fp32
        {"name": "adamw experts", "op": "adamw", "sizes": "184549376,92274688", "dtype": "bf16", "gdtype": "bf16",
         "master": False, "bits": 32, "wd": 0.1},
        # the same with states in 8 bits
        {"name": "adamw experts 8 bits", "op": "adamw", "sizes": "184549376,92274688", "dtype": "bf16",
         "gdtype": "bf16", "master": False, "bits": 8, "wd": 0.1},
        # one token through a dense projection
        {"name": "w4 1 token", "op": "w4", "M": 1, "K": 4096, "N": 4096, "group": 128, "zeros": True,
         "act": "none", "bias": False, "residual": False, "out": "bf16"},
        # a small batch through a wide projection, added to the routed output
        {"name": "w4 16 tokens", "op": "w4", "M": 16, "K": 8192, "N": 8192, "group": 128, "zeros": False,
         "act": "silu", "bias": True, "residual": True, "out": "f32"},
        # one token through its 8 experts
        {"name": "w4 experts 1 token", "op": "w4_experts", "T": 1, "k": 8, "E": 64, "K": 7168, "N": 2048, "group": 128,
         "zeros": True},
        # a decode batch through its experts
        {"name": "w4 experts decode", "op": "w4_experts", "T": 128, "k": 8, "E": 64, "K": 7168, "N": 2048, "group": 32,
         "zeros": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce", "ce", "adamw", "adamw", "w4", "w4_experts"])
    if op == "ce":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        K = _log_int(rng, 64, 8192)
        if rng.random() < 0.7:  # most models' widths are multiples of 8
            K = (K + 7) // 8 * 8
        V = _log_int(rng, 500, 131072)
        M = _log_int(rng, 1, max(1, min(8192, (1 << (39 if dtype == "bf16" else 35)) // (K * V))))
        return {"op": "ce", "M": M, "K": K, "V": V, "z": rng.choice([0.0, 1e-4]), "grad": rng.random() < 0.6,
                "dtype": dtype}
    if op == "adamw":
        dtype, bits = rng.choice(["f32", "bf16"]), rng.choice([32, 8])
        total, left = _log_int(rng, 1000, 1 << 27), rng.randint(1, 100)
        sizes = []
        while total > 0 and left > 0:
            n = total if left == 1 else _log_int(rng, 1, total)
            sizes.append(n)
            total, left = total - n, left - 1
        return {"op": "adamw", "sizes": ",".join(map(str, sizes)), "dtype": dtype,
                "gdtype": rng.choice(["f32", "bf16"]), "master": dtype == "bf16" and rng.random() < 0.5, "bits": bits,
                "wd": rng.choice([0.0, 0.1])}
    K = _log_int(rng, 32, 1280) * 8
    c = {"op": op, "K": K, "group": rng.choice([32, 64, 128]), "zeros": rng.random() < 0.5}
    if op == "w4":
        N = _log_int(rng, 16, 16384)
        c.update(M=_log_int(rng, 1, 64), N=N, act=rng.choice(["none", "relu", "gelu", "silu"]),
                 bias=rng.random() < 0.5, residual=rng.random() < 0.5, out=rng.choice(["bf16", "f32"]))
        return c
    E = _log_int(rng, 4, 128)
    N = _log_int(rng, 16, max(16, min(8192, (1 << 30) // (E * K))))
    c.update(E=E, N=N, k=rng.randint(1, min(8, E)), T=_log_int(rng, 1, 128))
    return c


# ---- the plain forms ---------------------------------------------------------------------------

def _ce(s, c):
    x, W = s["x"].float(), s["W"].float()
    M, V = x.shape[0], W.shape[0]
    t = s["targets"].long()
    counts = (t >= 0) & (t < V)
    at = torch.where(counts, t, torch.zeros_like(t))[:, None]
    logits = x @ W.t()
    m = logits.amax(1, keepdim=True)
    e = torch.exp(logits - m)
    total = e.sum(1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    zero = torch.zeros_like(lse)
    loss = torch.where(counts, lse - torch.gather(logits, 1, at)[:, 0] + c["z"] * lse * lse, zero)
    if not c["grad"]:
        return loss, lse
    g = torch.where(counts, s["g"], zero)
    d = e * ((g * (1.0 + 2.0 * c["z"] * lse))[:, None] / total)
    d.scatter_add_(1, at, -g[:, None])
    return loss, (d @ W).to(s["x"].dtype), (d.t() @ x).to(s["W"].dtype)


def _mix(h):
    """A 32-bit hash, held in 64-bit integers."""
    low = 0xFFFFFFFF
    h = ((h ^ (h >> 16)) * 0x6A09E667) & low
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & low
    return h ^ (h >> 16)


def _dither(sizes, seed, t, device):
    """Two uniform numbers, of 16 bits and a half, for every element of tensors that lie in whole blocks behind each other."""
    n = torch.tensor([-(-int(v) // BLOCK) * BLOCK for v in sizes.split(",")], device=device)
    keys = _mix((_mix((seed + 0x9E3779B9 * t) & 0xFFFFFFFF) + torch.arange(n.numel(), device=device)) & 0xFFFFFFFF)
    index = torch.arange(int(n.sum()), device=device) - torch.repeat_interleave(n.cumsum(0) - n, n)
    h = _mix(index ^ torch.repeat_interleave(keys, n))
    return ((h & 0xFFFF).float() + 0.5) * 2.0 ** -16, ((h >> 16).float() + 0.5) * 2.0 ** -16


def _pack8(a, u):
    """E4M3 codes and scales of whole blocks, rounded up where u says so."""
    b = a.view(-1, BLOCK)
    top = b.abs().amax(1, keepdim=True)
    some = top >= LEAST
    inv = torch.where(some, 448.0 / torch.where(some, top, torch.ones_like(top)), torch.zeros_like(top))
    y = b.abs() * inv
    e = torch.frexp(y)[1] - 1
    e = torch.where(y > 0, e, -6).clamp(min=-6)
    k = torch.floor(torch.ldexp(y, 3 - e) + u.view(-1, BLOCK))
    v = torch.ldexp(k, e - 3).clamp(max=448.0) * torch.sign(b)
    scale = torch.where(some, top / 448.0, torch.zeros_like(top))
    return v.view(-1).to(torch.float8_e4m3fn), scale[:, 0]


def _unpack8(q, scale):
    return (q.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s, c):
    """All tensors at once: they lie in one buffer, with zeros between them, and zeros stay zeros."""
    s["t"] += 1
    t, f = s["t"], s["flat"]
    eight = c["bits"] == 8
    if eight:
        m, r = _unpack8(f["m"], f["m_scale"]), _unpack8(f["v"], f["v_scale"])
        v = r * r
    else:
        m, v = f["m"], f["v"]
    b1, b2 = s["betas"]
    g = s["grad"].float() * s["grad_scale"]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * g * g
    w = f["master"] if c["master"] else f["p"].float()
    step = (m / (1.0 - b1 ** t)) / (torch.sqrt(v / (1.0 - b2 ** t)) + s["eps"])
    w = w * (1.0 - s["lr"] * c["wd"]) - s["lr"] * step
    f["p"].copy_(w)
    if c["master"]:
        f["master"].copy_(w)
    if eight:
        um, ur = _dither(c["sizes"], s["seed"], t, w.device)
        (q, scale), (qr, rscale) = _pack8(m, um), _pack8(torch.sqrt(v), ur)
        for key, a in (("m", q), ("m_scale", scale), ("v", qr), ("v_scale", rscale)):
            f[key].copy_(a)
    else:
        f["m"].copy_(m)
        f["v"].copy_(v)
    return f


def _unpack4(codes):
    """[..., N, bytes] -> [..., N, 2 * bytes] values 0..15.  16 bytes (four 32-bit words of eight codes each)
    for each quarter of 128 elements; word j of quarter q holds elements 32 j + 8 q + (0, 2, 4, 6, 1, 3, 5, 7)."""
    lead = codes.shape[:-1]
    v = torch.stack([codes & 15, codes >> 4], -1)
    v = v.view(*lead, -1, 4, 4, 2, 4)  # block, quarter, word, odd?, pair
    v = v.movedim(-4, -3).transpose(-1, -2)  # block, word, quarter, pair, odd?
    return v.reshape(*lead, -1)


def _dequant(codes, scales, zeros, N, K, group):
    q = _unpack4(codes)[..., :K].float()
    s = scales[..., :N].float().transpose(-1, -2).repeat_interleave(group, -1)[..., :K]
    z = 8.0 if zeros is None else zeros[..., :N].float().transpose(-1, -2).repeat_interleave(group, -1)[..., :K]
    return (q - z) * s


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _w4(s, c):
    z = s["x"].float() @ _dequant(s["codes"], s["scales"], s["zeros"], c["N"], c["K"], c["group"]).t()
    if s["bias"] is not None:
        z = z + s["bias"].float()
    z = _act(z, c["act"])
    if s["residual"] is not None:
        z = z + s["residual"].float()
    return z.to(DTYPES[c["out"]])


def _w4_experts(s, c):
    T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
    x, ids, zeros = s["x"].float(), s["ids"].long(), s["zeros"]
    if T * k <= E:  # the chosen experts alone
        i = ids.reshape(-1)
        W = _dequant(s["codes"][i], s["scales"][i], None if zeros is None else zeros[i], N, K, c["group"])
        each = (W @ x.repeat_interleave(k, 0)[:, :, None]).view(T, k, N)
    else:  # every expert's product, of which k are taken
        W = _dequant(s["codes"], s["scales"], zeros, N, K, c["group"])
        each = (x @ W.view(E * N, K).t()).view(T, E, N)
        each = torch.gather(each, 1, ids[:, :, None].expand(T, k, N))
    return (each * s["w"][:, :, None]).sum(1)


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(int(seed))

    def randn(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device=dev, dtype=dtype) * std

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    def whole(lo, hi, *shape, dtype=torch.int64):
        return torch.randint(lo, hi, shape, generator=gen, device=dev, dtype=dtype)

    s = {"case": c}
    if c["op"] == "ce":
        M, K, V = c["M"], c["K"], c["V"]
        dt = DTYPES[c["dtype"]]
        s["x"] = randn(M, K, dtype=dt)
        s["W"] = randn(V, K, std=1.5 / math.sqrt(K), dtype=dt)
        t = whole(0, V, M)
        if M > 8:  # a prompt's and the padding's tokens do not count
            t = torch.where(rand(M) < 0.1, torch.full_like(t, -100), t)
        s["targets"] = t
        s["g"] = torch.full((M,), 1.0 / M, device=dev)
        return s
    if c["op"] == "adamw":
        sizes = [int(n) for n in c["sizes"].split(",")]
        at, starts = 0, []
        for n in sizes:
            starts.append(at)
            at += -(-n // BLOCK) * BLOCK

        def parts(flat, per=1):
            return [flat[a // per:a // per + -(-n // per)] for a, n in zip(starts, sizes)]

        keep = torch.zeros(at, device=dev)
        for a in parts(keep):
            a.fill_(1.0)
        w = randn(at, std=0.02) * keep
        flat = {"p": w.to(DTYPES[c["dtype"]])}
        s["params"] = parts(flat["p"])
        if c["master"]:
            flat["master"] = w
            s["masters"] = parts(w)
        s["grad"] = (randn(at, std=1e-3) * keep).to(DTYPES[c["gdtype"]])
        s["grads"] = parts(s["grad"])
        # states in the course of training: m about a third of sqrt(v)
        m, v = randn(at, std=3e-4) * keep, (1e-3 * (0.25 + rand(at)) * keep) ** 2
        if c["bits"] == 8:
            flat["m"], flat["m_scale"] = _pack8(m, torch.full_like(m, 0.5))
            flat["v"], flat["v_scale"] = _pack8(torch.sqrt(v), torch.full_like(v, 0.5))
            s["m_scale"], s["v_scale"] = parts(flat["m_scale"], BLOCK), parts(flat["v_scale"], BLOCK)
        else:
            flat["m"], flat["v"] = m, v
        s["m"], s["v"] = parts(flat["m"]), parts(flat["v"])
        s.update(flat=flat, t=100, lr=1e-4, betas=(0.9, 0.95), eps=1e-8, seed=int(seed) & 0xFFFFFFFF,
                 grad_scale=torch.full((1,), 0.75, device=dev))
        return s
    K, N, group = c["K"], c["N"], c["group"]
    lead = (c["E"],) if c["op"] == "w4_experts" else ()
    groups, cols = -(-K // group), -(-N // 16) * 16
    s["codes"] = whole(0, 256, *lead, N, -(-K // 128) * 64, dtype=torch.uint8)
    # weights of about 1 / sqrt(K)
    s["scales"] = ((0.5 + rand(*lead, groups, cols)) / (4.6 * math.sqrt(K))).to(torch.bfloat16)
    s["zeros"] = whole(6, 10, *lead, groups, cols, dtype=torch.uint8) if c["zeros"] else None
    if c["op"] == "w4":
        M = c["M"]
        s["x"] = randn(M, K, dtype=torch.bfloat16)
        s["bias"] = randn(N, std=0.2, dtype=torch.bfloat16) if c["bias"] else None
        s["residual"] = randn(M, N, dtype=DTYPES[c["out"]]) if c["residual"] else None
        return s
    T, k, E = c["T"], c["k"], c["E"]
    s["x"] = randn(T, K, dtype=torch.bfloat16)
    s["ids"] = torch.sort(rand(T, E), dim=1)[1][:, :k].int().contiguous()
    w = rand(T, k) + 0.1
    s["w"] = w / w.sum(1, keepdim=True)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return _run_own(state, c)
    return {"ce": _ce, "adamw": _adamw, "w4": _w4, "w4_experts": _w4_experts}[c["op"]](state, c)


def _run_own(s, c):
    from moe_variable_size_amd import api
    if c["op"] == "ce":
        loss, lse = api.moe_linear_ce_fwd(s["x"], s["W"], s["targets"], z_weight=c["z"])
        if not c["grad"]:
            return loss, lse
        return (loss,) + api.moe_linear_ce_bwd(s["g"], s["x"], s["W"], s["targets"], lse, z_weight=c["z"])
    if c["op"] == "adamw":
        s["t"] += 1
        api.moe_adamw_step(s["params"], s["grads"], s["m"], s["v"], step=s["t"], lr=s["lr"], betas=s["betas"],
                           eps=s["eps"], weight_decay=c["wd"], masters=s.get("masters"), m_scales=s.get("m_scale"),
                           v_scales=s.get("v_scale"), grad_scale=s["grad_scale"], seed=s["seed"])
        return s["flat"]
    W = api.W4Weight(s["codes"], s["scales"], s["zeros"], c["N"], c["K"], c["group"])
    if c["op"] == "w4":
        return api.moe_linear_w4_fwd(s["x"], W, bias=s["bias"], act=c["act"], residual=s["residual"],
                                     out_dtype=DTYPES[c["out"]])
    if c["T"] * c["k"] <= c["E"]:
        return api.moe_token_fwd_w4(s["x"], W, s["ids"], s["w"])
    return api.moe_fused_fwd_w4(s["x"], W, api.moe_build_schedule(s["ids"], s["w"], c["E"]))


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "ce":
        M, K, V = c["M"], c["K"], c["V"]
        es = 4 if c["dtype"] == "f32" else 2
        once = (M * K + V * K) * es
        if not c["grad"]:
            return {"bytes": once + 16 * M, "flops": 2 * M * K * V}
        # no logits are kept: they are computed in the forward and again in the backward
        return {"bytes": 2 * once + 24 * M, "flops": 8 * M * K * V}
    if c["op"] == "adamw":
        n = sum(int(v) for v in c["sizes"].split(","))
        ps, gs = (4 if c["dtype"] == "f32" else 2), (4 if c["gdtype"] == "f32" else 2)
        weights = ps + 8 if c["master"] else 2 * ps
        states = 16 if c["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": int(n * (weights + gs + states)), "flops": 15 * n}
    K, N = c["K"], c["N"]
    per = N * K // 2 + N * -(-K // c["group"]) * (3 if c["zeros"] else 2)
    if c["op"] == "w4":
        M, es = c["M"], 4 if c["out"] == "f32" else 2
        return {"bytes": per + 2 * M * K + (2 * N if c["bias"] else 0) + M * N * es * (2 if c["residual"] else 1),
                "flops": 2 * M * N * K}
    T, k, E = c["T"], c["k"], c["E"]
    used = E * (1.0 - (1.0 - k / E) ** T)  # experts that are expected to have a token
    return {"bytes": int(used * per) + 2 * T * K + 4 * T * N + 8 * T * k, "flops": 2 * T * k * N * K}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    f64 = torch.float64
    if c["op"] == "ce":
        x, W, t = s["x"].to(f64), s["W"].to(f64), s["targets"]
        logp = torch.mm(x, W.t())
        lse = torch.logsumexp(logp, 1)
        keep = t.ge(0).logical_and(t.lt(W.shape[0]))
        rows = keep.nonzero()[:, 0]
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - logp[rows, t[rows]] + c["z"] * lse[rows].square()
        if not c["grad"]:
            return loss, lse
        g = s["g"].to(f64) * keep
        d = logp.sub_(lse[:, None]).exp_().mul_((g + 2 * c["z"] * g * lse)[:, None])
        d[rows, t[rows]] -= g[rows]
        return loss, torch.mm(d, W), torch.mm(d.t(), x)
    if c["op"] == "adamw":
        flat = s["flat"]
        b1, b2 = s["betas"]
        t = s["t"] + 1
        out = {k: torch.zeros_like(a, dtype=f64) for k, a in flat.items()}
        at = 0
        for i, n in enumerate(int(v) for v in c["sizes"].split(",")):
            blocks = -(-n // BLOCK)
            span = slice(at, at + blocks * BLOCK)
            rows = slice(at // BLOCK, at // BLOCK + blocks)
            at += blocks * BLOCK
            m, v = flat["m"][span].to(f64), flat["v"][span].to(f64)
            if c["bits"] == 8:
                m = (m.view(blocks, BLOCK) * flat["m_scale"][rows, None].to(f64)).view(-1)
                v = (v.view(blocks, BLOCK) * flat["v_scale"][rows, None].to(f64)).view(-1).square()
            # behind a tensor's end nothing changes
            tail = torch.arange(blocks * BLOCK, device=m.device) >= n
            g = torch.zeros_like(m)
            g[:n] = s["grads"][i].to(f64) * 0.75
            m1 = torch.lerp(g, m, b1)
            v1 = torch.lerp(g.square(), v, b2)
            w0 = flat["master" if c["master"] else "p"][span].to(f64)
            hat = (m1 / -math.expm1(t * math.log(b1))) / ((v1 / -math.expm1(t * math.log(b2))).sqrt() + s["eps"])
            w1 = torch.where(tail, w0, w0 - s["lr"] * (hat + c["wd"] * w0))
            out["p"][span] = torch.where(tail, flat["p"][span].to(f64), w1)
            if c["master"]:
                out["master"][span] = w1
            if c["bits"] == 32:
                out["m"][span] = torch.where(tail, m, m1)
                out["v"][span] = torch.where(tail, v, v1)
                continue
            index = torch.arange(blocks * BLOCK, device=m.device)
            low = (1 << 32) - 1

            def stir(a):
                for shift, by in ((16, 0x6A09E667), (15, 0xBB67AE85)):
                    a = (a ^ (a >> shift)) * by & low
                return a ^ (a >> 16)

            h = stir(index ^ stir((stir((s["seed"] + 0x9E3779B9 * t) & low) + i) & low))
            for key, a, bits in (("m", m1, h & 0xFFFF), ("v", v1.sqrt(), h >> 16)):
                a = torch.where(tail, torch.zeros_like(a), a).view(blocks, BLOCK)
                scale = a.abs().max(1).values / 448.0
                q = a.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
                # the step between neighbours: an eighth of the power of two below, 2^-9 at least
                step = torch.exp2(torch.floor(torch.log2(q.clamp(min=2.0 ** -6))) - 3)
                q = (torch.floor(q / step + (2 * bits.view(blocks, BLOCK).to(f64) + 1) / 131072) * step).clamp(max=448.0)
                q = (q * a.sign()).view(-1)
                out[key][span] = torch.where(tail, flat[key][span].to(f64), q)
                out[key + "_scale"][rows] = scale
        return out
    K, N, group = c["K"], c["N"], c["group"]

    def weight(codes, scales, zeros):
        # element by element: where its code lies, and its group
        k = torch.arange(K, device=codes.device)
        place = {0: 0, 2: 1, 4: 2, 6: 3, 1: 4, 3: 5, 5: 6, 7: 7}
        nib = torch.tensor([place[e] for e in range(8)], device=codes.device)[k % 8]
        byte = k // 128 * 64 + k % 32 // 8 * 16 + k % 128 // 32 * 4 + nib // 2
        q = (codes.index_select(1, byte).int() >> (4 * (nib % 2)).int()).bitwise_and(15).to(f64)
        z = 8.0 if zeros is None else zeros.to(f64)[k // group, :N].t()
        return (q - z) * scales.to(f64)[k // group, :N].t()

    x = s["x"].to(f64)
    if c["op"] == "w4":
        z = torch.mm(x, weight(s["codes"], s["scales"], s["zeros"]).t())
        if s["bias"] is not None:
            z += s["bias"].to(f64)
        F = torch.nn.functional
        z = {"none": lambda v: v, "relu": F.relu, "gelu": F.gelu, "silu": F.silu}[c["act"]](z)
        return z if s["residual"] is None else z + s["residual"].to(f64)
    y = torch.zeros((c["T"], N), dtype=f64, device=x.device)
    for e in range(c["E"]):
        t, j = (s["ids"] == e).nonzero(as_tuple=True)
        if t.numel():
            W = weight(s["codes"][e], s["scales"][e], None if s["zeros"] is None else s["zeros"][e])
            y.index_add_(0, t, torch.mm(x[t], W.t()) * s["w"][t, j].to(f64)[:, None])
    return y
