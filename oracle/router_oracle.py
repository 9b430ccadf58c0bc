"""Plain float64 forms of expert routing, the router losses and the dense linear
layer, straight from their formulas (loops over rows; small sizes).  Shares no
code with the HIP library."""
from __future__ import annotations

import math

import numpy as np


def _sigmoid(l):
    l = np.asarray(l, dtype=np.float64)
    e = np.exp(-np.abs(l))
    return np.where(l >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def softmax(l):
    l = np.asarray(l, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        e = np.where(l == -np.inf, 0.0, np.exp(l - np.max(l)))
        return e / e.sum()




def _better(a, b):
    """a, b = (value, index): a ranks before b."""
    na, nb = math.isnan(a[0]), math.isnan(b[0])
    if na != nb:
        return na
    if na or a[0] == b[0]:
        return a[1] < b[1]
    return a[0] > b[0]


def _ordered(pairs):
    out = []
    for p in pairs:
        i = 0
        while i < len(out) and _better(out[i], p):
            i += 1
        out.insert(i, p)
    return out


def route_row(l, k, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max",
              renormalize=True, scale=1.0):
    """(ids [k], weights [k]) of one row of logits."""
    l = np.asarray(l, dtype=np.float64)
    E = len(l)
    with np.errstate(all="ignore"):
        s = softmax(l) if score == "softmax" else _sigmoid(l)
    c = [float(l[e]) if bias is None else float(s[e] + np.float64(bias[e])) for e in range(E)]
    can = [l[e] != -np.inf and (bias is None or bias[e] != -np.inf) for e in range(E)]
    kept = range(groups)
    per = E // groups
    if groups > 1:
        vals = []
        for g in range(groups):
            src = c if (bias is not None or group_score == "max") else s
            mine = _ordered([(float(src[e]), e) for e in range(g * per, (g + 1) * per) if can[e]])
            if mine:
                v = mine[0][0]
                if group_score == "top2" and len(mine) > 1:
                    v = mine[0][0] + mine[1][0]
                vals.append((v, g))
        kept = [g for _, g in _ordered(vals)[:topk_groups]]
    best = _ordered([(c[e], e) for e in range(E) if can[e] and e // per in kept])[:k]
    ids = np.full(k, -1, dtype=np.int32)
    w = np.zeros(k)
    if best:
        chosen = [e for _, e in best]
        ids[:len(chosen)] = chosen
        if renormalize:
            # the ratios of the scores do not change with a common factor: take the largest out
            with np.errstate(all="ignore"):
                if score == "softmax":
                    p = np.exp(l[chosen] - np.max(l[chosen]))
                    if np.isnan(l).any():
                        p = p * np.nan
                else:
                    m = min(np.max(l[chosen]), 0.0)
                    p = np.exp(np.minimum(l[chosen], 0.0) - m) / (1.0 + np.exp(-np.abs(l[chosen])))
                p = p / p.sum()
        else:
            p = s[chosen]
        w[:len(chosen)] = scale * p
    return ids, w


def route(l, k, **opts):
    rows = [route_row(r, k, **opts) for r in np.asarray(l, dtype=np.float64)]
    return np.stack([r[0] for r in rows]), np.stack([r[1] for r in rows])


def route_grad(l, ids, g, score="softmax", renormalize=True, scale=1.0):
    """dL/dlogits of L = sum(g * weights) with the choice held fixed."""
    l = np.asarray(l, dtype=np.float64)
    d = np.zeros_like(l)
    for t in range(l.shape[0]):
        on = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < l.shape[1]]
        if not on:
            continue
        e = ids[t, on]
        s = softmax(l[t]) if score == "softmax" else _sigmoid(l[t])
        # dL/ds, then through the score
        if renormalize:
            P = s[e].sum()
            ds_c = scale / P * (g[t, on] - (g[t, on] * s[e]).sum() / P)
        else:
            ds_c = scale * g[t, on]
        ds = np.zeros(l.shape[1])
        np.add.at(ds, e, ds_c)
        d[t] = s * (ds - (ds * s).sum()) if score == "softmax" else ds * s * (1.0 - s)
    return d


def router_losses(l, ids, score="softmax"):
    """(balance, z, f, 1/V)."""
    l = np.asarray(l, dtype=np.float64)
    E = l.shape[1]
    c = np.zeros(E)
    for e in ids.ravel():
        if 0 <= e < E:
            c[e] += 1
    f = E * c / c.sum() if c.sum() else c
    rows = [r for r in l if not np.all(r == -np.inf)]
    if not rows:
        return 0.0, 0.0, f, 0.0
    P, z = np.zeros(E), 0.0
    for r in rows:
        s = softmax(r) if score == "softmax" else _sigmoid(r)
        P += s / s.sum()
        m = np.max(r)
        z += (m + math.log(np.exp(r - m).sum())) ** 2
    V = len(rows)
    return float((f * P).sum() / V), z / V, f, 1.0 / V


def router_losses_grad(l, ids, d_losses, score="softmax"):
    l = np.asarray(l, dtype=np.float64)
    _, _, f, inv = router_losses(l, ids, score)
    d = np.zeros_like(l)
    for t, r in enumerate(l):
        if np.all(r == -np.inf):
            continue
        p = softmax(r)
        s = p if score == "softmax" else _sigmoid(r)
        q = s / s.sum()
        b = q * (f - (f * q).sum())
        if score == "sigmoid":
            b = b * (1.0 - s)
        m = np.max(r)
        lse = m + math.log(np.exp(r - m).sum())
        d[t] = d_losses[0] * inv * b + 2.0 * d_losses[1] * inv * lse * p
    return d


_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return np.where(z > 0, z, 0.0)
    if kind == "gelu":
        return 0.5 * z * (1.0 + _erf(z / math.sqrt(2.0)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)))
    if kind == "silu":
        return z * _sigmoid(z)
    return z


def act_grad(z, kind):
    z = np.asarray(z, dtype=np.float64)
    if kind == "relu":
        return (z > 0).astype(np.float64)
    if kind == "gelu":
        return 0.5 * (1.0 + _erf(z / math.sqrt(2.0))) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        t = np.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)
    if kind == "silu":
        s = _sigmoid(z)
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def linear(x, W, bias=None, kind="none", residual=None):
    """(out, z)."""
    z = np.asarray(x, np.float64) @ np.asarray(W, np.float64).T
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    out = act(z, kind)
    return (out if residual is None else out + np.asarray(residual, np.float64)), z


def linear_grad(d_out, x, W, z, kind="none"):
    """(dX, dW, db) given the z the activation's derivative is taken at."""
    dz = np.asarray(d_out, np.float64) * (act_grad(z, kind) if kind != "none" else 1.0)
    return dz @ np.asarray(W, np.float64), dz.T @ np.asarray(x, np.float64), dz.sum(0)
