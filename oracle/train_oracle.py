"""CPU oracle, in 64 bits, of the linear cross entropy, the AdamW step and the
products with 4-bit weights, straight from their formulas.  numpy only; shares
no code with the library.
"""
import math

import numpy as np

# ---- linear cross entropy ---------------------------------------------------------------------


def linear_ce(x, W, targets, z_weight=0.0):
    """(loss [M], lse [M], {sum of loss, rows that count}) of logits x W^T."""
    l = x.astype(np.float64) @ W.astype(np.float64).T
    m = l.max(1)
    lse = m + np.log(np.exp(l - m[:, None]).sum(1))
    ok = (targets >= 0) & (targets < W.shape[0])
    at = np.where(ok, targets, 0)
    loss = np.where(ok, lse - l[np.arange(len(l)), at] + z_weight * lse ** 2, 0.0)
    return loss, lse, np.array([loss.sum(), ok.sum()])


def linear_ce_bwd(g, x, W, targets, z_weight=0.0):
    """(dX, dW, dl) of sum(g * loss)."""
    x, W = x.astype(np.float64), W.astype(np.float64)
    _, lse, _ = linear_ce(x, W, targets, z_weight)
    ok = (targets >= 0) & (targets < W.shape[0])
    d = np.exp(x @ W.T - lse[:, None]) * (np.where(ok, g, 0.0) * (1 + 2 * z_weight * lse))[:, None]
    for m in range(len(d)):
        if ok[m]:
            d[m, targets[m]] -= g[m]
    return d @ W, d.T @ x, d


# ---- AdamW ------------------------------------------------------------------------------------

BLOCK = 256


def adamw(w, g, m, v, t, lr, betas, eps, wd, s=1.0):
    b1, b2 = betas
    w, g, m, v = (np.asarray(a, np.float64) for a in (w, g, m, v))
    g = g * s
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    return w * (1 - lr * wd) - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps), m, v


def mix(h):
    h = ((h ^ (h >> 16)) * 0x6A09E667) & 0xFFFFFFFF
    h = ((h ^ (h >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
    return h ^ (h >> 16)


def dither(index, number, seed, t):
    """(u of m, u of sqrt v) of the elements ``index`` of a tensor."""
    index = np.asarray(index, np.uint64)
    out = np.zeros((2, len(index)))
    top = mix((seed + 0x9E3779B9 * t) & 0xFFFFFFFF)
    for hi in np.unique(index >> np.uint64(32)):
        at = (index >> np.uint64(32)) == hi
        key = mix((top + number + 0x9E3779B9 * int(hi)) & 0xFFFFFFFF)
        h = (index[at] & np.uint64(0xFFFFFFFF)) ^ np.uint64(key)
        h = ((h ^ (h >> np.uint64(16))) * np.uint64(0x6A09E667)) & np.uint64(0xFFFFFFFF)
        h = ((h ^ (h >> np.uint64(15))) * np.uint64(0xBB67AE85)) & np.uint64(0xFFFFFFFF)
        h = h ^ (h >> np.uint64(16))
        out[0, at] = (h & np.uint64(0xFFFF)).astype(float) / 65536 + 2.0 ** -17
        out[1, at] = (h >> np.uint64(16)).astype(float) / 65536 + 2.0 ** -17
    return out


def e4m3(codes):
    """The values of E4M3 codes."""
    c = np.asarray(codes).astype(np.int64)
    e, k = (c >> 3) & 15, c & 7
    v = np.where(e == 0, k / 8 * 2.0 ** -6, (1 + k / 8) * 2.0 ** (e - 7.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def unpack8(codes, scale):
    return e4m3(codes) * np.repeat(np.asarray(scale, np.float64), BLOCK)[:len(codes)]


def pack8(a, u):
    """(values over their scales, scales, distance of the rounding's place from the next whole number)."""
    n = len(a)
    rows = -(-n // BLOCK)
    b = np.zeros(rows * BLOCK)
    b[:n] = a
    b = b.reshape(rows, BLOCK)
    top = np.abs(b).max(1)
    scale = np.where(top >= 2.0 ** -100, top / 448.0, 0.0)
    y = np.abs(b) / np.where(scale > 0, scale, np.inf)[:, None]
    y = y.reshape(-1)[:n]
    d = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    k = y / d + u
    return np.sign(a) * np.minimum(np.floor(k) * d, 448.0), scale, np.abs(k - np.round(k)), d


# ---- 4-bit weights ----------------------------------------------------------------------------

def w4_place(k):
    """(byte of the row, shift) of reduction element k."""
    nib = {0: 0, 2: 1, 4: 2, 6: 3, 1: 4, 3: 5, 5: 6, 7: 7}[k % 8]
    return k // 128 * 64 + (k % 32 // 8) * 16 + (k % 128 // 32) * 4 + nib // 2, 4 * (nib % 2)


def w4_codes(codes, K):
    """codes [..., N, bytes] -> q [..., N, K]."""
    at = [w4_place(k) for k in range(K)]
    byte = np.array([a for a, _ in at])
    shift = np.array([s for _, s in at])
    return (codes[..., byte].astype(np.int64) >> shift) & 15


def w4_weight(codes, scales, zeros, N, K, group):
    """The weights [..., N, K] that codes, scales [..., groups, cols] and zeros (None: 8) stand for."""
    g = np.arange(K) // group
    s = np.swapaxes(np.asarray(scales, np.float64)[..., g, :N], -1, -2)
    z = 8.0 if zeros is None else np.swapaxes(np.asarray(zeros, np.float64)[..., g, :N], -1, -2)
    return (w4_codes(codes, K) - z) * s


def bf16(a):
    """Rounded to bf16, to nearest even."""
    u = np.asarray(a, np.float32).view(np.uint32).astype(np.uint64)
    u = (u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000
    return u.astype(np.uint32).view(np.float32)


def w4_quantize(W, group, symmetric):
    """(q [.., N, K], scales [.., N, groups], zeros [.., N, groups]) of W [.., N, K]."""
    W = np.asarray(W, np.float64)
    K = W.shape[-1]
    groups = -(-K // group)
    q = np.zeros(W.shape, np.int64)
    s = np.zeros(W.shape[:-1] + (groups,))
    z = np.full(s.shape, 8, np.int64)
    for j in range(groups):
        w = W[..., j * group:(j + 1) * group]
        if symmetric:
            sc = bf16(np.abs(w).max(-1) / 7).astype(np.float64)
        else:
            lo, hi = np.minimum(w.min(-1), 0), np.maximum(w.max(-1), 0)
            sc = bf16((hi - lo) / 15).astype(np.float64)
        inv = np.where(sc > 0, 1 / np.where(sc > 0, sc, 1), 0)
        if not symmetric:
            z[..., j] = np.clip(np.rint(-lo * inv), 0, 15)
        s[..., j] = sc
        q[..., j * group:(j + 1) * group] = np.clip(np.rint(w * inv[..., None]) + z[..., j][..., None], 0, 15)
    return q, s, z
