"""The block's operators in 64 bits, as plainly as their definitions read
(include/moe_block.h).  Test infrastructure: numpy and loops over tokens,
experts and groups; it shares no code with the library."""
import math

import numpy as np

U = 2.0 ** -24  # half a unit in the last place of FP32


def norm(x, residual, weight, eps):
    """(h, y) of float64 arrays."""
    h = x if residual is None else x + residual
    return h, h * weight / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)


def norm_grad(h, weight, dy, dres, eps):
    """(dh, dweight), and bounds of an FP32 evaluation's error in them."""
    T, H = h.shape
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    n, g = h * r, dy * weight
    dh = r * (g - n * (g * n).mean(axis=1, keepdims=True))
    # 16 sequential terms and 10 levels of a tree in each sum over H, the same
    # for the square root's argument, and a few roundings besides
    bound = 64 * U * r * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    if dres is not None:
        dh = dh + dres
        bound = bound + 2 * U * np.abs(dres)
    return dh, (dy * n).sum(axis=0), bound, (T + 100) * U * np.abs(dy * n).sum(axis=0)


def e4m3_values():
    """The value of every E4M3 code."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = (-1 if c & 128 else 1) * (math.nan if c & 127 == 127 else a)
    return v


def mx_values(codes, scales):
    """What MXFP8 rows stand for: codes uint8 [T,H], scales uint8 [T,>=H/32]."""
    T, H = codes.shape
    s = 2.0 ** (scales[:, : H // 32].astype(np.float64) - 127)
    return (e4m3_values()[codes].reshape(T, H // 32, 32) * s[..., None]).reshape(T, H)


def scores(logits, kind):
    l = logits.astype(np.float64)
    if kind == "sigmoid":
        return 1.0 / (1.0 + np.exp(-l))
    with np.errstate(invalid="ignore"):
        e = np.exp(l - l.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True)
    return np.where(np.isfinite(l.max(axis=1, keepdims=True)), s, 0.0)


def choice_values(logits, bias, kind):
    """What the choice goes by (float64; the logits themselves without a bias)."""
    l = logits.astype(np.float64)
    return l if bias is None else scores(logits, kind) + bias.astype(np.float64)


def group_ranks(c, groups, biased):
    v = c.reshape(c.shape[0], groups, -1)
    if not biased:
        return v.max(axis=2)
    top = -np.sort(-v, axis=2)[:, :, :2]
    return top.sum(axis=2)


def gate(logits, k, bias, kind, groups, topk_groups, renormalize, scale):
    """(idx, w): by repeated maximum, the lower index winning ties."""
    T, E = logits.shape
    c, s = choice_values(logits, bias, kind), scores(logits, kind)
    idx, w = np.zeros((T, k), np.int64), np.zeros((T, k))
    ranks = group_ranks(c, groups, bias is not None) if groups > 1 else None
    for t in range(T):
        open_ = set(range(E))
        if groups > 1:
            order = sorted(range(groups), key=lambda g: (-ranks[t, g], g))[:topk_groups]
            open_ = {e for e in range(E) if e // (E // groups) in order}
        for j in range(k):
            best = min(open_, key=lambda e: (-c[t, e], e))
            open_.remove(best)
            idx[t, j] = best
        p = s[t, idx[t]]
        w[t] = p
        if renormalize:
            w[t] = p / p.sum() if p.sum() != 0 else 0.0
    return idx, scale * w


def gate_gap(logits, bias, kind, groups):
    """Per token, the smallest distance between two values that the choice compares."""
    c = choice_values(logits, bias, kind)
    gap = np.diff(np.sort(c, axis=1), axis=1).min(axis=1)
    if groups > 1:
        r = group_ranks(c, groups, bias is not None)
        gap = np.minimum(gap, np.diff(np.sort(r, axis=1), axis=1).min(axis=1))
    return gap


def gate_grad(logits, idx, dw, kind, renormalize, scale):
    """dlogits; slots outside [0, E) or that repeat an earlier one count for nothing."""
    T, E = logits.shape
    s = scores(logits, kind)
    out = np.zeros((T, E))
    for t in range(T):
        used = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E and idx[t, j] not in idx[t, :j]]
        e, d = idx[t, used], scale * dw[t, used]
        p = s[t, e]
        P = p.sum()
        if renormalize:
            ds = (d - (d * p).sum() / P) / P if P != 0 else np.zeros_like(d)
        else:
            ds = d
        if kind == "sigmoid":
            out[t, e] = ds * p * (1 - p)
        else:
            full = np.zeros(E)
            full[e] = ds
            out[t] = s[t] * (full - (ds * p).sum())
    return out


def gate_grad_bound(logits, dw, kind, renormalize, scale):
    """An FP32 evaluation's error: the scores' (exp's argument, the sum over E
    in 32 lanes, a few roundings), relative to the largest terms of a row."""
    l = np.where(np.isfinite(logits), logits, 0).astype(np.float64)
    spread = (l.max(axis=1) - l.min(axis=1)) + np.abs(l).max(axis=1)
    rel = (64 + logits.shape[1] / 32 + dw.shape[1] + 2 * spread) * U
    size = np.abs(scale) * np.abs(dw).sum(axis=1)
    return (rel * size)[:, None]


def experts(x, idx, w, wgu, wd):
    """out [T,H]; slots outside [0, E) or that repeat an earlier one are dropped."""
    T, k = idx.shape
    E, H, I = wd.shape
    out = np.zeros((T, H))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E or e in idx[t, :j]:
                continue
            gu = wgu[e] @ x[t]
            g, u = gu[:I], gu[I:]
            out[t] += w[t, j] * (wd[e] @ (g / (1 + np.exp(-g)) * u))
    return out


def experts_grad(x, idx, w, wgu, wd, dout):
    """(dx, dw, dwgu, dwd) by the chain rule, one assignment at a time."""
    T, k = idx.shape
    E, H, I = wd.shape
    dx, dw, dwgu, dwd = np.zeros((T, H)), np.zeros((T, k)), np.zeros_like(wgu), np.zeros_like(wd)
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            if not 0 <= e < E or e in idx[t, :j]:
                continue
            gu = wgu[e] @ x[t]
            g, u = gu[:I], gu[I:]
            sg = 1 / (1 + np.exp(-g))
            a = g * sg * u
            q = wd[e].T @ dout[t]
            dw[t, j] = a @ q
            da = w[t, j] * q
            dgu = np.concatenate((da * u * sg * (1 + g * (1 - sg)), da * g * sg))
            dx[t] += wgu[e].T @ dgu
            dwgu[e] += np.outer(dgu, x[t])
            dwd[e] += np.outer(w[t, j] * dout[t], a)
    return dx, dw, dwgu, dwd


def orthogonalize(g, steps, coefficients, eps):
    """One matrix."""
    a, b, c = coefficients
    x = g / (np.sqrt((g * g).sum()) + eps)
    tall = x.shape[0] > x.shape[1]
    x = x.T if tall else x
    for _ in range(steps):
        m = x @ x.T
        x = a * x + (b * m + c * m @ m) @ x
    return x.T if tall else x


def rel(got, want):
    n = np.linalg.norm(want)
    d = np.linalg.norm(np.asarray(got, np.float64) - want)
    return d / n if n else d
