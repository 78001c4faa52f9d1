"""What a training step does after its gradients, in 64 bits, as plainly as the
definitions read (include/moe_block.h): the load-balance loss with its
gradient, the gradients' norm, AdamW.  Test infrastructure in numpy; it shares
no code with the library."""
import math

import numpy as np

from tests.block_ref import U, e4m3_values

BLOCK = 256     # elements that share a scale of an 8-bit state
TINY = 2.0 ** -126


def probabilities(logits, kind):
    """(s, logsumexp) per row, zeros for rows without a sum."""
    l = np.asarray(logits, np.float64)
    s, lse = np.zeros_like(l), np.zeros(len(l))
    for t, row in enumerate(l):
        top = row.max() if len(row) else -math.inf
        if top == -math.inf:
            continue
        with np.errstate(invalid="ignore", over="ignore"):
            e = np.exp(row - top)
            q = e if kind == "softmax" else 1.0 / (1.0 + np.exp(-row))
            s[t] = q / q.sum() if not q.sum() < TINY else 0.0
            lse[t] = top + np.log(e.sum())
    return s, lse


def bounds(offsets, T):
    return [0, T] if offsets is None else [int(v) for v in offsets]


def balance(logits, idx, kind, coef, z_coef, offsets=None):
    """(loss [3], counts [S,E], prob [S,E])."""
    T, E = logits.shape
    k, ends = idx.shape[1], bounds(offsets, logits.shape[0])
    S, N = len(ends) - 1, ends[-1] - ends[0]
    counts, prob = np.zeros((S, E), np.int64), np.zeros((S, E))
    bal = z = 0.0
    for i in range(S):
        rows = range(ends[i], ends[i + 1])
        if not len(rows):
            continue
        for t in rows:
            for e in {int(v) for v in idx[t] if 0 <= v < E}:
                counts[i, e] += 1
        s, lse = probabilities(logits[ends[i]: ends[i + 1]], kind)
        prob[i] = s.mean(axis=0)
        bal += len(rows) / N * E * (counts[i] / (k * len(rows)) * prob[i]).sum()
        if z_coef:
            z += (lse ** 2).sum() / N
    return np.array([coef * bal + z_coef * z, bal, z]), counts, prob


def balance_grad(logits, counts, k, kind, coef, z_coef, offsets=None, dloss=1.0, base=None):
    """(dlogits, a bound of an FP32 evaluation's error in it)."""
    T, E = logits.shape
    ends = bounds(offsets, T)
    N = ends[-1] - ends[0]
    out = np.zeros((T, E)) if base is None else np.array(base, np.float64)
    err = np.zeros((T, E))
    for i in range(len(ends) - 1):
        n = ends[i + 1] - ends[i]
        for t in range(ends[i], ends[i + 1]):
            l = np.asarray(logits[t], np.float64)
            a = dloss * coef * E * counts[i] / (k * n * N)
            s, lse = (v[0] for v in probabilities(logits[t: t + 1], kind))
            p = s if kind == "softmax" else probabilities(logits[t: t + 1], "softmax")[0][0]
            d = a - (a * s).sum()
            if kind == "sigmoid":
                q = 1.0 / (1.0 + np.exp(-np.where(l == -math.inf, -1000, l).clip(-700)))
                ds = s * (1.0 - q) * d
            else:
                ds = s * d
            zl = 2.0 * dloss * z_coef / N * lse * p
            rel = row_error(logits[t], E)
            err[t] = (2 * rel * s * (np.abs(a) + np.abs(a * s).sum()) + rel * np.abs(zl)
                      + abs(2.0 * dloss * z_coef / N) * p * rel * (1 + abs(lse)))
            out[t] += ds + zl
    return out, err + 4 * U * np.abs(out)


def row_error(row, E):
    """Relative error of an FP32 row's probabilities: expf's argument (its size
    times U) and result, the sum over the row, the reciprocals (a unit each),
    a few products."""
    l = np.asarray(row, np.float64)
    l = l[np.isfinite(l)]
    spread = 0.0 if not len(l) else (l.max() - l.min()) + np.abs(l).max()
    return (48 + E / 32 + 2 * spread) * U


def norm(grads, max_norm):
    n = math.sqrt(sum((g.astype(np.float64) ** 2).sum() for g in grads))
    return n, max_norm / n if n > max_norm else 1.0


# ------------------------------------------------------------------ AdamW
def adamw(w, g, m, v, step, lr, b1, b2, eps, decay):
    """(w, m, v) and bounds of an FP32 evaluation's error in them: the betas'
    own rounding and two products and a sum in each moment; root, sum,
    quotient and two factors in the step."""
    m2, v2 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    em = 5 * U * (np.abs(b1 * m) + np.abs((1 - b1) * g))
    ev = 6 * U * v2
    den = np.sqrt(v2 / (1 - b2 ** step)) + eps
    with np.errstate(invalid="ignore", divide="ignore"):
        up = m2 / (1 - b1 ** step) / den
        eu = em / (1 - b1 ** step) / den + 16 * U * np.abs(up)
    w2 = w - lr * decay * w - lr * up
    return w2, m2, v2, lr * eu + 3 * U * (np.abs(w) + np.abs(w2)), em, ev


_VALUES = np.sort(e4m3_values()[:127])  # 0 and the positive numbers


def to_codes(x):
    """The E4M3 numbers nearest to x / scale per block (ties to the even code),
    their scales, and how far x / scale is from a tie, relative to itself."""
    n = len(x)
    b = np.pad(x, (0, -n % BLOCK)).reshape(-1, BLOCK)
    scale = np.maximum(np.abs(b).max(axis=1) / 448.0, TINY)
    r = np.minimum(np.abs(b) / scale[:, None], 448.0)
    hi = np.searchsorted(_VALUES, r).clip(1, len(_VALUES) - 1)
    mid = (_VALUES[hi - 1] + _VALUES[hi]) / 2
    up = (r > mid) | ((r == mid) & (hi % 2 == 0))
    q = np.where(up, _VALUES[hi], _VALUES[hi - 1]) * np.sign(b)
    gap = np.abs(r - mid) / mid
    return q.reshape(-1)[:n], scale, gap.reshape(-1)[:n]


def from_codes(q, scale):
    return q * np.repeat(scale, BLOCK)[: len(q)]
