"""CPU oracle for the joins of a decoder layer (test infrastructure: only the
test suite may import it; it shares no code with the library).

The definitions in numpy float64: the residual's addition with the root-mean-square norm
and its block scales, the matrix product with its epilogue, and routing by scores.
"""
import math

import numpy as np

E4M3_MAX = 448.0


def add_norm(x, residual, weight, eps):
    """(s, y) of rows x [T, H]."""
    s = x.astype(np.float64) if residual is None else x.astype(np.float64) + residual.astype(np.float64)
    y = s / np.sqrt((s * s).mean(1, keepdims=True) + eps)
    return s, y if weight is None else y * weight.astype(np.float64)


def block_scale(amax, pow2):
    """Scale of blocks whose largest magnitude is amax."""
    amax = np.asarray(amax, np.float64)
    if not pow2:
        return np.where(amax > 0, amax / E4M3_MAX, 1.0)
    out = np.ones(amax.shape)
    for i, a in np.ndenumerate(amax):
        if a > 0:
            k = -126
            while 448.0 * 2.0 ** k < a:
                k += 1
            out[i] = 2.0 ** k
    return out


def activate(y, act):
    if act == "relu":
        return np.maximum(y, 0.0)
    if act == "silu":
        return y * 0.5 * (1 + np.tanh(y / 2))
    if act == "gelu":
        return np.array([0.5 * v * math.erfc(-v / math.sqrt(2)) for v in y.ravel()]).reshape(y.shape)
    if act == "gelu_tanh":
        return 0.5 * y * (1 + np.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def linear(x, w, bias, act, residual):
    """(out, the product with the bias, the sums of the products' magnitudes)."""
    x, w = x.astype(np.float64), w.astype(np.float64)
    y, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    out = activate(y, act)
    return (out if residual is None else out + residual), y, size


def scores(logits, score):
    """fp32 scores of rows of logits: one rounding of the float64 value."""
    l = np.array(logits, np.float64)
    l[np.isnan(l)] = -np.inf
    l = np.minimum(l, np.finfo(np.float32).max)
    if score == "sigmoid":
        return (1 / (1 + np.exp(-np.clip(l, -87, 87)))).astype(np.float32)
    out = np.zeros(l.shape, np.float32)
    for b, row in enumerate(l):
        if np.isneginf(row).all():
            continue
        e = np.array([math.exp(v - row.max()) if v - row.max() > -745 else 0.0 for v in row])
        out[b] = (e / math.fsum(e)).astype(np.float32)
    return out


def route_topk(logits, score, bias, n_group, topk_group, group_best, K, renorm, scale):
    """(ids, weights): selection by plain loops."""
    p = scores(logits, score)
    B, N = p.shape
    gs = N // n_group
    ids, w = np.zeros((B, K), np.int64), np.zeros((B, K))
    for b in range(B):
        c = p[b].copy()
        if bias is not None:
            with np.errstate(invalid="ignore"):
                c = c + np.asarray(bias, np.float32)
            c[np.isnan(c)] = -np.inf
        rank = []
        for g in range(n_group):
            best = sorted(c[g * gs:(g + 1) * gs], reverse=True)
            pair = group_best == 2 and gs > 1 and not (best[0] == np.inf and best[1] == -np.inf)
            rank.append(np.float32(best[0] + best[1]) if pair else best[0])
        kept = sorted(range(n_group), key=lambda g: (-rank[g], g))[:topk_group]
        cand = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
        ids[b] = sorted(cand, key=lambda e: (-c[e], e))[:K]
        chosen = p[b][ids[b]].astype(np.float64)
        if renorm:
            chosen = chosen / chosen.sum() if chosen.sum() > 0 else chosen * 0
        w[b] = chosen * scale
    return ids, w
