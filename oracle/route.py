"""Float64 references of the routing to experts, the order of their rows and the movement of rows (test infrastructure).

Token by token and slot by slot in float64; no code shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np

SOFTMAX, SIGMOID = 0, 1
FLT_MAX = float(np.finfo(np.float32).max)


def scores(x, kind):
    """The scores of one row of logits; 0 where a logit is -infinity or NaN."""
    x = np.asarray(x, dtype=np.float64)
    live = x > -np.inf
    x = np.where(live, np.minimum(x, FLT_MAX), 0.0)
    s = np.zeros(x.shape)
    if kind == SIGMOID:
        e = np.exp(-np.abs(x))
        s = np.where(x >= 0, 1 / (1 + e), e / (1 + e))
    elif live.any():
        with np.errstate(over="ignore"):  # (values that are not live are left out below)
            s = np.exp(np.clip(x - x[live].max(), -1500.0, 0.0))
        s = s / s[live].sum()
    return np.where(live, s, 0.0)


def weights_of(x, chosen, kind, renormalise, scale):
    """Weights of the chosen experts of one row, the proportions of very small scores kept."""
    if len(chosen) == 0:
        return np.zeros(0)
    x = np.minimum(np.asarray(x, dtype=np.float64), FLT_MAX)
    if not renormalise:
        return scale * scores(x, kind)[chosen]
    xs = x[chosen]
    log = xs if kind == SOFTMAX else np.minimum(xs, 0) - np.log1p(np.exp(-np.abs(xs)))
    e = np.exp(log - log.max())
    return scale * e / e.sum()


def route_reference(logits, top, kind, bias=None, groups=1, top_groups=1, group_sum=1, renormalise=True, scale=1.0):
    T, E = logits.shape
    expert, weight = np.full((T, top), -1, dtype=np.int64), np.zeros((T, top))
    by_logit = bias is None and (groups == 1 or group_sum == 1)
    for t in range(T):
        x = logits[t].astype(np.float64)
        sel = np.minimum(x, FLT_MAX) if by_logit else scores(x, kind) + (0 if bias is None else bias.astype(np.float64))
        sel = np.where((x > -np.inf) & (sel > -np.inf), sel, -np.inf)
        if groups > 1:
            size = E // groups
            worth = []
            for h in range(groups):
                best = sorted((v for v in sel[h * size:(h + 1) * size] if v > -np.inf), reverse=True)[:group_sum]
                worth.append(sum(best) if best else -np.inf)
            kept = sorted(range(groups), key=lambda h: (-worth[h], h))[:top_groups]
            for h in range(groups):
                if h not in kept:
                    sel[h * size:(h + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-sel[e], e)) if sel[e] > -np.inf][:top]
        expert[t, :len(order)] = order
        weight[t, :len(order)] = weights_of(x, order, kind, renormalise, scale)
    return expert, weight


def route_grad_reference(logits, expert, dweight, kind, renormalise, scale):
    """dlogits and, element by element, the sum of absolute terms behind it."""
    T, E = logits.shape
    dx, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        x = logits[t].astype(np.float64)
        slots = [s for s in range(expert.shape[1]) if 0 <= expert[t, s] < E]
        chosen = expert[t, slots].astype(int)
        g = scale * dweight[t, slots].astype(np.float64)
        s = scores(x, kind)
        w = weights_of(x, chosen, kind, renormalise, 1.0)
        w = np.where(np.asarray(x[chosen]) > -np.inf, w, 0.0)
        slope = 1 - s[chosen] if kind == SIGMOID else np.ones(len(chosen))
        if kind == SIGMOID:
            xs = x[chosen]
            slope = np.where(xs > 0, np.exp(-np.abs(xs)), 1.0) / (1 + np.exp(-np.abs(xs)))
        mean, spread = float((g * w).sum()), float(np.abs(g * w).sum())
        for i, e in enumerate(chosen):
            dx[t, e] += slope[i] * w[i] * (g[i] - (mean if renormalise else 0.0))
            size[t, e] += slope[i] * w[i] * (abs(g[i]) + (spread if renormalise else 0.0))
        if kind == SOFTMAX and not renormalise:
            dx[t] -= s * mean
            size[t] += s * spread
    return dx, size


def rows_reference(expert, E):
    """offsets, row, source by a walk over the experts."""
    flat = expert.reshape(-1)
    offsets, row, source = [0], np.full(flat.size, -1), []
    for e in range(E):
        for p in np.flatnonzero(flat == e):
            row[p] = len(source)
            source.append(p)
        offsets.append(len(source))
    return np.array(offsets), row.reshape(expert.shape), np.array(source + [-1] * (flat.size - len(source)))


def combine_reference(Y, row, weight=None, beta=0.0, out=None):
    """Out and the sum of absolute terms behind each element."""
    T, top = row.shape
    y, size = np.zeros((T, Y.shape[1])), np.zeros((T, Y.shape[1]))
    for t in range(T):
        for s in range(top):
            if 0 <= row[t, s] < Y.shape[0]:
                term = (1.0 if weight is None else float(weight[t, s])) * Y[row[t, s]]
                y[t] += term
                size[t] += np.abs(term)
    if beta != 0.0:
        y, size = y + beta * out, size + np.abs(beta * out)
    return y, size
