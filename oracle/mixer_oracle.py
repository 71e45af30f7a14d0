"""fp64 restatement of the routing with scores and groups, the residual norm, the causal convolution and the
selective scan (test infrastructure only): straightforward loops over tokens, experts or taps."""
from __future__ import annotations

import numpy as np


def sigmoid(x):
    with np.errstate(over="ignore"):
        return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))


# ------------------------------------------------------------------ routing

def scores(logits, kind):
    l = np.where(np.isfinite(logits), logits, -np.inf)
    if kind == "sigmoid":
        return sigmoid(l)
    top = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isfinite(top), top, 0.0))
    total = e.sum(1, keepdims=True)
    return e / np.where(total > 0, total, 1.0)


def route(logits, bias, k, kind="sigmoid", groups=1, group_k=None, group_top=2, renorm=True, scale=1.0):
    """(idx, w, s) as moe_route_scores defines them."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    group_k = groups if group_k is None else group_k
    s = scores(logits, kind)
    out = ~np.isfinite(logits)
    c = s.copy()
    if bias is not None:
        b = np.asarray(bias, dtype=np.float64)
        out = out | ~np.isfinite(b)
        c = s + np.where(np.isfinite(b), b, 0.0)
    order_by = np.where(out, -np.inf, logits if bias is None else c)
    idx = np.empty((T, k), dtype=np.int32)
    size = E // groups
    for t in range(T):
        allowed = np.ones(E, dtype=bool)
        if group_k < groups:
            value = np.full(groups, -np.inf)
            for g in range(groups):
                part = [c[t, e] if (bias is not None or group_top > 1) else logits[t, e]
                        for e in range(g * size, (g + 1) * size) if not out[t, e]]
                if part:
                    value[g] = sum(sorted(part, reverse=True)[:group_top])
            keep = sorted(range(groups), key=lambda g: (-value[g], g))[:group_k]
            allowed = np.isin(np.arange(E) // size, keep)
        live = np.flatnonzero(allowed)
        idx[t] = sorted(live, key=lambda e: (-order_by[t, e], e))[:k]
    at = np.take_along_axis
    chosen_out = at(out, idx.astype(np.int64), 1)
    sel = np.where(chosen_out, 0.0, at(s, idx.astype(np.int64), 1))
    if not renorm:
        return idx, scale * sel, sel
    l = at(np.where(out, -np.inf, logits), idx.astype(np.int64), 1)
    if kind == "sigmoid":  # log sigmoid(l) = min(l, 0) - log(1 + e^-|l|)
        l = np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))
    top = l.max(1, keepdims=True)
    with np.errstate(invalid="ignore"):
        rel = np.where(np.isfinite(l), np.exp(l - np.where(np.isfinite(top), top, 0.0)), 0.0)
    total = rel.sum(1, keepdims=True)
    return idx, scale * rel / np.where(total > 0, total, 1.0), sel


def route_backward(d_w, logits, idx, w, s, kind="sigmoid", renorm=True, scale=1.0):
    T, E = logits.shape
    d = np.zeros((T, E))
    i = idx.astype(np.int64)
    if renorm:
        v = w * (d_w - (w * d_w).sum(1, keepdims=True) / scale)
        np.put_along_axis(d, i, v if kind == "softmax" else v * (1 - s), 1)
    elif kind == "sigmoid":
        np.put_along_axis(d, i, d_w * w * (1 - s), 1)
    else:
        np.put_along_axis(d, i, d_w, 1)
        d = scale * scores(logits, kind) * (d - (s * d_w).sum(1, keepdims=True))
    return d


# ------------------------------------------------------------------ norm

def rmsnorm(u, weight, eps):
    return u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * weight


def rmsnorm_backward(dy, u, weight, eps, d_sum=None):
    """(du, dw)."""
    r = 1 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
    n, g = u * r, dy * weight
    du = r * (g - n * (g * n).mean(1, keepdims=True))
    return du + (0 if d_sum is None else d_sum), (dy * n).sum(0)


# ------------------------------------------------------------------ convolution

def _starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(int)


def conv(x, weight, bias, lens, silu=True, state=None):
    """(y, state_out)."""
    D, W = weight.shape
    y, out = np.zeros_like(x), np.zeros((len(lens), W - 1, D))
    at = _starts(lens)
    for n, L in enumerate(lens):
        ext = np.concatenate([np.zeros((W - 1, D)) if state is None else state[n], x[at[n]:at[n + 1]]])
        for t in range(L):
            p = (ext[t:t + W] * weight.T).sum(0) + (0 if bias is None else bias)
            y[at[n] + t] = p * sigmoid(p) if silu else p
        out[n] = ext[L:]
    return y, out


def conv_backward(dy, x, weight, bias, lens, silu=True, state=None, d_state=None):
    """(dx, dw, db, d_state_in)."""
    D, W = weight.shape
    dx, dw, db, d_in = np.zeros_like(x), np.zeros_like(weight), np.zeros(D), np.zeros((len(lens), W - 1, D))
    at = _starts(lens)
    for n, L in enumerate(lens):
        ext = np.concatenate([np.zeros((W - 1, D)) if state is None else state[n], x[at[n]:at[n + 1]]])
        de = np.zeros_like(ext)
        if d_state is not None:
            de[L:] += d_state[n]
        for t in range(L):
            d = dy[at[n] + t]
            if silu:
                p = (ext[t:t + W] * weight.T).sum(0) + (0 if bias is None else bias)
                sg = sigmoid(p)
                d = d * sg * (1 + p * (1 - sg))
            de[t:t + W] += d * weight.T
            dw += (d * ext[t:t + W]).T
            db += d
        d_in[n], dx[at[n]:at[n + 1]] = de[:W - 1], de[W - 1:]
    return dx, dw, db, d_in


# ------------------------------------------------------------------ selective scan

def softplus(x):
    return np.maximum(x, 0) + np.log1p(np.exp(-np.abs(x)))


def _steps(delta, dt_bias, soft):
    pre = delta + (0 if dt_bias is None else dt_bias)
    return (softplus(pre), sigmoid(pre)) if soft else (pre, np.ones_like(pre))


def scan(u, delta, A, B, C, lens, skip=None, z=None, dt_bias=None, state=None, soft=True, keep=None):
    """(y, state_out); B and C are [T, G, S]. `keep` receives the states before each token and the ungated y."""
    T, D = u.shape
    G, S = B.shape[1:]
    wide = lambda m, t: np.repeat(m[t], D // G, axis=0)  # noqa: E731
    dt, _ = _steps(delta, dt_bias, soft)
    y, out = np.zeros((T, D)), np.zeros((len(lens), D, S))
    at = _starts(lens)
    before = np.zeros((T, D, S)) if keep is not None else None
    for n in range(len(lens)):
        h = np.zeros((D, S)) if state is None else state[n].copy()
        for t in range(at[n], at[n + 1]):
            if before is not None:
                before[t] = h
            h = np.exp(dt[t][:, None] * A) * h + (dt[t] * u[t])[:, None] * wide(B, t)
            y[t] = (h * wide(C, t)).sum(1) + (0 if skip is None else skip * u[t])
        out[n] = h
    if keep is not None:
        keep.update(before=before, y=y)
    return (y if z is None else y * z * sigmoid(z)), out


def scan_backward(dy, u, delta, A, B, C, lens, skip=None, z=None, dt_bias=None, state=None, d_state=None, soft=True, size=False):
    """Gradients by name. `size`: of non-negative operands, how large the terms of each sum are (A's sign does not cancel)."""
    T, D = u.shape
    G, S = B.shape[1:]
    keep = {}
    scan(u, delta, A, B, C, lens, skip, z, dt_bias, state, soft, keep)
    dt, slope = _steps(delta, dt_bias, soft)
    out = dict(du=np.zeros((T, D)), ddelta=np.zeros((T, D)), dB=np.zeros_like(B), dC=np.zeros_like(C), dA=np.zeros_like(A),
               dskip=np.zeros(D), d_state_in=np.zeros((len(lens), D, S)))
    g = dy
    if z is not None:
        sg = sigmoid(z)
        out["dz"] = dy * keep["y"] * sg * (1 + z * (1 - sg))
        g = dy * z * sg
    at = _starts(lens)
    group = lambda m: m.reshape(G, D // G, S).sum(1)  # noqa: E731
    for n in range(len(lens)):
        X = np.zeros((D, S)) if d_state is None else d_state[n].copy()
        for t in range(at[n + 1] - 1, at[n] - 1, -1):
            Bw, Cw = np.repeat(B[t], D // G, axis=0), np.repeat(C[t], D // G, axis=0)
            a = np.exp(dt[t][:, None] * A)
            h = a * keep["before"][t] + (dt[t] * u[t])[:, None] * Bw
            out["dC"][t] = group(h * g[t][:, None])
            X = X + g[t][:, None] * Cw
            out["dB"][t] = group(X * (dt[t] * u[t])[:, None])
            to_b = (X * Bw).sum(1)
            q = X * a * keep["before"][t]
            out["dA"] += q * dt[t][:, None]
            out["du"][t] = to_b * dt[t] + (0 if skip is None else skip * g[t])
            out["ddelta"][t] = ((q * (np.abs(A) if size else A)).sum(1) + to_b * u[t]) * slope[t]
            out["dskip"] += g[t] * u[t]
            X = X * a
        out["d_state_in"][n] = X
    out["d_dt_bias"] = out["ddelta"].sum(0)
    return out
