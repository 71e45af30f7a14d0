"""fp64 CPU oracle of the sequence mixer and of the optimizer step (test
infrastructure only): the recurrences and formulas of include/moe.h written out
token by token and value by value, sharing no code with the GPU path.
"""
from __future__ import annotations

import numpy as np


# ------------------------------------------------------------------ linear attention

def linattn_forward(q, k, v, log_decay, lens, scale, state_in=None):
    """q [T,Hs*r,Dk], k [T,Hs,Dk], v [T,Hs,Dv] (fp64), lens: the packed sequences' lengths.
    Returns o [T,Hs*r,Dv] and the states after each sequence [N,Hs,Dk,Dv]."""
    T, Hs, Dk = k.shape
    Dv, r = v.shape[2], q.shape[1] // Hs
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]
    o = np.zeros((T, Hs * r, Dv))
    states = np.zeros((len(lens), Hs, Dk, Dv))
    t = 0
    for n, length in enumerate(lens):
        S = np.zeros((Hs, Dk, Dv)) if state_in is None else np.array(state_in[n], dtype=np.float64)
        for _ in range(length):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * (q[t].reshape(Hs, r, Dk) @ S).reshape(Hs * r, Dv)
            t += 1
        states[n] = S
    return o, states


def linattn_backward(dout, q, k, v, log_decay, lens, scale, state_in=None, d_state_out=None):
    """Gradients (dq, dk, dv, d_state_in) of linattn_forward."""
    T, Hs, Dk = k.shape
    Dv, r = v.shape[2], q.shape[1] // Hs
    lam = np.exp(np.asarray(log_decay, dtype=np.float64))[:, None, None]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dS = np.zeros((len(lens), Hs, Dk, Dv))
    end = 0
    for n, length in enumerate(lens):
        start, end = end, end + length
        S = np.zeros((Hs, Dk, Dv)) if state_in is None else np.array(state_in[n], dtype=np.float64)
        for t in range(start, end):
            S = lam * S + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * (dout[t].reshape(Hs, r, Dv) @ S.transpose(0, 2, 1)).reshape(Hs * r, Dk)
        X = np.zeros((Hs, Dk, Dv)) if d_state_out is None else np.array(d_state_out[n], dtype=np.float64)
        for t in range(end - 1, start - 1, -1):
            R = X + scale * (q[t].reshape(Hs, r, Dk).transpose(0, 2, 1) @ dout[t].reshape(Hs, r, Dv))
            dk[t] = (R @ v[t][:, :, None])[:, :, 0]
            dv[t] = (k[t][:, None, :] @ R)[:, 0, :]
            X = lam * R
        dS[n] = X
    return dq, dk, dv, dS


# ------------------------------------------------------------------ AdamW

def _mix(x):
    x = x.astype(np.uint32)
    x ^= x >> np.uint32(16)
    x *= np.uint32(0x45D9F3B5)
    x ^= x >> np.uint32(15)
    x *= np.uint32(0x2F7D9D4B)
    return x ^ (x >> np.uint32(16))


def rounding_numbers(seed, step, tensor, n):
    """The 16-bit numbers (for m, sqrt(v) and the weight) that round value i of a tensor
    at a step, in [0, 1)."""
    one = lambda x: np.array([x & 0xFFFFFFFF], dtype=np.uint32)  # noqa: E731
    key = _mix(one(int(_mix(one(seed ^ int(_mix(one(step))[0])))[0]) + 0x9E3779B9 * (tensor + 1)))
    i = np.arange(n, dtype=np.uint64)
    high = _mix(((i >> np.uint64(32)) + np.uint64(int(key[0]))).astype(np.uint32))
    h = _mix(i.astype(np.uint32) ^ high)
    third = (h ^ (h >> np.uint32(15))) * np.uint32(0x1B56C4E9)
    return [(x & np.uint32(0xFFFF)).astype(np.float64) / 65536
            for x in (h, h >> np.uint32(16), third >> np.uint32(16))]


def round_stochastic(x, unit, u):
    """x to a multiple of unit: down in magnitude where the part cut off plus u stays below 1."""
    return np.sign(x) * np.floor(np.abs(x) / unit + u) * unit


def e4m3_unit(y):
    """Distance of neighbouring E4M3 values at magnitude y."""
    return np.ldexp(1.0, np.maximum(np.frexp(np.abs(y))[1] - 1, -6) - 3)


def block_scales(x, block=256):
    n = x.size
    b = np.pad(np.abs(x), (0, -n % block)).reshape(-1, block)
    return b.max(axis=1) / 448.0


def adamw_update(p, g, m, v, step, lr, beta1, beta2, eps, weight_decay, clip=1.0):
    """(p, m, v) after step number `step` (from 1), all in fp64."""
    g = g * clip
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p * (1 - lr * weight_decay) - lr * mh / (np.sqrt(vh) + eps), m, v


def clip_factor(grads, max_norm):
    norm = np.sqrt(sum(float(np.sum(np.square(g.astype(np.float64)))) for g in grads))
    return norm, min(1.0, max_norm / (norm + 1e-6))
