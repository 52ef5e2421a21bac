"""float64 definitions of the layer operators (include/gdn_layer.h): numpy, one token after another.

TEST INFRASTRUCTURE ONLY, like the rest of this package: no code is shared with the CUDA library.
"""
from __future__ import annotations

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def rule_step(S, q, k, v, g, beta, scale=1.0):
    """One token through one head: (o [d_v], new S [d_v, d_k])."""
    S = np.exp(_f64(g)) * S
    u = beta * (v - S @ k)
    S = S + np.outer(u, k)
    return scale * (S @ q), S


def prefill(q, k, v, g, beta, offsets, S0=None, slots=None, fresh=None, scale=1.0, n_states=None):
    """(o [T, Hv, d_v], pool of states): the rule over each prompt; slots, fresh as in gdn_prefill."""
    q, k, v, g, beta = map(_f64, (q, k, v, g, beta))
    T, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    B = len(offsets) - 1
    pool = np.zeros((n_states or B, Hv, dv, dk)) if S0 is None else _f64(S0).copy()
    o = np.zeros((T, Hv, dv))
    for b in range(B):
        s = b if slots is None else int(slots[b])
        for h in range(Hv):
            S = np.zeros((dv, dk)) if S0 is None or (fresh is not None and fresh[b]) else pool[s, h].copy()
            hk = h // (Hv // Hk)
            for t in range(int(offsets[b]), int(offsets[b + 1])):
                o[t, h], S = rule_step(S, q[t, hk], k[t, hk], v[t, h], g[t, h], beta[t, h], scale)
            pool[s, h] = S
    return o, pool


def decode(q, k, v, g, beta, S, slots=None, scale=1.0):
    """(o [B, Hv, d_v], pool): one token a request; a negative slot is a row of zeros."""
    q, k, v, g, beta = map(_f64, (q, k, v, g, beta))
    pool = _f64(S).copy()
    B, Hv, dv = v.shape
    o = np.zeros((B, Hv, dv))
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if s < 0:
            continue
        for h in range(Hv):
            hk = h // (Hv // q.shape[1])
            o[b, h], pool[s, h] = rule_step(pool[s, h], q[b, hk], k[b, hk], v[b, h], g[b, h], beta[b, h], scale)
    return o, pool


def qk_gates(q, k, a, b, A_log, dt_bias, eps):
    q, k, a, b = map(_f64, (q, k, a, b))
    unit = [x / np.sqrt(np.sum(x * x, axis=-1, keepdims=True) + eps) for x in (q, k)]
    x = a + _f64(dt_bias)
    g = -np.exp(_f64(A_log)) * np.logaddexp(x, 0.0)
    return unit[0], unit[1], g, 1.0 / (1.0 + np.exp(-b))


def norm_gate(o, z, weight, eps, act="silu"):
    o, z = _f64(o), _f64(z)
    gate = 1.0 / (1.0 + np.exp(-z))
    if act == "silu":
        gate = gate * z
    return o / np.sqrt(np.mean(o * o, axis=-1, keepdims=True) + eps) * _f64(weight) * gate


def residual_norm(x, y, weight, scale, post_weight, eps):
    x, y = _f64(x), _f64(y)
    if post_weight is not None:
        y = y / np.sqrt(np.mean(y * y, axis=-1, keepdims=True) + eps) * _f64(post_weight)
    h = x + scale * y
    return h, h / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps) * _f64(weight)
