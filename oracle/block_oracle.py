"""Float64 numpy oracle of the operators around the linears of a transformer block.

Test infrastructure only, written from the formulas; shares no code with the
library.  bf16 values travel as float64 arrays that hold them exactly.
"""
from __future__ import annotations

import numpy as np


def attention(Q, K, V, cu_q, cu_k, scale, causal):
    """(O [Tq, Hq, D], lse [Hq, Tq], A) in float64; A = sum_j p_ij |V_j|, which scales the
    error that a relative error of the weights p makes in O.  Rows outside the sequences: NaN."""
    Tq, Hq, D = Q.shape
    G = Hq // K.shape[1]
    O = np.full(Q.shape, np.nan)
    A = np.full(Q.shape, np.nan)
    lse = np.full((Hq, Tq), np.nan)
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        nq, nk = q1 - q0, k1 - k0
        if nq == 0:
            continue
        seen = np.ones((nq, nk), bool)
        if causal:
            seen = np.arange(nk)[None, :] <= np.arange(nq)[:, None] + nk - nq
        for h in range(Hq):
            s = scale * (Q[q0:q1, h] @ K[k0:k1, h // G].T)
            s = np.where(seen, s, -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
            l = e.sum(axis=1)
            p = e / np.where(l > 0, l, 1.0)[:, None]
            O[q0:q1, h] = p @ V[k0:k1, h // G]
            A[q0:q1, h] = p @ np.abs(V[k0:k1, h // G])
            with np.errstate(divide="ignore"):
                lse[h, q0:q1] = m + np.log(l)
    return O, lse, A


def sees(nq, nk, causal, left=-1, right=-1, sinks=0):
    """bool [nq, nk]: query i, at key p = i + nk - nq, sees key j in [p - left, p + right] (-1: no
    limit) or among the first `sinks`; causal: none past p."""
    p = np.arange(nq)[:, None] + nk - nq
    j = np.arange(nk)[None, :]
    window = np.ones((nq, nk), bool)
    if left >= 0:
        window &= j >= p - left
    if right >= 0:
        window &= j <= p + right
    window |= j < sinks
    return window & (j <= p) if causal else window


def attention_spans(Q, K, V, cu_q, cu_k, scale, causal, left=-1, right=-1, sinks=0, PK=None, PV=None):
    """attention() over a window and first keys, and over keys PK, PV [P, Hkv, D] that every query
    sees: (O, lse, A) as there, and M [Hq, Tq] = max_j sum_d |q_d k_d| over the keys that are seen."""
    Tq, Hq, D = Q.shape
    G = Hq // K.shape[1]
    O, A = np.full(Q.shape, np.nan), np.full(Q.shape, np.nan)
    lse, M = np.full((Hq, Tq), np.nan), np.zeros((Hq, Tq))
    for b in range(len(cu_q) - 1):
        q0, q1, k0, k1 = cu_q[b], cu_q[b + 1], cu_k[b], cu_k[b + 1]
        if q1 == q0:
            continue
        own = sees(q1 - q0, k1 - k0, causal, left, right, sinks)
        for h in range(Hq):
            q, k, v, seen = Q[q0:q1, h], K[k0:k1, h // G], V[k0:k1, h // G], own
            if PK is not None:
                k, v = np.concatenate([PK[:, h // G], k]), np.concatenate([PV[:, h // G], v])
                seen = np.concatenate([np.ones((q1 - q0, len(PK)), bool), own], axis=1)
            used = seen.any(axis=0)              # what no query sees may hold anything
            k, v, seen = k[used], v[used], seen[:, used]
            s = np.where(seen, scale * (q @ k.T), -np.inf)
            m = s.max(axis=1, initial=-np.inf)
            e = np.exp(s - np.where(np.isfinite(m), m, 0.0)[:, None])
            l = e.sum(axis=1)
            p = e / np.where(l > 0, l, 1.0)[:, None]
            O[q0:q1, h], A[q0:q1, h] = p @ v, p @ np.abs(v)
            with np.errstate(divide="ignore"):
                lse[h, q0:q1] = m + np.log(l)
            M[h, q0:q1] = np.where(seen, np.abs(q) @ np.abs(k).T, 0.0).max(axis=1, initial=0.0)
    return O, lse, A, M


def _norm(v, kind, eps):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(axis=1, keepdims=True)
    return v / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def block_norm(x, y, cu, post, w_post, gate, a, c, pre, w_pre, b_pre, scale, shift, eps):
    """(x', h) in float64: x' = a x + c gate post(y), h = (pre(x') w + b)(1 + scale) + shift;
    None stands for an absent operand.  Rows outside the sequences: NaN."""
    xo = np.full(x.shape, np.nan)
    h = np.full(x.shape, np.nan)
    for b in range(len(cu) - 1):
        r = slice(cu[b], cu[b + 1])
        v = a * x[r]
        if y is not None:
            u = _norm(y[r], post, eps)
            if w_post is not None:
                u = u * w_post
            if gate is not None:
                u = u * gate[b]
            v = v + c * u
        xo[r] = v
        n = _norm(v, pre, eps)
        if w_pre is not None:
            n = n * w_pre
        if b_pre is not None:
            n = n + b_pre
        if scale is not None:
            n = n * (1 + scale[b])
        if shift is not None:
            n = n + shift[b]
        h[r] = n
    return xo, h


def qk_norm_rope(v, cu, positions, kind, w, bias, eps, cos, sin, halves):
    """One of Q, K [rows, H, D] in float64: (turned, n, pairs' cosines and sines [rows, 1, r / 2]); n the
    normalised values before weight and bias.  positions None: a token's number in its sequence; one outside
    of the tables [positions, r / 2] turns nothing.  Rows outside the sequences: NaN."""
    rows, H, D = v.shape
    n = _norm(v.reshape(rows * H, D), kind, eps).reshape(v.shape)
    t = n * (1.0 if w is None else w) + (0.0 if bias is None else bias)
    at = np.full(rows, -1, np.int64)
    for b in range(len(cu) - 1):
        at[cu[b]:cu[b + 1]] = np.arange(cu[b + 1] - cu[b]) if positions is None else positions[cu[b]:cu[b + 1]]
    r = 0 if cos is None else 2 * cos.shape[1]
    c, s = np.ones((rows, 1, r // 2)), np.zeros((rows, 1, r // 2))
    if r:
        known = (at >= 0) & (at < len(cos))
        c[known, 0], s[known, 0] = cos[at[known]], sin[at[known]]
    out = t.copy()
    first, second = pairs_of(r, halves)
    out[..., first] = t[..., first] * c - t[..., second] * s
    out[..., second] = t[..., second] * c + t[..., first] * s
    out[:cu[0]], out[cu[-1]:] = np.nan, np.nan
    return out, n, c, s


def pairs_of(r, halves):
    """The channels of the pairs' first and second members."""
    i = np.arange(r // 2)
    return (i, i + r // 2) if halves else (2 * i, 2 * i + 1)


def activation(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z**3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


def linear(X, W, bias, act, residual):
    """act(X W^T + bias) + residual in float64."""
    z = X @ W.T
    if bias is not None:
        z = z + bias
    y = activation(z, act)
    return y if residual is None else y + residual
