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
