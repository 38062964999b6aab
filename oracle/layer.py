"""fp64 numpy oracle of the layer operators around the memory (test
infrastructure only): attention with a decay per head, group norm with an
activation, matrix product with bias, activation and residual.  Each follows
its definition (include/atlas_decay.h, atlas_norm.h, atlas_linear.h) token by
token, set by set, without chunks or tiles."""
from __future__ import annotations

import math

import numpy as np


def _act(z, act):
    if act == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + np.vectorize(math.erf, otypes=[np.float64])(z / math.sqrt(2.0)))
    assert act == "none"
    return z


def decay_attention(q, k, v, decay, lens=None, S0=None, scale=1.0):
    """q, k [B, Hq, T, d_k], v [B, H, T, d_v], decay [H]; returns y [B, H, T,
    d_v] and the final states [B, H, d_k, d_v].  Tokens past a row's length
    are not looked at."""
    q, k, v, decay = (np.asarray(a, np.float64) for a in (q, k, v, decay))
    B, H, T, d_v = v.shape
    share = H // q.shape[1]
    S = np.zeros((B, H, q.shape[3], d_v)) if S0 is None else np.array(S0, np.float64)
    y = np.zeros((B, H, T, d_v))
    for b in range(B):
        for t in range(T if lens is None else int(lens[b])):
            for h in range(H):
                S[b, h] = decay[h] * S[b, h] + np.outer(k[b, h // share, t], v[b, h, t])
                y[b, h, t] = scale * (q[b, h // share, t] @ S[b, h])
    return y, S


def group_norm(x, groups, weight=None, bias=None, act="none", eps=1e-5, layout="channels_last"):
    """x [N, S, C] (channels_last: statistics over the S positions of a
    group) or [N, groups, S, C / groups] (heads: over a group of a position);
    returns [N, S, C]."""
    x = np.asarray(x, np.float64)
    if layout == "heads":
        N, G, S, Cg = x.shape
        x = x.transpose(0, 2, 1, 3).reshape(N * S, 1, G * Cg)
    N_, S_, C = x.shape
    y = np.empty_like(x)
    Cg = C // groups
    for n in range(N_):
        for g in range(groups):
            part = x[n, :, g * Cg:(g + 1) * Cg]
            mean = part.mean()
            y[n, :, g * Cg:(g + 1) * Cg] = (part - mean) / np.sqrt(((part - mean) ** 2).mean() + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    y = _act(y, act)
    return y.reshape(N, S, C) if layout == "heads" else y


def linear(x, W, bias=None, residual=None, act="none"):
    """act(x W + bias) + residual."""
    y = np.asarray(x, np.float64) @ np.asarray(W, np.float64)
    if bias is not None:
        y = y + np.asarray(bias, np.float64)
    y = _act(y, act)
    return y if residual is None else y + np.asarray(residual, np.float64)
