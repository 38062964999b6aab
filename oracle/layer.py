"""fp64 numpy oracle of the layer operators around the memory (test
infrastructure only): attention with a decay per head, group norm with an
activation, matrix product with bias, activation and residual; short causal
convolution, root-mean-square norm with the residual, matrix product with 4-bit
weights, scan with per-token decays and steps.  Each follows its definition
(include/atlas_decay.h, atlas_norm.h, atlas_linear.h, atlas_conv.h, atlas_rms.h,
atlas_qlinear.h, atlas_scan.h) token by token, set by set, without chunks or
tiles."""
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


def short_conv(x, w, bias=None, cache=None, lens=None, act="none"):
    """y_t = act(bias + sum_j w[:, K-1-j] x_{t-j}) and the next call's cache:
    the last K - 1 rows of [cache, x] (include/atlas_conv.h).  x [B, T, C], w [C,
    K], cache [B, K-1, C] (zero without one)."""
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    B, T, C = x.shape
    K = w.shape[1]
    before = np.zeros((B, K - 1, C)) if cache is None else np.asarray(cache, np.float64)
    y, keep = np.zeros((B, T, C)), np.zeros((B, K - 1, C))
    for b in range(B):
        n = T if lens is None else int(lens[b])
        rows = np.concatenate([before[b], x[b, :n]])
        for t in range(n):
            z = np.zeros(C) if bias is None else np.array(bias, np.float64)
            for i in range(K):
                z = z + w[:, i] * rows[t + i]
            y[b, t] = _act(z, act)
        keep[b] = rows[len(rows) - (K - 1):]
    return y, keep


def rms_norm(x, residual=None, weight=None, eps=1e-6):
    """h = x + residual, y = h / sqrt(mean h^2 + eps) * weight, per row."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    return (y if weight is None else y * np.asarray(weight, np.float64)), h


def e4m3_scales(y, block):
    """max(2^-100, largest |y|) / 448 of each run of `block` values of a row (0: of the row)."""
    M, C = y.shape
    step = block or C
    return np.stack([np.maximum(np.abs(y[:, i:i + step]).max(axis=1), 2.0 ** -100) / 448 for i in range(0, C, step)], 1)


def quant_weights(q, scales, zeros, K, group):
    """scale (q - zero) as [K, N], q [ceil(K / 2), N] with two rows in a byte."""
    N = q.shape[1]
    W = np.zeros((K, N))
    for k in range(K):
        v = (q[k // 2] >> (4 * (k % 2))) & 15
        zero = 8.0 if zeros is None else (zeros[k // group] & 15).astype(np.float64)
        W[k] = np.asarray(scales[k // group], np.float64) * (v.astype(np.float64) - zero)
    return W


def quant_linear(x, W, x_scale=None, x_block=0, bias=None, residual=None, act="none"):
    """act((x x_scale) W + bias) + residual, W from quant_weights."""
    x = np.asarray(x, np.float64)
    if x_scale is not None:
        x = x * np.repeat(np.asarray(x_scale, np.float64), x_block or x.shape[1], axis=1)[:, :x.shape[1]]
    return linear(x, W, bias, residual, act)


def selective_scan(q, k, v, step, decay, D=None, lens=None, S0=None, scale=1.0):
    """S_t = g_t S_{t-1} + s_t k_t^T v_t, y_t = scale q_t S_t + D v_t, token by
    token (include/atlas_scan.h).  q, k [B, Hq, T, d_k], v [B, H, T, d_v], step s
    and decay g [B, H, T], D [H]."""
    q, k, v, step, decay = (np.asarray(a, np.float64) for a in (q, k, v, step, decay))
    B, H, T, d_v = v.shape
    share = H // q.shape[1]
    S = np.zeros((B, H, q.shape[3], d_v)) if S0 is None else np.array(S0, np.float64)
    y = np.zeros((B, H, T, d_v))
    for b in range(B):
        for t in range(T if lens is None else int(lens[b])):
            for h in range(H):
                S[b, h] = decay[b, h, t] * S[b, h] + step[b, h, t] * np.outer(k[b, h // share, t], v[b, h, t])
                y[b, h, t] = scale * (q[b, h // share, t] @ S[b, h])
                if D is not None:
                    y[b, h, t] += D[h] * v[b, h, t]
    return y, S


def step_gates(dt, dt_bias, A):
    """s = softplus(dt + dt_bias), g = exp(s A); dt [B, H, T], dt_bias and A [H]."""
    x = np.asarray(dt, np.float64) + (0.0 if dt_bias is None else np.asarray(dt_bias, np.float64)[:, None])
    s = np.maximum(x, 0.0) + np.log1p(np.exp(-np.abs(x)))
    return s, np.exp(s * np.asarray(A, np.float64)[:, None])
