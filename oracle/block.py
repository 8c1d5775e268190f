"""The steps around the expert layer in float64: residual addition + RMSNorm,
the top-k router, their gradients, and the expert layer for a few tokens.

Plain definitions for the tests; each gradient is the formula's, and
tests/test_oracle_block.py checks it against central differences.
"""
from __future__ import annotations

import numpy as np

from . import quant as OQ
from .formats import E4M3, decode, encode, f32


# ---- residual addition + RMSNorm ----------------------------------------------

def rmsnorm(x, residual, w, eps):
    """(s, rstd, y): s = x + residual, y = s / sqrt(mean(s^2) + eps) * w."""
    s = np.asarray(x, np.float64) + (0.0 if residual is None else np.asarray(residual, np.float64))
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=-1) + eps)
    return s, rstd, s * rstd[:, None] * w


def rmsnorm_bwd(dy, s, w, rstd, dsum=None):
    """(dx, dw) of y = s * rstd * w with rstd = 1 / sqrt(mean(s^2) + eps)."""
    xh = s * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - xh * np.mean(g * xh, axis=-1, keepdims=True))
    return dx + (0.0 if dsum is None else dsum), np.sum(dy * xh, axis=0)


# ---- top-k router ----------------------------------------------------------------

def _scores(logits, score):
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, np.float64))
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return l, 1.0 / (1.0 + np.exp(-l))
    m = l.max(axis=-1, keepdims=True)
    e = np.exp(l - np.where(np.isinf(m), 0.0, m))
    z = e.sum(axis=-1, keepdims=True)
    return l, np.where(z > 0, e / np.where(z > 0, z, 1.0), 0.0)


def _one_minus(l):
    """1 - sigmoid(l), without the cancellation of that subtraction near 1."""
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(l))


def router_topk(logits, k, score="softmax", renorm=True, scale=1.0):
    """(topk_idx, probs): the k largest logits (ties to the lower id)."""
    l, s = _scores(logits, score)
    idx = np.argsort(-l, axis=-1, kind="stable")[:, :k]
    sel = np.take_along_axis(s, idx, axis=1)
    if renorm:
        S = sel.sum(axis=1, keepdims=True)
        sel = np.where(S > 0, sel / np.where(S > 0, S, 1.0), 0.0)
    return idx, scale * sel


def router_topk_bwd(logits, idx, dprobs, score="softmax", renorm=True, scale=1.0):
    """(dlogits, bound): the gradient and, per element, the sum of the magnitudes it is made of."""
    l, s = _scores(logits, score)
    T, E = l.shape
    d = np.asarray(dprobs, np.float64)
    sel = np.take_along_axis(s, idx, axis=1)
    G = np.zeros((T, E))
    A = np.zeros((T, E))
    if renorm:
        S = sel.sum(axis=1, keepdims=True)
        q = np.where(S > 0, sel / np.where(S > 0, S, 1.0), 0.0)
        inner, mag = (d * q).sum(1, keepdims=True), (np.abs(d) * q).sum(1, keepdims=True)
        f = q * _one_minus(np.take_along_axis(l, idx, axis=1)) if score == "sigmoid" else q
        np.put_along_axis(G, idx, scale * f * (d - inner), axis=1)
        np.put_along_axis(A, idx, scale * f * (np.abs(d) + mag), axis=1)
        return G, A
    np.put_along_axis(G, idx, scale * d, axis=1)
    A = np.abs(G)
    if score == "sigmoid":
        f = s * _one_minus(l)
        return G * f, A * f
    return s * (G - (G * s).sum(1, keepdims=True)), s * (A + (A * s).sum(1, keepdims=True))


# ---- the expert layer for a few tokens -------------------------------------------

def _blockwise_rows(v):
    """1x128 blocks with s = 448 * (1 / amax), each step rounded to float32."""
    b = f32(v).astype(np.float64).reshape(v.shape[0], -1, 128)
    amax = np.abs(b).max(-1, keepdims=True)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        s = f32(448.0 * f32(1.0 / amax).astype(np.float64)).astype(np.float64)
    s = np.where(amax == 0, 1.0, np.where(np.isinf(s), OQ.FLT_MAX, s))
    codes = encode(f32(b * s).astype(np.float64), E4M3)
    return (decode(codes, E4M3) * f32(1.0 / s).astype(np.float64)).reshape(v.shape)


def quantize_rows(v, recipe, scale=None):
    """The values that the few-token layer's row-wise quantisation of v [R, K] stands for."""
    v = np.asarray(v, np.float64)
    if v.shape[0] == 0:
        return v
    if recipe == "mxfp8":
        return OQ.dequantize_mx(*OQ.quantize_mx(v, "e4m3"))
    if recipe == "blockwise":
        return _blockwise_rows(v)
    if recipe == "nvfp4":
        return OQ.dequantize_nvfp4(*OQ.quantize_nvfp4(v, np.float32(scale)), np.float32(scale), v.shape[1])
    return OQ.dequantize_tensor(OQ.quantize_tensor(v, np.float32(scale))[0], np.float32(scale))


def moe_few(x, idx, probs, w1, w2, recipe, x_scale=None, h_scale=None, nudge=0.0):
    """out[t] = sum_j probs[t, j] W2_e Q(silu(g) u), [g | u] = W1_e Q(x_t), e = idx[t, j];
    w1 [E, 2F, H], w2 [E, H, F]: the values of the quantised weights. nudge:
    relative change of h before its quantisation."""
    T, k = idx.shape
    E, F = w1.shape[0], w2.shape[2]
    xq = quantize_rows(x, recipe, x_scale)
    out = np.zeros((T, w2.shape[1]))
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if t.size == 0:
            continue
        gu = xq[t] @ w1[e].T
        g, u = gu[:, :F], gu[:, F:]
        h = quantize_rows(g / (1.0 + np.exp(-g)) * u * (1.0 + nudge), recipe, h_scale)
        np.add.at(out, t, (h @ w2[e].T) * np.asarray(probs, np.float64)[t, j][:, None])
    return out
