"""Float64 oracle of the operators around the layer: 8-bit activation
checkpoints, layer norm / RMS norm, and linear cross entropy.

Test infrastructure only.  Everything is written from the definitions; bounds
for the kernels' rounding are derived in the tests that use them.
"""
from __future__ import annotations

import numpy as np

CKPT_BLOCK = 32


def ckpt8_quantize(x: np.ndarray):
    """(q int8 [T, d], scale uint8 [T, d/32]) of the checkpoint of x (float64
    values of bf16 numbers): e is the least integer with max|x| <= 127 * 2^e,
    kept in [-126, 121]; q = x / 2^e to nearest, ties to even."""
    T, d = x.shape
    b = x.reshape(T, d // CKPT_BLOCK, CKPT_BLOCK)
    q = np.zeros(b.shape, dtype=np.int8)
    scale = np.full(b.shape[:2], 255, dtype=np.uint8)
    finite = np.isfinite(b).all(axis=-1)
    top = np.abs(b[finite]).max(axis=-1, initial=0.0)
    e = np.full(top.shape, -126)
    for cand in range(121, -127, -1):                       # the smallest exponent that still fits
        e[top <= 127.0 * 2.0 ** cand] = cand
    e[top > 127.0 * 2.0 ** 121] = 121
    q[finite] = np.clip(np.rint(b[finite] / (2.0 ** e)[:, None]), -127, 127).astype(np.int8)
    scale[finite] = (e + 127).astype(np.uint8)
    return q.reshape(T, d), scale


def ckpt8_values(q: np.ndarray, scale: np.ndarray) -> np.ndarray:
    """The values (float64) that a checkpoint stands for."""
    T, d = q.shape
    step = np.where(scale == 255, np.nan, 2.0 ** (scale.astype(np.float64) - 127.0))
    return (q.reshape(T, -1, CKPT_BLOCK).astype(np.float64) * step[..., None]).reshape(T, d)


def norm_forward(x, w, b, eps: float, rms: bool):
    """(y, mean, rstd) in float64."""
    mu = np.zeros((x.shape[0], 1)) if rms else x.mean(axis=1, keepdims=True)
    r = 1.0 / np.sqrt(((x - mu) ** 2).mean(axis=1, keepdims=True) + eps)
    y = (x - mu) * r * w
    return (y if b is None else y + b), mu[:, 0], r[:, 0]


def norm_backward(dy, x, w, eps: float, rms: bool):
    """(dx, dw, db) in float64."""
    _, mu, r = norm_forward(x, w, None, eps, rms)
    xh = (x - mu[:, None]) * r[:, None]
    u = dy * w
    m1 = 0.0 if rms else u.mean(axis=1, keepdims=True)
    dx = r[:, None] * (u - m1 - xh * (u * xh).mean(axis=1, keepdims=True))
    return dx, (dy * xh).sum(axis=0), dy.sum(axis=0)


def cross_entropy(h, w, target, ignore_index: int, reduction: str, dloss=None):
    """(loss, dH, dW, P) in float64; P = c (softmax - onehot) per token."""
    T, V = h.shape[0], w.shape[0]
    keep = (target != ignore_index) & (target >= 0) & (target < V)
    logits = h @ w.T
    top = logits.max(axis=1, keepdims=True)
    ex = np.exp(logits - top)
    s = ex.sum(axis=1, keepdims=True)
    safe = np.where(keep, target, 0)
    rows = np.arange(T)
    losses = np.where(keep, (top + np.log(s))[:, 0] - logits[rows, safe], 0.0)
    c = keep.astype(np.float64)
    if reduction == "mean":
        c = c / max(1, int(keep.sum()))
    loss = losses if reduction == "none" else (losses * c).sum()
    if dloss is not None:
        c = c * dloss
    p = ex / s
    at = p[rows, safe].copy()
    p[rows, safe] = 0.0
    p[rows, safe] = -np.where(at < 0.5, 1.0 - at, p.sum(axis=1))
    P = p * c[:, None]
    return loss, P @ w, P.T @ h, P
