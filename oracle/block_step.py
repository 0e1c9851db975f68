"""CPU oracle of the operators around the MoE layer: the norms before and after the block with its
gate and residual scale, the softmax cross entropy over a vocabulary, and gradient clipping.

TEST INFRASTRUCTURE, as oracle/moe_oracle.py: plain numpy definitions in float64 and the closed-form
backward of each, no blocking and no fusion.  Pins (tests/test_oracle_block_step.py): torch float64
autograd of the plain formulas, central finite differences, and hand values.
"""
from __future__ import annotations

import numpy as np

D = np.float64


def rms_rstd(v, eps):
    v = np.asarray(v, D)
    return 1.0 / np.sqrt((v * v).mean(axis=1) + eps)


def gate_of_rows(gate, gate_rows, T, d):
    """The gate row of every token, ones without a gate."""
    if gate is None:
        return np.ones((T, d))
    return np.asarray(gate, D)[np.arange(T) // gate_rows]


def norm_in(x, w, eps):
    r = rms_rstd(x, eps)
    return np.asarray(x, D) * r[:, None] * np.asarray(w, D), r


def norm_out(y, x, w, gate, gate_rows, res_scale, eps):
    T, d = np.shape(x)
    r = rms_rstd(y, eps)
    n = np.asarray(y, D) * r[:, None]
    return res_scale * np.asarray(x, D) + gate_of_rows(gate, gate_rows, T, d) * (n * np.asarray(w, D)), r


def _through_norm(u, v, r):
    """Gradient of v for the gradient u of v * r(v)."""
    n = v * r[:, None]
    return r[:, None] * (u - n * (u * n).mean(axis=1, keepdims=True))


def norm_out_bwd(dout, y, w, gate, gate_rows, r):
    dout, y, w = np.asarray(dout, D), np.asarray(y, D), np.asarray(w, D)
    T, d = y.shape
    g = gate_of_rows(gate, gate_rows, T, d)
    n = y * r[:, None]
    dy = _through_norm(dout * g * w, y, r)
    dw = (dout * g * n).sum(axis=0)
    dgate = None
    if gate is not None:
        dgate = np.zeros(np.shape(gate))
        np.add.at(dgate, np.arange(T) // gate_rows, dout * n * w)
    return dy, dw, dgate


def norm_in_bwd(dxn, x, w, r, dres, res_scale):
    dxn, x, w = np.asarray(dxn, D), np.asarray(x, D), np.asarray(w, D)
    dx = _through_norm(dxn * w, x, r)
    if dres is not None:
        dx = dx + res_scale * np.asarray(dres, D)
    return dx, (dxn * x * r[:, None]).sum(axis=0)


def vocab_loss(h, w, target):
    """Per-token loss (0 where the target is no word) and log sum of exponentials."""
    logits = np.asarray(h, D) @ np.asarray(w, D).T
    top = logits.max(axis=1)
    lse = top + np.log(np.exp(logits - top[:, None]).sum(axis=1))
    loss = np.zeros(len(target))
    ok = (np.asarray(target) >= 0) & (np.asarray(target) < logits.shape[1])
    loss[ok] = lse[ok] - logits[ok, np.asarray(target)[ok]]
    return loss, lse


def vocab_loss_bwd(h, w, target, dloss):
    h, w, target = np.asarray(h, D), np.asarray(w, D), np.asarray(target)
    logits = h @ w.T
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    ok = (target >= 0) & (target < w.shape[0])
    p[ok, target[ok]] -= 1.0
    p *= np.where(ok, np.asarray(dloss, D), 0.0)[:, None]
    return p @ w, p.T @ h


def grad_norm(grads):
    return float(np.sqrt(sum((np.asarray(g, D) ** 2).sum() for g in grads)))


def clip(grads, max_norm):
    norm = grad_norm(grads)
    with np.errstate(over="ignore"):
        c = min(1.0, max_norm / (norm + 1e-6)) if np.isfinite(np.float32(norm)) else 1.0   # as the norm is reported
    return [np.asarray(g, D) * c for g in grads], norm
