"""CPU oracle of routing by scores, of products in block-scaled 8-bit floating point and of AdamW.

TEST INFRASTRUCTURE, as oracle/moe_oracle.py: plain numpy definitions in float64, no blocking and no
fusion.  Pins (tests/test_oracle_train_step.py): torch float64 autograd, torch's E4M3 type and its AdamW,
central finite differences, and hand values.
"""
from __future__ import annotations

import numpy as np

D = np.float64
BLOCK = 128
TOP = 448.0
TINY = 2.0 ** -100


# ---- routing by scores ------------------------------------------------------------------------------

def scores(logits, sigmoid):
    l = np.asarray(logits, D)
    if sigmoid:
        with np.errstate(over="ignore"):
            return 1.0 / (1.0 + np.exp(-l))
    m = l.max(axis=1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0.0, m))
    s = e.sum(axis=1, keepdims=True)
    return np.divide(e, s, out=np.zeros_like(e), where=s > 0)


def _descending(v):
    """Order of the last axis: largest first, equal values by index, NaN behind every number."""
    key = np.where(np.isnan(v), -np.inf, v)
    return np.lexsort((np.broadcast_to(np.arange(v.shape[-1]), v.shape), -key, np.isnan(v)), axis=-1)


def choose(logits, bias, k, groups, topk_groups, sigmoid):
    """topk_idx [T, k]."""
    l = np.asarray(logits, D)
    T, E = l.shape
    c = scores(l, sigmoid) + (0.0 if bias is None else np.asarray(bias, D))
    open_ = np.ones((T, E), bool)
    if groups > 1:
        size = E // groups
        g = np.where(np.isnan(c), -np.inf, c).reshape(T, groups, size)
        g = np.sort(g, axis=2)[:, :, ::-1]
        best = g[:, :, 0] + g[:, :, 1] if size > 1 else g[:, :, 0]
        chosen = _descending(best)[:, :topk_groups]
        flags = np.zeros((T, groups), bool)
        np.put_along_axis(flags, chosen, True, axis=1)
        open_ = np.repeat(flags, size, axis=1)
    order = _descending(c if bias is not None else l)
    keep = np.take_along_axis(open_, order, axis=1)
    return np.stack([o[f][:k] for o, f in zip(order, keep)]) if T else np.zeros((0, k), np.int64)


def gates(logits, idx, sigmoid, renormalize, scale):
    l = np.asarray(logits, D)
    if renormalize:   # formed from the chosen logits, so that no sum underflows
        c = np.take_along_axis(l, idx, axis=1)
        low = np.minimum(c, 0.0) if sigmoid else c
        m = low.max(axis=1, keepdims=True)
        w = np.exp(low - np.where(np.isneginf(m), 0.0, m)) / (1.0 + np.exp(-np.abs(c)) if sigmoid else 1.0)
        s = w.sum(axis=1, keepdims=True)
        return scale * np.divide(w, s, out=np.zeros_like(w), where=s > 0)
    return scale * np.take_along_axis(scores(l, sigmoid), idx, axis=1)


def gates_bwd(dgate, logits, idx, sigmoid, renormalize, scale):
    """Gradient of all logits [T, E]."""
    l, dg = np.asarray(logits, D), np.asarray(dgate, D)
    g = gates(l, idx, sigmoid, renormalize, 1.0)
    dl = np.zeros(l.shape)
    if not sigmoid and not renormalize:
        p = scores(l, False)
        dl = -p * (g * dg).sum(axis=1, keepdims=True) * scale
        own = g * dg * scale
    else:
        rest = 1.0 - scores(np.take_along_axis(l, idx, axis=1), True) if sigmoid else 1.0
        inner = dg - (g * dg).sum(axis=1, keepdims=True) if renormalize else dg
        own = scale * g * rest * inner
    t = np.arange(l.shape[0])[:, None]
    np.add.at(dl, (t, idx), own)
    return dl


def move_bias(counts, rate, bias):
    n = np.asarray(counts, np.int64)
    return np.asarray(bias, D) + rate * np.sign(n.sum() - n * n.size)


# ---- 8-bit floating point with a scale for each block of 128 -----------------------------------------

def _e4m3_table():
    c = np.arange(256)
    s, e, m = c >> 7, (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(s == 1, -v, v)
    v[[0x7F, 0xFF]] = np.nan
    return v


E4M3 = _e4m3_table()
_MAGNITUDES = E4M3[:0x7F]


def e4m3(v):
    """Codes of values within +-448, to nearest, ties to the even code."""
    v = np.asarray(v, D)
    a = np.minimum(np.abs(v), TOP)
    hi = np.searchsorted(_MAGNITUDES, a)          # the first not below
    hi = np.minimum(hi, 0x7E)
    lo = np.maximum(hi - 1, 0)
    up, down = _MAGNITUDES[hi] - a, a - _MAGNITUDES[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = np.where(_MAGNITUDES[hi] == a, hi, code)
    return (code | (np.signbit(v) << 7)).astype(np.uint8)


def quantize(blocks):
    """Codes and scales of blocks [..., n]."""
    b = np.asarray(blocks, D)
    top = np.maximum(np.abs(b).max(axis=-1), TINY)
    return e4m3(np.divide(b * TOP, top[..., None])), top / TOP


def quantize_rows(x):
    """x [R, K]: codes [R, K], scales [K / 128, R]."""
    R, K = np.shape(x)
    codes, s = quantize(np.reshape(x, (R, K // BLOCK, BLOCK)))
    return codes.reshape(R, K), s.T


def quantize_weights(w):
    """w [G, N, K]: codes [G, N, K], scales [G, N / 128, K / 128]."""
    G, N, K = np.shape(w)
    b = np.reshape(w, (G, N // BLOCK, BLOCK, K // BLOCK, BLOCK)).transpose(0, 1, 3, 2, 4)
    codes, s = quantize(b.reshape(*b.shape[:3], BLOCK * BLOCK))
    codes = codes.reshape(b.shape).transpose(0, 1, 3, 2, 4).reshape(G, N, K)
    return codes, s


def rows_of(codes, scales):
    return E4M3[codes] * np.repeat(np.asarray(scales, D).T, BLOCK, axis=1)


def weights_of(codes, scales):
    return E4M3[codes] * np.repeat(np.repeat(np.asarray(scales, D), BLOCK, axis=1), BLOCK, axis=2)


def grouped_product(a, b, offsets):
    """a [M, K], b [G, N, K]: [M, N], rows outside every group NaN; the sum of magnitudes; and of each 8
    neighbouring products a bound of the largest magnitude, summed."""
    M, N = a.shape[0], b.shape[1]
    out, size, tops = (np.full((M, N), np.nan) for _ in range(3))
    top = lambda t: np.abs(t).reshape(*t.shape[:-1], -1, 8).max(axis=-1)
    for g in range(b.shape[0]):
        r0, r1 = (min(max(int(o), 0), M) for o in offsets[g:g + 2])
        if r1 > r0:
            out[r0:r1] = a[r0:r1] @ b[g].T
            size[r0:r1] = np.abs(a[r0:r1]) @ np.abs(b[g]).T
            tops[r0:r1] = top(a[r0:r1]) @ top(b[g]).T
    return out, size, tops


# ---- AdamW ------------------------------------------------------------------------------------------

def clip(sumsq, max_norm):
    return 1.0 if sumsq is None else min(1.0, max_norm / (np.sqrt(sumsq) + 1e-6))


def adamw(p, g, m, v, lr, beta1, beta2, eps, step, decay, c=1.0):
    """New p, m, v."""
    p, g, m, v = (np.asarray(t, D) for t in (p, g, m, v))
    g = c * g
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    p = (1 - lr * decay) * p - lr / (1 - beta1 ** step) * m / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p, m, v


def state_of(codes, scales):
    """An 8-bit state's values: codes [n], scales [ceil(n / 128)]."""
    return E4M3[codes] * np.repeat(np.asarray(scales, D), BLOCK)[:len(codes)]


def block_tops(v):
    """Largest magnitude of each run of 128."""
    a = np.abs(np.asarray(v, D))
    return np.array([a[i:i + BLOCK].max() for i in range(0, len(a), BLOCK)])
