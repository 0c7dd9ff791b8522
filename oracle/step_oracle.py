"""Plain 64-bit forms of the norm, of microscaled 4-bit rows and products, and of sampling.

Test infrastructure only: numpy float64 and Python integers, no code shared with the
library.  bfloat16 values are bit patterns (uint16), as in :mod:`.q4moe_oracle`.
"""
import numpy as np

from .q4moe_oracle import bf16_to_f64


def f64_to_bf16(x):
    """float64 values rounded to the nearest bfloat16 (ties to even), as float64."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        _, e = np.frexp(x)
        step = np.ldexp(1.0, np.maximum(e - 8, -133))  # the last bit's weight; subnormals below 2^-126
        r = np.rint(x / step) * step
        r = np.where(np.abs(r) >= 2.0 ** 128, np.copysign(np.inf, x), r)
    return np.where(np.isfinite(x), r, x)


# ------------------------------------------------------------------------ norm --

def rms_norm(X, weight, eps, residual=None):
    """(t, y) in float64 of bfloat16 bits X [rows][k]."""
    t = bf16_to_f64(X)
    if residual is not None:
        t = f64_to_bf16(t + bf16_to_f64(residual))
    with np.errstate(invalid="ignore", over="ignore"):
        rms = np.sqrt(np.mean(t * t, axis=1, keepdims=True) + eps)
        return t, t / rms * bf16_to_f64(weight)


# ---------------------------------------------------------- microscaled 4 bits --

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mx4_quantize(x):
    """(codes uint8 [rows][k/2], scales uint8 [rows][k/32]) of float64 rows."""
    x = np.asarray(x, dtype=np.float64)
    rows, k = x.shape
    g = x.reshape(rows, k // 32, 32)
    top = np.abs(g).max(axis=2)
    bad = ~np.isfinite(g).all(axis=2)
    e = np.zeros(top.shape, dtype=np.int64) - 127
    there = ~bad & (top > 0)
    e[there] = np.maximum(np.frexp(top[there])[1] - 1 - 2, -127)
    a = np.where(bad[..., None], 0.0, np.ldexp(np.abs(np.where(np.isfinite(g), g, 0.0)), -e[..., None]))
    code = np.zeros(a.shape, dtype=np.uint8)
    for c in range(7):
        border = (LEVELS[c] + LEVELS[c + 1]) / 2
        code = np.where((a > border) | ((a == border) & (c % 2 == 1)), c + 1, code)
    code = (code | np.where(np.signbit(g) & ~bad[..., None], 8, 0)).astype(np.uint8).reshape(rows, k)
    return code[:, 0::2] | code[:, 1::2] << 4, np.where(bad, 255, e + 127).astype(np.uint8)


def mx4_values(codes, scales):
    """float64 [.., k] of codes [.., k/2] and scales [.., k/32] (255: NaN)."""
    c = np.stack((codes & 15, codes >> 4), axis=-1).reshape(*codes.shape[:-1], -1)
    v = np.where(c > 7, -1.0, 1.0) * LEVELS[c & 7]
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return v * np.repeat(s, 32, axis=-1)


def mx4_round(x):
    """float64 rows as what their 4-bit form stands for."""
    return mx4_values(*mx4_quantize(x))


# -------------------------------------------------------------------- sampling --

def sample(logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """(ids, probabilities) of float64 logits [B][V] and numbers u [B]; -1 and 0 where no logit is open."""
    B, V = logits.shape
    ids, probs = np.full(B, -1, dtype=np.int32), np.zeros(B)
    for b in range(B):
        l = np.where(np.isnan(logits[b]), -np.inf, logits[b])
        top = l.max()
        if top == -np.inf:
            continue
        order = np.lexsort((np.arange(V), -l))
        t = 1.0 if temperature is None else float(temperature[b])
        if not t > 0:
            ids[b], probs[b] = order[0], 1.0
            continue
        n = V
        if top_k is not None and top_k[b] > 0:
            n = min(n, int(top_k[b]))
        with np.errstate(invalid="ignore", over="ignore"):
            d = np.where(l[order] == top, 0.0, (top - l[order]) / t)
        w = np.where(l[order] == -np.inf, 0.0, np.exp(-np.where(np.isnan(d), np.inf, d)))[:n]
        if top_p is not None and top_p[b] < 1:
            n = min(n, int((np.cumsum(w) < float(top_p[b]) * w.sum()).sum()) + 1)
            w = w[:n]
        if min_p is not None and min_p[b] > 0:
            n = max(1, int((w >= min(float(min_p[b]), 1.0)).sum()))
            w = w[:n]
        back = np.argsort(order[:n])
        c = np.cumsum(w[back])
        x = min(max(float(u[b]), 0.0), 1.0) if u[b] == u[b] else 0.0
        at = int((c <= x * c[-1]).sum())
        if at >= n:  # u of 1 and more: the last token that has a weight
            at = int(np.nonzero(w[back] > 0)[0][-1])
        ids[b], probs[b] = order[:n][back][at], w[back][at] / c[-1]
    return ids, probs
