"""Plain 64-bit forms of the routing rules and of the 8-bit integer products.

Test infrastructure only: numpy float64 and Python integers, no code shared with the
library.  Activations are bfloat16 bit patterns (uint16), as in :mod:`.q4moe_oracle`.
"""
import numpy as np

from .q4moe_oracle import bf16_to_f64


# --------------------------------------------------------------------- routing --

def route_rule(logits, top_k, score="softmax", bias=None, n_groups=1, top_groups=1, group_terms=2,
               renormalise=True, scale=1.0):
    """(ids int32, weights float64), both [T][top_k], of logits [T][E]."""
    logits = np.asarray(logits, dtype=np.float64)
    T, E = logits.shape
    b = np.zeros(E) if bias is None else np.asarray(bias, dtype=np.float64)
    per = E // n_groups
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k))
    for t in range(T):
        l = logits[t]
        there = ~(np.isnan(l) | (l == -np.inf))
        s = np.zeros(E)
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                s[there] = 1.0 / (1.0 + np.exp(-l[there]))
        elif there.any():
            top = l[there].max()
            with np.errstate(invalid="ignore"):
                s[there] = np.where(l[there] == top, 1.0, np.exp(l[there] - top))
            s /= s.sum()
        open_ = [e for e in range(E) if there[e] and not (np.isnan(b[e]) or b[e] == -np.inf)]
        # without a bias the order is the logits' own (a sigmoid of 40 and of 50 are both 1.0)
        by_logit = bias is None and (n_groups == 1 or group_terms == 1)
        c = {e: float(l[e]) if by_logit else float(s[e] + b[e]) for e in open_}
        groups = []
        for g in range(n_groups):
            mine = sorted((c[e] for e in open_ if e // per == g), reverse=True)[:group_terms]
            if mine:
                groups.append((-sum(mine), g))
        kept = {g for _, g in sorted(groups)[:top_groups]}
        order = sorted((e for e in open_ if e // per in kept), key=lambda e: (-c[e], e))[:top_k]
        w = np.array([s[e] for e in order])
        if renormalise and len(w):
            w = w / w.sum() if w.sum() > 0 else np.zeros_like(w)
        ids[t, :len(order)] = order
        weights[t, :len(order)] = w * scale
    return ids, weights


# ---------------------------------------------------------------- 8-bit products --

def quantize_rows(x):
    """(codes int64 [m][k], scales float64 [m] holding fp32 values) of float64 rows."""
    x = np.asarray(x, dtype=np.float64)
    most = np.abs(x).max(axis=1)
    scale = (most / 127.0).astype(np.float32).astype(np.float64)
    bad = ~np.isfinite(x).all(axis=1)
    scale[bad] = np.nan
    step = np.where((scale > 0) & ~bad, scale, 1.0)[:, None]
    # a quotient of an 8- or 24-bit by a 24-bit significand is never nearer than 2^-50 to a
    # border that it does not lie on, so float64 division rounds to the right integer
    codes = np.where(((scale > 0) & ~bad)[:, None], np.rint(np.where(bad[:, None], 0.0, x) / step), 0.0)
    return np.clip(codes, -127, 127).astype(np.int64), scale


def i8_gemm(codes, scales, X_bits):
    """Y [m][n] in float64 of bfloat16 rows against int8 codes [n][k] with row scales."""
    q, sx = quantize_rows(bf16_to_f64(X_bits))
    sums = q.astype(np.float64) @ np.asarray(codes, dtype=np.float64).T  # integers below 2^53: exact
    return sums * sx[:, None] * np.asarray(scales, dtype=np.float64)[None, :]


# A computed silu(g) * u is off by at most this share of itself for |g| <= 40: g and u come
# from an exact sum through three roundings each (3 * 2^-24); an error d of g moves silu(g)
# relatively by d * (1 + |g|), here 3 * 2^-24 * 41; exp, the sum, the quotient and the
# product add at most 6 roundings more.
ACT_REL = (3 * 41 + 3 + 6) * 2.0 ** -24


def expert_rows(expert, X):
    """(y [m][H], slack [m][H]) of float64 rows through ((codes, scales) of gate, up, down).

    slack bounds how far a result may lie from y whose activations were computed in fp32: an
    activation within ACT_REL of a border between two codes may fall on either side."""
    (gc, gs), (uc, us), (dc, ds) = [(np.asarray(c, np.float64), np.asarray(s, np.float64)) for c, s in expert]
    q, sx = quantize_rows(X)
    q = q.astype(np.float64)
    g = (q @ gc.T) * sx[:, None] * gs
    u = (q @ uc.T) * sx[:, None] * us
    assert not (np.abs(g) > 40).any()
    h = g / (1.0 + np.exp(-g)) * u
    step = np.abs(h).max(axis=1) / 127.0
    safe = np.where(step > 0, step, 1.0)[:, None]
    exact = h / safe
    a = np.rint(exact)
    # the scale and the value may both be off: 127 * 2 * ACT_REL of a code at most
    near = np.abs(np.abs(exact - np.floor(exact)) - 0.5) <= 127 * 2 * ACT_REL
    unit = step[:, None] * np.abs(ds)
    slack = (near.astype(np.float64) @ np.abs(dc).T) * unit
    slack += (np.abs(a) @ np.abs(dc).T) * unit * (ACT_REL + 4 * 2.0 ** -24)
    return (a @ dc.T) * step[:, None] * ds, slack


def experts_i8(gate, up, down, X_bits, ids, weights, shared=None):
    """(y, slack, parts): the layer's output [T][H] in float64, the bound of expert_rows summed
    over the slots (with fp32 sums of up to 2 + slots roundings), and the sum of the slots'
    magnitudes (what a rounding of each summand is relative to)."""
    X = bf16_to_f64(X_bits)
    T, H = X.shape
    E = np.asarray(gate[0]).shape[0]
    y, slack, parts = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in sorted({int(v) for v in np.asarray(ids).ravel() if 0 <= v < E}):
        rows, slot = np.nonzero(np.asarray(ids) == e)
        r, s = expert_rows([(m[0][e], m[1][e]) for m in (gate, up, down)], X[rows])
        w = np.asarray(weights, np.float64)[rows, slot][:, None]
        np.add.at(y, rows, r * w)
        np.add.at(slack, rows, s * np.abs(w))
        np.add.at(parts, rows, np.abs(r * w))
    if shared is not None:
        r, s = expert_rows([(m[0][0], m[1][0]) for m in shared], X)
        y, slack, parts = y + r, slack + s, parts + np.abs(r)
    return y, slack + parts * (np.asarray(ids).shape[1] + 5) * 2.0 ** -24, parts
