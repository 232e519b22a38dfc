"""Plain numpy oracle of the microscaled 4-bit and expert operators (fp64).

Independent of the library: values are found by distance to the levels, scales
by exact powers of two, choices by sorting, products by fp64 sums. Every
product also returns ``B``, the sum of the magnitudes of its terms, from which
callers derive rounding bounds.
"""

from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BLOCK = 32


def quantize(x, rule="floor"):
    """codes uint8 [rows, K/2] (even k low) and scales uint8 [rows, K/32]."""
    x = np.asarray(x, dtype=np.float64)
    rows, K = x.shape
    codes = np.zeros((rows, K), np.uint8)
    scales = np.zeros((rows, K // BLOCK), np.uint8)
    for r in range(rows):
        for b in range(K // BLOCK):
            v = x[r, b * BLOCK:(b + 1) * BLOCK]
            if not np.isfinite(v).all():
                scales[r, b] = 255
                continue
            top = np.abs(v).max()
            if top == 0.0:
                e = -127
            else:
                e = int(np.frexp(top)[1]) - 1 - 2          # floor(log2 top) - 2
                if rule == "ceil" and top > 6.0 * 2.0 ** e:
                    e += 1
            e = max(-127, min(127, e))
            scales[r, b] = e + 127
            d = np.abs(np.abs(v)[:, None] / 2.0 ** e - LEVELS[None, :])
            near = d == d.min(1, keepdims=True)
            # of two equally near levels the one with the even code
            c = np.array([min(np.flatnonzero(n), key=lambda i: (i % 2, i)) for n in near])
            codes[r, b * BLOCK:(b + 1) * BLOCK] = c + 8 * np.signbit(v)
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def dequantize(codes, scales):
    """fp64 values [..., K]."""
    n = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    v = LEVELS[n & 7] * np.where(n & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(int) - 127))
    return v * np.repeat(s, BLOCK, -1)


def matmul(x, w):
    """x . w^T and the sum of its terms' magnitudes."""
    return x @ w.T, np.abs(x) @ np.abs(w).T


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=1, group_best=1, renorm=True,
          scale=1.0):
    """ids int32 and weights fp64, both [T, k]."""
    l = np.asarray(logits, dtype=np.float64)
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    weights = np.zeros((T, k))
    for t in range(T):
        with np.errstate(all="ignore"):
            if score == "softmax":
                p = np.exp(l[t] - np.max(l[t]))
                s = p / p.sum()
            else:
                s = 1.0 / (1.0 + np.exp(-l[t]))
            by_logit = bias is None and (groups == 1 or group_best == 1)
            key = l[t].copy() if by_logit else s + (0.0 if bias is None else np.asarray(bias, np.float64))
            key[np.isnan(key) | np.isneginf(l[t])] = -np.inf
            if groups > 1:
                per = key.reshape(groups, -1)
                rank = np.sort(per, -1)[:, ::-1][:, :group_best].sum(-1)
                keep = np.argsort(-rank, kind="stable")[:top_groups]
                mask = np.zeros(groups, bool)
                mask[keep] = True
                key = np.where(mask[:, None], per, -np.inf).reshape(-1)
            order = [e for e in np.argsort(-key, kind="stable") if key[e] > -np.inf][:k]
            ids[t, :len(order)] = order
            w = s[order]
            if renorm:
                w = w / (w.sum() + (1e-20 if score == "sigmoid" else 0.0))
            if score == "softmax" and not (l[t] < np.inf).all():
                w = np.full(len(order), np.nan)
            weights[t, :len(order)] = w * scale
    return ids, weights


def plan(ids, experts):
    """offsets [E + 1] and order [T * k]: the pairs grouped by expert, in rising order."""
    flat = np.asarray(ids).reshape(-1)
    lists = [np.flatnonzero(flat == e) for e in range(experts)]
    offsets = np.concatenate(([0], np.cumsum([len(a) for a in lists]))).astype(np.int32)
    order = np.full(flat.size, -1, np.int32)
    order[:offsets[-1]] = np.concatenate(lists) if experts else []
    return offsets, order


def moe_mlp(x, gate_up, down, ids, weights, u_h, depth1, depth2, eps=2.0 ** -23):
    """The experts' block, and a bound on the error of an evaluation that sums
    chains of depth1 and depth2 fp32 additions and rounds h to u_h."""
    T, D = x.shape
    E, _, F = down.shape
    y, err = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < E:
                continue
            g, bg = matmul(x[t:t + 1], gate_up[e, :F])
            u, bu = matmul(x[t:t + 1], gate_up[e, F:])
            s = g / (1.0 + np.exp(-g))
            h = s * u
            # |silu'| <= 1.1; 32 eps: the exponential, the division, the products
            dh = 1.1 * np.abs(u) * depth1 * eps * bg + (np.abs(s) + 1.1 * depth1 * eps * bg) * depth1 * eps * bu
            dh = dh + np.abs(h) * (u_h + 32 * eps)
            o, bo = matmul(h, down[e])
            w = weights[t, j]
            y[t] += w * o[0]
            err[t] += np.abs(w) * (dh @ np.abs(down[e]).T + (depth2 + 8) * eps * bo)[0]
    return y, err
