"""Oracle: the router and its gradient, 4-bit weights, and the expert layer for few tokens (test infrastructure).

Plain numpy, float64 arithmetic on whatever values the caller passes.  The pages take a router's top-K output as given
([P2] "Core problem") and name neither scores nor weight formats, so the definitions here are the textbook ones.

Router scores of a token's logits l: softmax(l) or sigmoid(l); NaN and -inf mask an expert (score 0, never chosen), +inf
counts as the largest float32.  The K experts are the largest l, or with a bias the largest score + bias, descending, the
lowest id first among equals; -1 (gate 0) where fewer are left.

4-bit weights: per column and G rows, scale = bfloat16(float32(largest magnitude * float32(1/7))), code = the nearest
whole number (ties to even) to the float32 quotient of value and scale, held within [-8, 7].
"""
from __future__ import annotations

import numpy as np

from . import layer

LARGEST = float(np.finfo(np.float32).max)


def _masked(a):
    """float64 values as they count: NaN as -inf, at most the largest float32."""
    a = np.asarray(a, dtype=np.float64)
    return np.where(a > -np.inf, np.minimum(a, LARGEST), -np.inf)


def scores(logits, score: str):
    """Scores of logits [T, E]."""
    l = _masked(logits)
    on = l > -np.inf
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(np.where(on, l, 0.0)))
            return np.where(on, np.where(l >= 0, 1.0, e) / (1.0 + e), 0.0)
        top = np.where(on, l, -np.inf).max(axis=1, keepdims=True)
        p = np.where(on, np.exp(np.where(on, l - np.where(np.isfinite(top), top, 0.0), 0.0)), 0.0)
    total = p.sum(axis=1, keepdims=True)
    return p / np.where(total > 0, total, 1.0)


def _relative(logits, ids, score: str):
    """Scores of the chosen experts times a factor per token under which the largest is at least 1/2 (0 for no expert)."""
    l = _masked(logits)
    x = np.where(ids >= 0, np.take_along_axis(l, np.maximum(ids, 0), axis=1), -np.inf)
    on = x > -np.inf
    low = np.minimum(x, 0.0) if score == "sigmoid" else x
    top = low.max(axis=1, keepdims=True)
    w = np.where(on, np.exp(np.where(on, low - np.where(np.isfinite(top), top, 0.0), 0.0)), 0.0)
    if score == "sigmoid":
        w = w / (1.0 + np.exp(-np.abs(np.where(on, x, 0.0))))
    return w


def route(logits, bias, K: int, score: str, renorm: bool, scale: float):
    """(ids int64 [T, K], gates float64 [T, K]) of logits [T, E]."""
    l = _masked(logits)
    T, E = l.shape
    s = scores(logits, score)
    if bias is None:
        key = l
    else:
        b = _masked(bias)[None, :]
        key = np.where((l > -np.inf) & (b > -np.inf), s + np.where(b > -np.inf, b, 0.0), -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :K]
    ids = np.where(np.take_along_axis(key, order, axis=1) > -np.inf, order, -1)
    if renorm:
        w = _relative(logits, ids, score)
        total = w.sum(axis=1, keepdims=True)
        gates = w / np.where(total > 0, total, 1.0)
    else:
        gates = np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    return ids, scale * gates


def gates_of(logits, ids, score: str, renorm: bool, scale: float):
    """Gates of given experts (ids outside [0, E) have gate 0), as a function of the logits."""
    T, E = np.asarray(logits).shape
    ids = np.where((ids >= 0) & (ids < E), ids, -1)
    if renorm:
        w = _relative(logits, ids, score)
        total = w.sum(axis=1, keepdims=True)
        return scale * w / np.where(total > 0, total, 1.0)
    s = scores(logits, score)
    return scale * np.where(ids >= 0, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)


def route_backward(logits, ids, dgates, score: str, renorm: bool, scale: float):
    """(dlogits [T, E], the size of its terms [T, E]) from dgates [T, K]."""
    l = _masked(logits)
    T, E = l.shape
    ids = np.where((ids >= 0) & (ids < E), ids, -1)
    on = (ids >= 0) & (np.take_along_axis(l, np.maximum(ids, 0), axis=1) > -np.inf)
    c = np.where(on, scale * np.asarray(dgates, dtype=np.float64), 0.0)
    s = scores(logits, score)
    sk = np.where(on, np.take_along_axis(s, np.maximum(ids, 0), axis=1), 0.0)
    dl, size = np.zeros((T, E)), np.zeros((T, E))
    if renorm:
        w = _relative(logits, ids, score) * on
        total = w.sum(axis=1, keepdims=True)
        q = w / np.where(total > 0, total, 1.0)
        v = q * (c - (q * c).sum(axis=1, keepdims=True))
        z = q * (np.abs(c) + (q * np.abs(c)).sum(axis=1, keepdims=True))
        if score == "sigmoid":
            x = np.where(on, np.take_along_axis(l, np.maximum(ids, 0), axis=1), 0.0)
            rest = scores(-x, "sigmoid")
            v, z = v * rest, z * rest
    elif score == "sigmoid":
        x = np.where(on, np.take_along_axis(l, np.maximum(ids, 0), axis=1), 0.0)
        v = c * sk * scores(-x, "sigmoid")
        z = np.abs(v)
    else:
        v, z = sk * c, sk * np.abs(c)
        # an expert without a score has no part in an infinite or undefined sum
        with np.errstate(invalid="ignore"):
            dl -= np.where(s > 0, s * (sk * c).sum(axis=1, keepdims=True), 0.0)
        size += s * (sk * np.abs(c)).sum(axis=1, keepdims=True)
    for t, k in zip(*np.nonzero(on)):
        dl[t, ids[t, k]] += v[t, k]
        size[t, ids[t, k]] += z[t, k]
    return dl, size


def _bf16(a):
    """float32 values rounded to bfloat16 (nearest even), as float32; NaN for NaN."""
    a = np.asarray(a, dtype=np.float32)
    u = a.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(a), np.float32(np.nan), r)


def save4(W, G: int):
    """(codes int64 [E, H, N], scales float64 [E, ceil(H/G), N]) of float32-representable weights [E, H, N]."""
    W = np.asarray(W, dtype=np.float32)
    E, H, N = W.shape
    groups = -(-H // G)
    codes, scales = np.zeros((E, H, N), dtype=np.int64), np.zeros((E, groups, N))
    for g in range(groups):
        w = W[:, g * G:(g + 1) * G]
        ok = np.isfinite(w).all(axis=1)
        top = np.where(ok, np.abs(np.where(np.isfinite(w), w, 0)).max(axis=1), 0).astype(np.float32)
        s = _bf16(top * np.float32(1 / 7))
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            q = np.clip(np.rint(np.where(np.isfinite(w), w, 0) / s[:, None]), -8, 7)
        codes[:, g * G:(g + 1) * G] = np.where((ok & (s > 0))[:, None], q, 0)
        scales[:, g] = np.where(ok, s, np.nan)
    return codes, scales


def load4(codes, scales, G: int):
    """The float64 values of 4-bit weights."""
    H = codes.shape[1]
    return np.asarray(codes, dtype=np.float64) * np.repeat(np.asarray(scales, dtype=np.float64), G, axis=1)[:, :H]


def pack4(codes):
    """Codes [E, H, N] as int32 words [E, ceil(H/8), N]."""
    E, H, N = codes.shape
    wide = np.zeros((E, -(-H // 8) * 8, N), dtype=np.int64)
    wide[:, :H] = codes
    wide = (wide + 8).reshape(E, -1, 8, N)
    words = np.zeros((E, wide.shape[1], N), dtype=np.int64)
    for i in range(8):
        words += wide[:, :, i] << (4 * (i // 2) + 16 * (i % 2))
    return words.astype(np.uint32).view(np.int32)


def unpack4(words, H: int):
    """The codes [E, H, N] of int32 words."""
    u = np.ascontiguousarray(words).view(np.uint32).astype(np.int64)
    E, J, N = u.shape
    codes = np.zeros((E, J, 8, N), dtype=np.int64)
    for i in range(8):
        codes[:, :, i] = ((u >> (4 * (i // 2) + 16 * (i % 2))) & 15) - 8
    return codes.reshape(E, J * 8, N)[:, :H]


def few_layer(X, ids, gates, W, size=np.abs):
    """(out [T, N], the size of its terms [T, N]) of rows X [T, H], ids and gates [T, K] and weights W[e] [H, N]; ids
    outside [0, len(W)) are left out.  size(W[e]) is what stands for the weights' size."""
    X = np.asarray(X, dtype=np.float64)
    T, K = ids.shape
    out = scale = None
    for t in range(T):
        for k in range(K):
            if not 0 <= ids[t, k] < len(W):
                continue
            w = np.asarray(W[ids[t, k]], dtype=np.float64)
            if out is None:
                out, scale = np.zeros((T, w.shape[1])), np.zeros((T, w.shape[1]))
            out[t] += float(gates[t, k]) * (X[t] @ w)
            scale[t] += abs(float(gates[t, k])) * (np.abs(X[t]) @ size(w))
    return (np.zeros((T, W[0].shape[1])),) * 2 if out is None else (out, scale)


def few_ffn(X, ids, gates, W_gu, W_down, unit: float, size_gu=np.abs, size_down=np.abs):
    """(out [T, H], bound [T, H]) of the gated expert layer.  The bound follows an error of `unit` times the terms' size in
    each of the three products: d silu(g) <= 1.1 dg, and 16 * 2^-24 of the activation itself."""
    X = np.asarray(X, dtype=np.float64)
    T, K = ids.shape
    H = X.shape[1]
    out, bound = np.zeros((T, H)), np.zeros((T, H))
    for t in range(T):
        for k in range(K):
            e = ids[t, k]
            if not 0 <= e < len(W_gu):
                continue
            wg, wd = np.asarray(W_gu[e], dtype=np.float64), np.asarray(W_down[e], dtype=np.float64)
            Hp = wd.shape[0]
            y = X[t] @ wg
            dy = unit * (np.abs(X[t]) @ size_gu(wg))
            act = layer.silu(y[:Hp])
            a = act * y[Hp:]
            da = 1.1 * dy[:Hp] * (np.abs(y[Hp:]) + dy[Hp:]) + np.abs(act) * dy[Hp:] + 16 * 2.0 ** -24 * np.abs(a)
            g = float(gates[t, k])
            out[t] += g * (a @ wd)
            bound[t] += abs(g) * (da @ np.abs(wd) + unit * ((np.abs(a) + da) @ size_down(wd)))
    return out, bound
