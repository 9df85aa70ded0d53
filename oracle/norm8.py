"""Oracle: layer norm, 8-bit rows, and the backward of the gated expert FFN from 8-bit checkpoints (test
infrastructure).

Plain numpy, float64 arithmetic on whatever values the caller passes.  The pages
([P2] "Core technique") say that the backward pass runs through the forward's
buffers and are silent on norms and on what is kept between the passes, so the
definitions here are the textbook ones: the norm and its chain rule, and rows
kept as whole multiples of a power-of-two step per 32 columns.

8-bit rows: a block of up to 32 columns of a row with largest magnitude a has
exponent b = max(1, floor(log2 a) + 127) (a as float32; 1 for a = 0, 255 when a
is not finite), step 2^(b - 133), and each value is kept as the nearest whole
multiple of the step (ties to even) within +-127.
"""
from __future__ import annotations

import numpy as np

from . import layer

BLOCK = 32


def blocks(C: int) -> int:
    return (C + BLOCK - 1) // BLOCK


def save8(X: np.ndarray):
    """(codes int64 [rows, C], exps int64 [rows, blocks(C)]) of float32-representable rows."""
    rows, C = X.shape
    codes = np.zeros((rows, C), dtype=np.int64)
    exps = np.zeros((rows, blocks(C)), dtype=np.int64)
    for j in range(blocks(C)):
        v = np.asarray(X[:, j * BLOCK:(j + 1) * BLOCK], dtype=np.float64)
        with np.errstate(invalid="ignore"):
            a = np.abs(v).max(axis=1)
        ok = np.isfinite(v).all(axis=1)
        e = np.frexp(np.where(ok, a, 1.0))[1] - 1  # floor(log2 a) for a > 0
        b = np.where(ok, np.where(a > 0, np.maximum(1, e + 127), 1), 255)
        exps[:, j] = b
        scaled = np.ldexp(np.where(ok[:, None], v, 0.0), (133 - b)[:, None])
        codes[:, j * BLOCK:(j + 1) * BLOCK] = np.clip(np.rint(scaled), -127, 127).astype(np.int64)
    return codes, exps


def load8(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    """The float64 values that 8-bit rows stand for."""
    C = codes.shape[1]
    b = np.repeat(np.asarray(exps, dtype=np.int64), BLOCK, axis=1)[:, :C]
    return np.where(b == 255, np.nan, np.ldexp(np.asarray(codes, dtype=np.float64), b - 133))


def steps(exps: np.ndarray, C: int) -> np.ndarray:
    """Each value's step [rows, C]."""
    return np.ldexp(1.0, np.repeat(np.asarray(exps, dtype=np.int64), BLOCK, axis=1)[:, :C] - 133)


def layernorm(X: np.ndarray, gamma: np.ndarray, beta, eps: float):
    """(Y, mean, rstd, z) of rows X [rows, H]."""
    X = np.asarray(X, dtype=np.float64)
    m = X.mean(axis=1)
    v = ((X - m[:, None]) ** 2).mean(axis=1)
    r = 1.0 / np.sqrt(v + eps)
    z = (X - m[:, None]) * r[:, None]
    return z * gamma + (0.0 if beta is None else beta), m, r, z


def layernorm_backward(dY: np.ndarray, z: np.ndarray, rstd: np.ndarray, gamma: np.ndarray):
    """(dX, dgamma, dbeta) from the normalised rows z and rstd."""
    gy = dY * gamma
    s1 = gy.mean(axis=1, keepdims=True)
    s2 = (gy * z).mean(axis=1, keepdims=True)
    return rstd[:, None] * (gy - s1 - z * s2), (dY * z).sum(axis=0), dY.sum(axis=0)


def swiglu_backward8(Ygu: np.ndarray, dA: np.ndarray, row_gate: np.ndarray):
    """(A, dYgu, row_dgate): the activation times each row's gate, its gradient for dA taken through the ungated
    expert output, and the gradient of each row's gate."""
    h = layer.swiglu(Ygu)
    w = np.asarray(row_gate, dtype=np.float64)[:, None]
    return w * h, layer.swiglu_backward(Ygu, w * dA), (dA * h).sum(axis=1)


def dispatch8(values: np.ndarray, gamma, beta, dest_idx: np.ndarray) -> np.ndarray:
    """Rows by expert of token rows [R, S, H], times gamma plus beta."""
    v = values if gamma is None else values * gamma + (0.0 if beta is None else beta)
    return layer.dispatch(v, dest_idx)


def combine_backward_ungated(dout: np.ndarray, dest_idx: np.ndarray) -> np.ndarray:
    """The output gradient's rows by expert, without gates."""
    return layer.dispatch(dout, dest_idx)
