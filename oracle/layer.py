"""The 8-bit integer operators and the gated feed-forward block in float64:
rows quantised with one scale each, the scaled product, the activations with
their slopes, the block and its gradients.  Written from the formulas alone;
matrices are numpy arrays, C = A.B^T with B's rows the outputs."""
import numpy as np
from scipy import special

ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


def quantize(X):
    """(Q int8, S float32) of X (float64 values), row by row: S the largest
    magnitude over 127 as a float, 2^-126 at least; Q the quotient's nearest whole
    number, ties to even.  A row that is not finite: NaN and zeros."""
    X = np.asarray(X, dtype=np.float64)
    ok = np.isfinite(X).all(axis=1)
    Y = np.where(ok[:, None], X, 0.0)
    top = np.abs(Y).max(axis=1, initial=0.0)
    # the float32 quotient of two float32 numbers: the float64 one, rounded again, would do
    # but for ties of ties; float32 arithmetic itself is exact about it
    S = np.maximum(top.astype(np.float32) / np.float32(127), np.float32(2.0 ** -126))
    Q = np.rint(Y / S.astype(np.float64)[:, None]).astype(np.int8)
    return Q, np.where(ok, S, np.float32(np.nan)).astype(np.float32)


def dequantize(Q, S):
    return Q.astype(np.float64) * S.astype(np.float64)[:, None]


def product(A, SA, B, SB):
    """The scaled product: exact sums, scaled in float64."""
    s = A.astype(np.int64) @ B.astype(np.int64).T
    return s.astype(np.float64) * SA.astype(np.float64)[:, None] * SB.astype(np.float64)[None, :]


def act(name, x):
    x = np.asarray(x, dtype=np.float64)
    if name == "none":
        return x
    if name == "relu":
        return np.where(x < 0, 0.0, x)
    if name == "silu":
        return x * special.expit(x)
    if name == "gelu":
        return x * special.ndtr(x)
    # (1 + tanh y) / 2 is the logistic function of 2 y, which does not cancel
    return x * special.expit(2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))


def slope(name, x):
    x = np.asarray(x, dtype=np.float64)
    if name == "none":
        return np.ones_like(x)
    if name == "relu":
        return np.where(x <= 0, 0.0, 1.0)
    if name == "silu":
        s = special.expit(x)
        return s * (1 + x * special.expit(-x))
    if name == "gelu":
        return special.ndtr(x) + x * np.exp(-0.5 * x * x) / np.sqrt(2 * np.pi)
    c = np.sqrt(2 / np.pi)
    y = c * (x + 0.044715 * x ** 3)
    s = special.expit(2 * y)
    return s + 2 * x * s * special.expit(-2 * y) * c * (1 + 3 * 0.044715 * x * x)


def gated(name, X, WG, WU):
    """(H, G, U) of the block."""
    G, U = X @ WG.T, X @ WU.T
    return act(name, G) * U, G, U


def gated_slopes(name, G, U, DH):
    """(DG, DU)."""
    return DH * U * slope(name, G), DH * act(name, G)


def gated_products(DG, DU, X, WG, WU):
    """(DX, DWG, DWU)."""
    return DG @ WG + DU @ WU, DG.T @ X, DU.T @ X
