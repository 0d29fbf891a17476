"""Float64 CPU oracle of the low-rank adapters beside a shared projection:
one request at a time, straight from the formulas

  H_t = X_t A_a^T,  Y_t = base_t + s_a H_t B_a^T
  G_t = s_a dY_t B_a,  dX_t = dX_base_t + G_t A_a,
  dA_a = sum_t G_t^T X_t,  dB_a = sum_t s_a dY_t^T H_t

Besides the values it returns, for each, the sum of the magnitudes of the
products the value is a sum of: what a bound on a rounding error scales with.
"""
from __future__ import annotations

import numpy as np


def _requests(offsets, slots, n_slots, rank, scale, r):
    for b, a in enumerate(slots):
        lo, hi = int(offsets[b]), int(offsets[b + 1])
        if 0 <= a < n_slots and hi > lo:
            k = r if rank is None else int(rank[a])
            yield lo, hi, int(a), k, 1.0 if scale is None else float(scale[a])


def forward(X, A, B, offsets, slots, base=None, rank=None, scale=None):
    """(Y, H, |Y| terms, |H| terms)."""
    n, r, c2 = X.shape[0], A.shape[1], B.shape[1]
    Y = np.zeros((n, c2)) if base is None else base.copy()
    aY, H, aH = np.abs(Y) * 0, np.zeros((n, r)), np.zeros((n, r))
    for lo, hi, a, k, s in _requests(offsets, slots, A.shape[0], rank, scale, r):
        W1, W2, x = A[a, :k], B[a, :, :k], X[lo:hi]
        H[lo:hi, :k] = x @ W1.T
        aH[lo:hi, :k] = np.abs(x) @ np.abs(W1).T
        Y[lo:hi] += s * (H[lo:hi, :k] @ W2.T)
        aY[lo:hi] = abs(s) * (aH[lo:hi, :k] @ np.abs(W2).T)
    return Y, H, aY, aH


def backward(X, dY, H, A, B, offsets, slots, dX_base=None, rank=None, scale=None):
    """(dX, dA, dB, and the magnitudes of their terms in the same order)."""
    dX = np.zeros(X.shape) if dX_base is None else dX_base.copy()
    dA, dB = np.zeros(A.shape), np.zeros(B.shape)
    aX, aA, aB = np.zeros(X.shape), np.zeros(A.shape), np.zeros(B.shape)
    for lo, hi, a, k, s in _requests(offsets, slots, A.shape[0], rank, scale, A.shape[1]):
        W1, W2, x, dy, h = A[a, :k], B[a, :, :k], X[lo:hi], dY[lo:hi], H[lo:hi, :k]
        G, aG = s * (dy @ W2), abs(s) * (np.abs(dy) @ np.abs(W2))
        dX[lo:hi] += G @ W1
        aX[lo:hi] += aG @ np.abs(W1)
        dA[a, :k] += G.T @ x
        aA[a, :k] += aG.T @ np.abs(x)
        dB[a, :, :k] += s * (dy.T @ h)
        aB[a, :, :k] += abs(s) * (np.abs(dy).T @ np.abs(h))
    return dX, dA, dB, aX, aA, aB
