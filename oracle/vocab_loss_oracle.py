"""Float64 CPU oracle of softmax cross entropy over a vocabulary, straight from

  a = scale H W^T,  lse_t = log sum_v exp a_tv,  loss_t = lse_t - a_t,target
  d_tv = scale dloss_t (exp(a_tv - lse_t) - [v = target_t]),  dH = d W,  dW = d^T H

A row whose target is none of the vocabulary's has loss 0 and d = 0.
"""
from __future__ import annotations

import numpy as np


def live_rows(targets, v):
    return np.nonzero((targets >= 0) & (targets < v))[0]


def forward(H, W, targets, scale=1.0):
    """(loss, lse, a)."""
    a = scale * (H @ W.T)
    top = a.max(1)
    lse = top + np.log(np.exp(a - top[:, None]).sum(1))
    loss = np.zeros(H.shape[0])
    r = live_rows(targets, W.shape[0])
    loss[r] = lse[r] - a[r, targets[r]]
    return loss, lse, a


def backward(H, W, targets, lse, dloss, scale=1.0):
    """(dH, dW, d, p) with p = exp(a - lse) of the live rows, 0 elsewhere."""
    n, v = H.shape[0], W.shape[0]
    r = live_rows(targets, v)
    p = np.zeros((n, v))
    p[r] = np.exp(scale * (H[r] @ W.T) - lse[r, None])
    d = p.copy()
    d[r, targets[r]] -= 1.0
    d[r] *= scale * dloss[r, None]
    dH = d @ W
    dW = d[r].T @ H[r]
    return dH, dW, d, p
