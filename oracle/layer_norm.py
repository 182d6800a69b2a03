"""CPU oracle for the layer norm / RMS norm and its backward pass.

TEST INFRASTRUCTURE ONLY (see oracle/linear.py). Plain float64 on float64 views
of the inputs; the backward pass takes the forward's mean and rstd, as the entry
point does.
"""
from __future__ import annotations

import numpy as np


def forward(x, weight, bias, eps: float, rms: bool):
    """(y, mean, rstd) in float64."""
    x = np.asarray(x, np.float64)
    m = np.zeros(x.shape[0]) if rms else x.mean(1)
    c = x - m[:, None]
    r = 1.0 / np.sqrt((c * c).mean(1) + eps)
    y = c * r[:, None] * np.asarray(weight, np.float64)
    return (y if bias is None else y + np.asarray(bias, np.float64)), m, r


def backward(dy, x, weight, mean, rstd, rms: bool):
    """(dx, dweight, dbias) in float64; a row whose dy is all zeros counts as zeros."""
    dy = np.asarray(dy, np.float64)
    live = (dy != 0).any(1)[:, None]
    r = np.where(live, np.asarray(rstd, np.float64)[:, None], 0.0)
    c = np.where(live, np.asarray(x, np.float64), 0.0)
    if not rms:
        c = c - np.where(live, np.asarray(mean, np.float64)[:, None], 0.0)
    hat = c * r
    g = np.where(live, dy * np.asarray(weight, np.float64), 0.0)
    dx = g - hat * (g * hat).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    return dx * r, (dy * hat).sum(0), dy.sum(0)
