"""CPU oracle for the gradient of the fused linear + logprob.

TEST INFRASTRUCTURE ONLY (see oracle/linear.py). Plain float64: the BF16 logits
x = bf16(h w^T) of ``oracle.linear``, the gradient G of each row's logits by
``oracle.logp.grad_row`` (statistics and support from the logits themselves, not
from a forward call), then grad_hidden = G w and grad_weight = G^T h.

A row whose upstream gradients are zero, or whose temperature is 0, has no
gradient: zeros, and nothing of it enters grad_weight (its hidden states may be
anything).
"""
from __future__ import annotations

import numpy as np

from . import linear as _linear
from . import logp as _logp


def logit_grad(logits_bits, vocab_real: int, temperature, target, g_ref, g_pol=None, top_p: float = 1.0,
               top_k: int = -1) -> np.ndarray:
    """G, float64 [n_rows, vocab_real], of BF16 logits [n_rows, vocab_padded]."""
    bits = np.asarray(logits_bits)
    n, padded = bits.shape
    g_ref = np.zeros(n) if g_ref is None else np.asarray(g_ref, np.float64)
    g_pol = np.zeros(n) if g_pol is None else np.asarray(g_pol, np.float64)
    out = np.zeros((n, vocab_real))
    for i in range(n):
        out[i] = _logp.grad_row(bits[i], padded, vocab_real, float(temperature[i]), int(target[i]), float(g_ref[i]),
                                float(g_pol[i]), top_p, top_k)[:vocab_real]
    return out


def products(G, hidden_bits, weight_bits):
    """(grad_hidden, grad_weight, and the sums of the magnitudes of their terms)."""
    w = _linear.bf16_to_f64(weight_bits)
    live = (G != 0).any(1)  # NaN rows count
    h = np.where(live[:, None], _linear.bf16_to_f64(hidden_bits), 0.0)
    return G @ w, G.T @ h, np.abs(G) @ np.abs(w), np.abs(G).T @ np.abs(h)


def linear_logp_backward(hidden_bits, weight_bits, vocab_padded: int, temperature, target, g_ref, g_pol=None,
                         top_p: float = 1.0, top_k: int = -1):
    """(grad_hidden, grad_weight) in float64."""
    x = _linear.logits_bf16(hidden_bits, weight_bits, vocab_padded)
    G = logit_grad(x, np.asarray(weight_bits).shape[0], temperature, target, g_ref, g_pol, top_p, top_k)
    return products(G, hidden_bits, weight_bits)[:2]
