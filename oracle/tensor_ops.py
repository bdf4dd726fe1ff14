"""64-bit oracle of the operators over lists of tensors: the global norm with
its clip factor, clipping, and the AdamW update with decoupled weight decay
(Loshchilov and Hutter, "Decoupled Weight Decay Regularization", Algorithm 2).
"""
from __future__ import annotations

import math

import numpy as np


def grad_norm(grads, ord=2, max_norm=math.inf, eps=1e-6, inv_scale=1.0):
    """(norm, clip factor, norm of every array) of float64 arrays."""
    if ord == 2:
        each = [math.sqrt(math.fsum(np.square(g).ravel())) if np.isfinite(g).all()
                else float(np.sqrt(np.sum(np.square(g)))) for g in grads]
        each = [e * inv_scale for e in each]
        norm = math.sqrt(math.fsum(e * e for e in each)) if np.isfinite(each).all() else float(np.sum(each))
    else:
        each = [float(np.max(np.abs(g))) * inv_scale if g.size else 0.0 for g in grads]
        norm = float(np.max(each)) if each else 0.0
    if not math.isfinite(norm):
        return norm, math.nan, each
    bound = math.inf if norm + eps == 0 else max_norm / (norm + eps)
    return norm, inv_scale * min(1.0, bound), each


def adamw(p, g, m, v, step, lr, betas, eps, weight_decay, grad_scale=1.0):
    """(p, m, v) after the step-th update of float64 arrays."""
    b1, b2 = betas
    g = g * grad_scale
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    update = (m / (1 - b1 ** step)) / (np.sqrt(v / (1 - b2 ** step)) + eps)
    return (1 - lr * weight_decay) * p - lr * update, m, v
