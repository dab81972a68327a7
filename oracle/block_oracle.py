"""CPU oracle (numpy, fp64) of the operators around the grouped linear layer.

The RMS norm with the residual's addition, the activations that the grouped
products apply in their epilogue, and a whole mixture-of-experts layer, each
written from its formula and sharing no code with the CUDA path.  Test
infrastructure only.
"""
from __future__ import annotations

import math
from typing import Optional

import numpy as np

from . import gl_oracle as orc


# ------------------------------------------------------------------- RMS norm

def rmsnorm(x: np.ndarray, residual: Optional[np.ndarray], gamma: np.ndarray, eps: float):
    """(s, rstd, y): s = x + residual, y = s / sqrt(mean(s^2) + eps) * gamma."""
    s = np.asarray(x, dtype=np.float64)
    if residual is not None:
        s = s + residual
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return s, rstd, s * rstd[:, None] * gamma


def rmsnorm_bwd(dy: np.ndarray, s: np.ndarray, gamma: np.ndarray, rstd: np.ndarray,
                dsum: Optional[np.ndarray]):
    """(dx, dgamma) of :func:`rmsnorm` for the gradients of y and of s."""
    xh = s * rstd[:, None]
    g = dy * gamma
    dx = rstd[:, None] * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    if dsum is not None:
        dx = dx + dsum
    return dx, np.sum(dy * xh, axis=0)


# ---------------------------------------------------------------- activations

ACTS = ("none", "relu", "relu2", "gelu", "silu", "swiglu", "geglu")
GATED = {"swiglu": "silu", "geglu": "gelu"}


def act(name: str, u: np.ndarray) -> np.ndarray:
    """An activation of the last dimension (gated ones halve it)."""
    u = np.asarray(u, dtype=np.float64)
    if name == "none":
        return u
    if name == "relu":
        return np.maximum(u, 0)
    if name == "relu2":
        return np.maximum(u, 0) ** 2
    if name == "gelu":
        return 0.5 * u * (1 + np.tanh(math.sqrt(2 / math.pi) * (u + 0.044715 * u ** 3)))
    if name == "silu":
        return u * 0.5 * (1 + np.tanh(0.5 * u))
    F = u.shape[-1] // 2
    return act(GATED[name], u[..., :F]) * u[..., F:]


def slope(name: str, u: np.ndarray) -> np.ndarray:
    """Derivative of an activation of one argument (0 for relu at 0)."""
    u = np.asarray(u, dtype=np.float64)
    if name == "none":
        return np.ones_like(u)
    if name == "relu":
        return (u > 0).astype(np.float64)
    if name == "relu2":
        return 2 * np.maximum(u, 0)
    if name == "silu":
        q = 0.5 * (1 + np.tanh(0.5 * u))
        return q + u * q * (1 - q)
    c = math.sqrt(2 / math.pi)
    t = np.tanh(c * (u + 0.044715 * u ** 3))
    return 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * c * (1 + 3 * 0.044715 * u * u)


def act_bwd(name: str, z: np.ndarray, dh: np.ndarray) -> np.ndarray:
    """Gradient of an activation's input for the gradient of its output."""
    if name not in GATED:
        return dh * slope(name, z)
    F = z.shape[-1] // 2
    g, u = z[..., :F], z[..., F:]
    return np.concatenate([dh * u * slope(GATED[name], g), dh * act(GATED[name], g)], axis=-1)


def fwd_act(x, w, bias, m_splits, name: str, residual: Optional[np.ndarray]):
    """(y, u): the grouped product u, and act(u) + residual."""
    u = orc.fwd(x, w, bias, m_splits)
    y = act(name, u)
    return (y if residual is None else y + residual), u


def dgrad_act(dy, w, m_splits, name: str, z: np.ndarray) -> np.ndarray:
    """Gradient of the pre-activations z behind the grouped product's input."""
    return act_bwd(name, z, orc.dgrad(dy, w, m_splits))


# ------------------------------------------ a mixture-of-experts layer, few tokens

def route(x: np.ndarray, router: np.ndarray, k: int, renorm: bool):
    """(idx, w, logits): the k largest of softmax(x router^T), lower index first where equal."""
    logits = x @ router.T
    p = np.exp(logits - logits.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    idx = np.argsort(-p, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, idx, axis=1)
    if renorm:
        w = w / w.sum(axis=1, keepdims=True)
    return idx, w, logits


def experts(x: np.ndarray, idx: np.ndarray, w: np.ndarray, w1, w2, name: str) -> np.ndarray:
    """sum_i w[t, i] * W2_e act(W1_e x_t), e = idx[t, i] (-1: none)."""
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        for i in range(idx.shape[1]):
            e = int(idx[t, i])
            if e >= 0:
                y[t] += w[t, i] * (w2[e] @ act(name, w1[e] @ x[t]))
    return y
