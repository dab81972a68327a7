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
