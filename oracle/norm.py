"""Plain float64 CPU oracle of the residual's addition and the root-mean-square norm in front of the MoE layer (test
infrastructure, like the rest of this package).

    h = x + r,  y = h / sqrt(mean(h^2) + eps) * w,  scale = max |y| / 448 over the row or over 128 columns (1 where that is 0)
"""
from __future__ import annotations

import numpy as np


def add_rms_norm(x: np.ndarray, residual: np.ndarray | None, w: np.ndarray, eps: float):
    """x, residual [T, H] -> (h, y) [T, H] float64."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(w, np.float64)
    return h, y


def act_scales(y: np.ndarray, group: int | None) -> np.ndarray:
    """[T, 1] or [T, H / group] float64 scales of the rows' values for e4m3 codes."""
    T, H = y.shape
    most = np.abs(y.reshape(T, -1, group or H)).max(axis=2)
    return np.where(most > 0, most / 448.0, 1.0)
