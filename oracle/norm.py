"""Residual RMSNorm and its gradient, in fp64 numpy.

    h = x + r,  rstd = (mean h^2 + eps)^(-1/2),  y = h rstd w
    dx = rstd (g - xh mean(g xh)) + dh  with g = dy w, xh = h rstd
    dw = sum over rows of dy xh

Inputs are arrays of any float type, read as fp64; nothing is rounded.
"""
import numpy as np


def add_rmsnorm(x, w, r=None, eps=1e-6):
    """(h, y, rstd)"""
    h = np.asarray(x, np.float64)
    if r is not None:
        h = h + np.asarray(r, np.float64)
    rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, h * rstd[:, None] * np.asarray(w, np.float64), rstd


def add_rmsnorm_backward(dy, h, rstd, w, dh=None):
    """(dx, dw, mag_dx, mag_dw): the gradients, and the sums of the magnitudes
    of the terms each element is made of (what a rounding error scales with)."""
    dy, h = np.asarray(dy, np.float64), np.asarray(h, np.float64)
    rstd, w = np.asarray(rstd, np.float64)[:, None], np.asarray(w, np.float64)
    xh = h * rstd
    g = dy * w
    dx = rstd * (g - xh * np.mean(g * xh, axis=1, keepdims=True))
    mag = rstd * (np.abs(g) + np.abs(xh) * np.mean(np.abs(g * xh), axis=1, keepdims=True))
    if dh is not None:
        dh = np.asarray(dh, np.float64)
        dx, mag = dx + dh, mag + np.abs(dh)
    return dx, (dy * xh).sum(0), mag, np.abs(dy * xh).sum(0)
