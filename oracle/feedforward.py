"""References of the feed-forward operators in fp64: RMS norm and its backward pass, the
activations with their slopes, a product's epilogue and its backward pass.

    norm:      n = h / sqrt(mean h^2 + eps), y = n w      (h: x, or x + residual in bf16)
    backward:  g = dy w,  dx = rstd (g - n mean(g n)) + dh,  dw = sum over rows of dy n
    epilogue:  y = act(z) + residual, with a gate y = act(z_gate) z_up
    backward:  dz = dy act'(z), with a gate dz_gate = dy z_up act'(z_gate), dz_up = dy act(z_gate)

Records are made by ``nvfp4.quantize`` and ``mxfp4.quantize`` of bf16 values.
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit, ndtr

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def rmsnorm64(h, w, eps):
    """(y, rstd) of fp64 rows h [M, K]."""
    rstd = 1.0 / np.sqrt((h * h).mean(-1) + eps)
    return h * rstd[:, None] * w, rstd


def rmsnorm_bwd64(dy, h, w, rstd, dh=None):
    """(dx, dw, magnitudes of dx's terms, of dw's)."""
    n, g = h * rstd[:, None], dy * w
    c = (g * n).mean(-1, keepdims=True)
    ca = np.abs(g * n).mean(-1, keepdims=True)
    dx = rstd[:, None] * (g - n * c)
    size = rstd[:, None] * (np.abs(g) + np.abs(n) * ca)
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, (dy * n).sum(0), size, np.abs(dy * n).sum(0)


def activation64(name, z):
    """(act(z), act'(z))."""
    z = np.asarray(z, dtype=np.float64)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.maximum(z, 0.0), (z > 0).astype(np.float64)
    if name == "gelu":
        return z * ndtr(z), ndtr(z) + z * np.exp(-0.5 * z * z) / np.sqrt(2 * np.pi)
    zc = np.clip(z, -1e30, 1e30)
    u = zc if name == "silu" else np.sqrt(8 / np.pi) * (zc + 0.044715 * zc ** 3)
    du = 1.0 if name == "silu" else np.sqrt(8 / np.pi) * (1 + 3 * 0.044715 * zc ** 2)
    return z * expit(u), expit(u) + zc * (expit(u) * expit(-u)) * du


def epilogue64(z, name, gated, residual=None):
    if gated:
        half = z.shape[1] // 2
        y = activation64(name, z[:, :half])[0] * z[:, half:]
    else:
        y = activation64(name, z)[0]
    return y if residual is None else y + residual


def epilogue_bwd64(dy, z, name, gated):
    if not gated:
        return dy * activation64(name, z)[1]
    half = z.shape[1] // 2
    f, df = activation64(name, z[:, :half])
    return np.concatenate((dy * z[:, half:] * df, dy * f), 1)
