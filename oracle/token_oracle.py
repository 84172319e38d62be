"""Float64 CPU oracle for the token operators around the attention branches:
layer norm, rotary positions over three axes, and 8-bit checkpoints.

TEST INFRASTRUCTURE ONLY.  Nothing in the product path may import, call or
execute this module: only ``tests/`` and ``__graft_entry__.smoke()`` use it.
It shares no code, constant or helper with the CUDA library.

Everything is float64.  The 8-bit format is written down as the set of values
that a code can stand for, and a value goes to the nearest of them.
"""

from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_backward", "rope", "rope_grid", "checkpoint", "checkpoint_values", "BLOCK"]

BLOCK = 32


def layer_norm(x, w=None, b=None, eps=1e-6):
    """Rows of x normalised: returns y, mean, rstd and the normalised rows."""
    x = np.asarray(x, dtype=np.float64)
    mean = x.mean(-1)
    rstd = 1.0 / np.sqrt(((x - mean[..., None]) ** 2).mean(-1) + eps)
    xh = (x - mean[..., None]) * rstd[..., None]
    y = xh if w is None else xh * np.asarray(w, dtype=np.float64)
    y = y if b is None else y + np.asarray(b, dtype=np.float64)
    return y, mean, rstd, xh


def layer_norm_backward(dy, xh, rstd, w=None):
    """dx, dw, db of sum(dy * y) at the normalised rows xh [rows, D] with rstd [rows]."""
    dy, xh = np.asarray(dy, dtype=np.float64), np.asarray(xh, dtype=np.float64)
    g = dy if w is None else dy * np.asarray(w, dtype=np.float64)
    dx = np.asarray(rstd, dtype=np.float64)[:, None] * (
        g - g.mean(-1, keepdims=True) - xh * (g * xh).mean(-1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def rope_grid(T, height, width, pos0=(0.0, 0.0, 0.0), step=(1.0, 1.0, 1.0)):
    """Positions [T * height * width, 3] of a grid's tokens."""
    out = np.empty((T, height, width, 3))
    for axis, n in enumerate((T, height, width)):
        shape = [1, 1, 1]
        shape[axis] = n
        out[..., axis] = (pos0[axis] + step[axis] * np.arange(n)).reshape(shape)
    return out.reshape(-1, 3)


def rope(x, positions, axes, theta=10000.0, halves=False, inverse=False):
    """x [N, H, d] turned by positions [N, 3]; `axes` channels per axis.  Each pair is a complex number times
    e^(i angle); inverse: e^(-i angle), which is also the gradient's way."""
    x = np.asarray(x, dtype=np.float64)
    pos = np.asarray(positions, dtype=np.float64)
    angles = np.concatenate([pos[:, [a]] * theta ** (-np.arange(0, n, 2) / max(n, 1)) for a, n in enumerate(axes)], 1)
    turn = np.exp((-1j if inverse else 1j) * angles)[:, None, :]
    rot = sum(axes)
    out = x.copy()
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if halves else (slice(0, rot, 2), slice(1, rot, 2))
    with np.errstate(invalid="ignore"):
        z = (x[..., first] + 1j * x[..., second]) * turn
    out[..., first], out[..., second] = z.real, z.imag
    return out


# The magnitudes a code can stand for, by code: 0, 1/512, ..., 448.
_MAGNITUDES = np.array([(m / 8 + (e > 0)) * 2.0 ** (max(e, 1) - 7) for e in range(16) for m in range(8)][:127])


def checkpoint(x):
    """Rows x [rows, D] as (codes uint8 [rows, D], scale bytes uint8 [rows, ceil(D / 32)])."""
    x = np.asarray(x, dtype=np.float64)
    rows, D = x.shape
    codes = np.empty((rows, D), dtype=np.uint8)
    scales = np.empty((rows, -(-D // BLOCK)), dtype=np.uint8)
    for j in range(scales.shape[1]):
        v = x[:, j * BLOCK: (j + 1) * BLOCK]
        fine = np.isfinite(v)
        top = np.where(fine, np.abs(v), 0.0).max(1)
        e = np.full(rows, -127)
        while np.any(short := top > 448.0 * 2.0 ** e):   # the least e that covers the block
            e[short] += 1
        m = np.where(fine, np.abs(v), 0.0) / 2.0 ** e[:, None]
        hi = np.clip(np.searchsorted(_MAGNITUDES, m), 1, 126)
        below, above = m - _MAGNITUDES[hi - 1], _MAGNITUDES[hi] - m
        code = np.where((below < above) | ((below == above) & (hi % 2 == 1)), hi - 1, hi)
        # 256 at the largest exponent would be 2^128, beyond float32: the value below it.
        code = np.where((e == 120)[:, None] & (code > np.searchsorted(_MAGNITUDES, 240.0)),
                        np.searchsorted(_MAGNITUDES, 240.0), code)
        code = np.where(fine, code | np.where(np.signbit(v), 0x80, 0), 0x7F)
        codes[:, j * BLOCK: (j + 1) * BLOCK] = code
        scales[:, j] = e + 127
    return codes, scales


def checkpoint_values(codes, scales):
    """The float64 values that codes and scale bytes stand for."""
    codes = np.asarray(codes)
    m = np.concatenate([_MAGNITUDES, [np.nan]])[codes & 0x7F] * np.where(codes & 0x80, -1.0, 1.0)
    s = 2.0 ** (np.asarray(scales, dtype=np.float64) - 127.0)
    return m * np.repeat(s, BLOCK, axis=1)[:, : codes.shape[1]]
