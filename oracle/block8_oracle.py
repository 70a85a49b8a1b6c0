"""Oracle of the 8-bit layer operators: the form with a scale for each block of
128, the root-mean-square norm with its gradients, and the product.  TEST
INFRASTRUCTURE ONLY, plain numpy in float64, sharing no code with the HIP
library.

* a block is 128 consecutive values of a row, or 128 x 128 values; its scale
  is 2^(e - 127) with the smallest e >= 1 that keeps the largest magnitude
  within 448 scales, and e = 255 if a value is inf or NaN (every code of the
  block is then NaN);
* a value over its scale is rounded to e4m3, to nearest with ties to even; at
  the scale 2^120 it is at most 240.
"""
from __future__ import annotations

import numpy as np

from .tensor_oracle import _codes_of, code_values

F32, F64 = np.float32, np.float64
B = 128


def blocks_of(n: int) -> int:
    return -(-n // B)


def _blocked(x, tiles: bool):
    r, c = x.shape
    h = B if tiles else 1
    full = np.zeros((-(-r // h) * h, blocks_of(c) * B), x.dtype)
    full[:r, :c] = x
    return full.reshape(-(-r // h), h, blocks_of(c), B)


def encode(x, tiles: bool = False):
    """A matrix -> (codes uint8 [r, c], scale bytes uint8 [r or tiles, blocks])."""
    x = np.asarray(x, F64)
    r, c = x.shape
    y = _blocked(x, tiles)
    bad = ~np.isfinite(y).all(axis=(1, 3))
    y = np.where(np.isfinite(y), y, 0.0)
    top = np.abs(y).max(axis=(1, 3), initial=0.0)
    # frexp: top = m 2^k with 0.5 <= m < 1; 448 = 0.875 * 2^9
    m, k = np.frexp(top)
    e = np.where(top > 0, k - 9 + (m > 0.875), -200) + 127
    e = np.clip(e, 1, 247)
    y = y / np.exp2(e - 127.0)[:, None, :, None]
    y = np.where((e == 247)[:, None, :, None], np.clip(y, -240.0, 240.0), y)
    u = np.abs(y)
    step = np.exp2(np.floor(np.log2(np.maximum(u, 2.0 ** -6))) - 3)
    codes = _codes_of(np.round(u / step) * step, np.signbit(y))
    codes = np.where(bad[:, None, :, None], np.uint8(0x7F), codes)
    e = np.where(bad, 255, e).astype(np.uint8)
    return np.ascontiguousarray(codes.reshape(-1, y.shape[2] * B)[:r, :c]), e


def decode(codes, e):
    """The float64 values that codes and scale bytes stand for (blocks by the
    scales' shape)."""
    r, c = codes.shape
    s = np.where(e == 255, np.nan, np.exp2(e.astype(F64) - 127.0))
    if e.shape[0] != r:
        s = np.repeat(s, B, axis=0)[:r]
    return code_values()[codes] * np.repeat(s, B, axis=1)[:, :c]


def rstd(h, eps):
    with np.errstate(over="ignore", invalid="ignore"):
        return 1.0 / np.sqrt(np.square(np.asarray(h, F64)).mean(axis=1) + eps)


def normed(h, rstd32, w):
    """y in fp32, one operation at a time."""
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        return (np.asarray(h, F32) * np.asarray(rstd32, F32)[:, None]) * np.asarray(w, F32)


def norm_backward(dy, h, w, rstd32, dh=None):
    """(dx, dw) in float64, with the rstd that the norm stored."""
    dy, h, w, r = (np.asarray(a, F64) for a in (dy, h, w, rstd32))
    xh, g = h * r[:, None], dy * w
    dx = (g - xh * (g * xh).mean(axis=1, keepdims=True)) * r[:, None]
    return (dx if dh is None else dx + np.asarray(dh, F64)), (dy * xh).sum(axis=0)


def product(a, b, add=None):
    out = a @ b.T
    return out if add is None else out + np.asarray(add, F64)
