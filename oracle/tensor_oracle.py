"""Oracle of the tensor-list operators: gradient norm, AdamW over a list with
float32 or 8-bit states, and the 8-bit form.  TEST INFRASTRUCTURE ONLY, plain
numpy, sharing no code with the HIP library.

The AdamW arithmetic is zero_oracle's (float64, one IEEE operation at a
time), on g = raw * (coef / L).  The 8-bit form is written from its
definition, in powers and floors on float64:

* a block is 32 consecutive elements (the last one of an array may be
  short); its scale is 2^(e - 127) with the smallest e >= 1 that keeps the
  largest magnitude within 448 scales, and e = 255 if an element is inf or
  NaN (every code of the block is then NaN);
* an element is y = |x| / scale rounded to e4m3: steps of 2^(k - 3) for
  2^k <= y < 2^(k + 1), and of 2^-9 below 2^-6; nearest with ties to even, or
  floor(y / step + R / 2^20) steps with 20 random bits R;
* at the scale 2^120 y is at most 240 (256 * 2^120 would be inf in fp32);
* a root is fp32(sqrt(x)), and one that is positive keeps y >= 2^-9.
"""
from __future__ import annotations

import math

import numpy as np

from . import zero_oracle as zo

F32, F64 = np.float32, np.float64
M32 = 0xFFFFFFFF


def _mix(x, k):
    x = np.asarray(x, dtype=np.uint64)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0xACE5F457)) & np.uint64(M32)
    x = ((x ^ (x >> np.uint64(15)) ^ np.uint64(k)) * np.uint64(0x7B639EB3)) & np.uint64(M32)
    return x ^ (x >> np.uint64(16))


def random_words(n: int, seed: int, step: int, flat_off: int = 0) -> np.ndarray:
    """The 32-bit words of elements 0..n-1 of a tensor at a step."""
    k1 = int(_mix(int(_mix(int(_mix(step & M32, 0)) ^ (seed >> 32) & M32, 0)) ^ (seed & M32), 0))
    k2 = int(_mix(k1 ^ M32, 0))
    c = (np.uint64(flat_off) + np.arange(n, dtype=np.uint64)) & np.uint64(M32)
    return _mix(c ^ np.uint64(k1), k2)


def _codes_of(y, sign):
    """e4m3 code of non-negative float64 values that are e4m3 values."""
    k = np.floor(np.log2(np.maximum(y, 2.0 ** -6))).astype(np.int64)
    mant = np.round(y * 2.0 ** (3 - k)).astype(np.int64)  # 8..15, or below 8 for a subnormal
    code = np.where(mant >= 8, ((k + 7) << 3) + mant - 8, mant)
    return (code | (sign.astype(np.int64) << 7)).astype(np.uint8)


def code_values() -> np.ndarray:
    """The 256 values of e4m3 (OCP: no infinities, 0x7F and 0xFF are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e.astype(F64) - 10), m * 2.0 ** -9)
    v[(c & 0x7F) == 0x7F] = np.nan
    return np.where(c & 0x80, -v, v)


def mx8_encode(x, root: bool = False, words=None, taken: bool = False):
    """float32 array -> (codes uint8[n], scale bytes uint8[ceil(n/32)]); words
    None rounds to nearest.  taken: x are the roots themselves."""
    x = np.asarray(x, dtype=F32)
    n = x.size
    with np.errstate(invalid="ignore"):
        x = np.sqrt(x) if root and not taken else x
    pad = -n % 32
    b = np.concatenate([x, np.zeros(pad, F32)]).reshape(-1, 32).astype(F64)
    bad = ~np.isfinite(b).all(axis=1)
    big = np.abs(np.where(np.isfinite(b), b, 0.0)).max(axis=1, initial=0.0)
    e = np.ones(big.size, dtype=np.int64)
    some = big > 0
    e[some] = np.maximum(1, np.ceil(np.log2(big[some] / 448.0)).astype(np.int64) + 127)
    # log2 may err by an ulp next to a power of two
    e += big > 448.0 * 2.0 ** (e - 127.0)
    down = (e > 1) & (big <= 448.0 * 2.0 ** (e - 128.0))
    e -= down
    y = np.abs(np.where(bad[:, None], 0.0, b)) / 2.0 ** (e - 127.0)[:, None]
    if root:
        y = np.where(b > 0, np.maximum(y, 2.0 ** -9), y)
    y = np.where((e == 247)[:, None], np.minimum(y, 240.0), y)  # 256 * 2^120 is no float32
    step = 2.0 ** (np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    if words is None:
        y = np.round(y / step) * step  # ties to even
    else:
        w = np.concatenate([np.asarray(words, dtype=np.uint64), np.zeros(pad, np.uint64)]).reshape(-1, 32)
        r = (w & np.uint64(0xFFFF)) * np.uint64(16) if root else w >> np.uint64(12)
        y = np.floor(y / step + r.astype(F64) * 2.0 ** -20) * step
    codes = _codes_of(y, np.signbit(b))
    codes[bad] = 0x7F
    e[bad] = 255
    return codes.reshape(-1)[:n], e.astype(np.uint8)


def mx8_decode(codes, scales, root: bool = False) -> np.ndarray:
    """float32 values of codes and scale bytes (squares for a root)."""
    codes, scales = np.asarray(codes), np.asarray(scales)
    s = 2.0 ** (scales.astype(F64) - 127)
    s[scales == 255] = np.nan
    with np.errstate(over="ignore", under="ignore", invalid="ignore"):
        x = (code_values()[codes] * np.repeat(s, 32)[:codes.size]).astype(F32)
        return x * x if root else x


def raw_grad(g) -> np.ndarray:
    """A gradient array's values in float64 (bfloat16 comes as uint16 bits)."""
    g = np.asarray(g)
    if g.dtype == np.uint16:
        g = (g.astype(np.uint32) << np.uint32(16)).view(F32)
    return g.astype(F64)


def grad_norm(grads, loss_scale: float):
    """(overflow, sum g^2) of a list; the sum is exact over the raw squares,
    then scaled."""
    inv = zo._inverse(loss_scale)
    with np.errstate(over="ignore", invalid="ignore"):
        parts = [raw_grad(g) for g in grads]
        finite = all(np.isfinite(x).all() for x in parts)
        total = math.fsum(float(v) for x in parts for v in x * x) if finite else math.inf
        total = total * inv * inv if not (total == 0 and math.isinf(inv)) else math.nan
    return (not math.isfinite(total)), total


class TensorAdam:
    """The list's step: masters (float32), states as float32 arrays or as
    (codes, scales) pairs, one control block."""

    def __init__(self, masters, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0,
                 stochastic=True, seed=0, flat_offs=None):
        self.p = [np.array(x, dtype=F32) for x in masters]
        self.bits, self.stochastic, self.seed = state_bits, stochastic, seed
        self.hp = (lr, beta1, beta2, eps, weight_decay)
        self.offs = flat_offs or list(np.cumsum([0] + [x.size for x in self.p[:-1]]))
        self.m = [self._enc(np.zeros(x.size, F32), False, None) for x in self.p]
        self.v = [self._enc(np.zeros(x.size, F32), True, None) for x in self.p]
        self.t, self.b1p, self.b2p = 0, 1.0, 1.0

    def _enc(self, x, root, words):
        return mx8_encode(x, root, words) if self.bits == 8 else x

    def _step8(self, i, g, sc, words):
        """In float64 throughout, rounded to fp32 at the end; the root of a
        variance past fp32's range is that of the float64 value."""
        m = mx8_decode(*self.m[i]).astype(F64)
        v = mx8_decode(*self.v[i]).astype(F64) ** 2
        p, m, v = zo.adam_update(self.p[i].astype(F64), m, v, g, sc)
        r = np.sqrt(v.astype(F32))
        past = np.isinf(r)
        r[past] = np.sqrt(v[past]).astype(F32)
        return p.astype(F32), mx8_encode(m.astype(F32), False, words), mx8_encode(r, True, words, taken=True)

    def step(self, grads, loss_scale=1.0, coef=1.0):
        sc = zo.step_scalars(*self.hp, self.b1p, self.b2p)
        factor = coef * (1.0 / loss_scale)
        with np.errstate(all="ignore"):
            for i, g in enumerate(grads):
                g = raw_grad(g).reshape(-1) * factor
                if self.bits == 32:
                    self.p[i], self.m[i], self.v[i] = zo.adam_update(self.p[i], self.m[i], self.v[i], g, sc)
                    continue
                w = random_words(g.size, self.seed, self.t + 1, int(self.offs[i])) if self.stochastic else None
                self.p[i], self.m[i], self.v[i] = self._step8(i, g, sc, w)
        self.t, self.b1p, self.b2p = self.t + 1, sc["b1t"], sc["b2t"]
