"""The paged 4-bit key/value cache in 64-bit NumPy, from its definition: E2M1
codes with one E8M0 exponent for 32 channels (OCP microscaling MXFP4), the
block layout, the position rotation, and causal attention.  It shares no code
with the GPU path; its own pins are in tests/test_kv_cpu.py.

A cache is a uint8 array [n_pages, H, P, 17 D / 16]; every function takes one
sequence at a time and walks over its tokens.
"""
from __future__ import annotations

import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E_MIN, E_MAX, POISON = 2, 252, 255


def encode(x):
    """(codes, exponents) of x [..., D], one code a channel."""
    x = np.asarray(x, np.float64)
    blocks = x.reshape(*x.shape[:-1], -1, 32)
    most = np.abs(blocks).max(-1)
    with np.errstate(divide="ignore"):
        e = np.where(most > 0, np.frexp(most)[1] - 1, -10000) - 2 + 127
    e = np.clip(e, E_MIN, E_MAX)
    a = np.abs(blocks) / np.exp2(e - 127.0)[..., None]
    # the nearest magnitude; of two at the same distance the even code
    dist = np.abs(np.minimum(a, 6.0)[..., None] - MAGNITUDES)
    code = np.argmin(dist + 1e-300 * (np.arange(8) % 2), -1)
    tie = dist == dist.min(-1, keepdims=True)
    both = tie.sum(-1) == 2
    even = np.argmax(tie & (np.arange(8) % 2 == 0), -1)
    code = np.where(both, even, code)
    code = code + 8 * ((blocks < 0) & (code > 0))
    return code.reshape(x.shape).astype(np.uint8), e.astype(np.uint8)


def decode(codes, exps):
    """Values of codes [..., D] with exponents [..., D / 32]; NaN for 255."""
    c = np.asarray(codes).astype(int)
    x = np.where(c & 8, -1.0, 1.0) * MAGNITUDES[c & 7]
    s = np.where(np.asarray(exps) == POISON, np.nan, np.exp2(np.asarray(exps, np.float64) - 127.0))
    return x * np.repeat(s, 32, -1)


class Block:
    """The four arrays of one (page, head) block, as views of its bytes."""

    def __init__(self, raw):
        P, width = raw.shape
        D = width * 16 // 17
        flat = raw.reshape(-1)
        self.kc = flat[:P * D // 2].reshape(P, D // 2)
        self.vc = flat[P * D // 2:P * D].reshape(P, D // 2)
        self.ke = flat[P * D:P * D + P * D // 32].reshape(P, D // 32)
        self.ve = flat[P * D + P * D // 32:].reshape(D // 32, P)

    @staticmethod
    def _pack(c):
        return (c[0::2] | (c[1::2] << 4)).astype(np.uint8)

    @staticmethod
    def _unpack(b):
        return np.stack([b & 15, b >> 4], -1).reshape(-1)

    def store(self, row, k, v):
        """One token of float64 key and value channels."""
        if np.isfinite(k).all() and np.isfinite(v).all():
            kc, ke = encode(k)
            vc, ve = encode(v)
        else:
            n = k.shape[0]
            kc = vc = np.zeros(n, np.uint8)
            ke, ve = np.full(n // 32, POISON, np.uint8), np.full(n // 32, E_MIN, np.uint8)
        self.kc[row], self.ke[row] = self._pack(kc), ke
        self.vc[row], self.ve[:, row] = self._pack(vc), ve

    def load(self, row):
        return decode(self._unpack(self.kc[row]), self.ke[row]), decode(self._unpack(self.vc[row]), self.ve[:, row])


def rotate(x, cos, sin, interleaved):
    """x [..., D] (64 bits) turned by one position's cos, sin [r / 2]."""
    x = np.array(x, np.float64)
    half = cos.shape[0]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    cos, sin = cos.astype(np.float64), sin.astype(np.float64)
    xa, xb = x[..., a].copy(), x[..., b].copy()
    with np.errstate(invalid="ignore"):
        x[..., a] = xa * cos - xb * sin
        x[..., b] = xb * cos + xa * sin
    return x


def append(pool, table, past, k, v, q=None, cos=None, sin=None, interleaved=False):
    """Stores tokens k, v [n, H, D] of one sequence behind its `past` ones;
    returns the turned q [n, Hq, D] in 64 bits."""
    P = pool.shape[2]
    none = np.zeros(0)
    out = None if q is None else np.array(q, np.float64)
    for i in range(k.shape[0]):
        p = past + i
        c, s = (none, none) if cos is None else (cos[p], sin[p])
        for h in range(k.shape[1]):
            Block(pool[table[p // P], h]).store(p % P, rotate(k[i, h], c, s, interleaved), np.array(v[i, h], np.float64))
        if q is not None:
            out[i] = rotate(q[i], c, s, interleaved)
    return out


def read(pool, table, first, n):
    """Cached keys and values [n, H, D] of positions first .. first + n - 1."""
    P, H, D = pool.shape[2], pool.shape[1], pool.shape[3] * 16 // 17
    k, v = np.empty((n, H, D)), np.empty((n, H, D))
    for i in range(n):
        for h in range(H):
            k[i, h], v[i, h] = Block(pool[table[(first + i) // P], h]).load((first + i) % P)
    return k, v


def attend(k, v, q, past, scale):
    """Causal attention of rows q [n, Hq, D] at positions past + i over cached
    k, v [T, H, D].  Returns the outputs and, for error bounds, the largest
    sum of |q_c k_c| |scale| a row sees [n, Hq] and the largest |v| [n, Hq]."""
    n, heads, D = q.shape
    group = heads // k.shape[1]
    out, mass, most = np.zeros(q.shape), np.zeros((n, heads)), np.zeros((n, heads))
    for i in range(n):
        seen = past + i + 1
        for h in range(heads):
            kk, vv, x = k[:seen, h // group], v[:seen, h // group], q[i, h].astype(np.float64)
            s = kk @ x * scale
            w = np.exp(s - s.max()) if np.isfinite(s).all() else np.full(seen, np.nan)
            out[i, h] = w @ vv / w.sum()
            mass[i, h] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
            most[i, h] = np.abs(vv).max()
    return out, mass, most
