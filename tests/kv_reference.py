"""Plain numpy forms, in 64 bits, of the microscaled cache of keys and values
(test infrastructure; include/sq_kv.h has the definitions), and caches whose
unused places hold what no kernel may let through."""
import math

import numpy as np

from tests import mx_reference as mx

# half a step of each type, relative to the value
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def rotated(x, positions, inv_freq, amplitude, interleaved):
    """x float32 [T, heads, D] -> its rotation, each fp32 operation rounded."""
    r = 2 * len(inv_freq)
    angle = positions.astype(np.float64)[:, None] * inv_freq[None, :]
    c = (np.cos(angle) * amplitude).astype(np.float32)[:, None, :]
    s = (np.sin(angle) * amplitude).astype(np.float32)[:, None, :]
    one = np.arange(r // 2) * (2 if interleaved else 1)
    two = one + (1 if interleaved else r // 2)
    y = x.copy()
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., two] * c + x[..., one] * s
    return y


def quantized(v, fmt):
    """float32 [.., D] -> codes [.., D/2 | D] and scale bytes [.., D/32]."""
    q, e = mx.quantize(v.reshape(-1, v.shape[-1]), fmt)
    return q.reshape(*v.shape[:-1], -1), e.reshape(*v.shape[:-1], -1)


def values(q, e, fmt):
    """float64 values [.., D] of codes and scale bytes (NaN where e is 255, or
    an e4m3 code is a NaN)."""
    if e.size == 0:
        return np.zeros(e.shape[:-1] + (e.shape[-1] * 32,))
    nan = (q & 0x7f) == 0x7f if fmt == mx.E4M3 else np.zeros((), bool)
    q = np.where(nan, 0, q).astype(np.uint8)
    x = mx.decode(q.reshape(-1, q.shape[-1]), e.reshape(-1, e.shape[-1]), fmt).reshape(*e.shape[:-1], -1)
    return np.where(nan, np.nan, x)


class Cache:
    """Sequences' keys and values in pages of no order.  Places that hold no
    token, and pages of no sequence, hold random codes with scales of NaN; the
    table's entries behind a sequence's pages are no pages."""

    def __init__(self, rng, lens, heads, page, dim, fmt, k=None, v=None, spare=2, width=None):
        need = [-(-n // page) for n in lens]
        self.lens, self.heads, self.page, self.dim, self.fmt = list(lens), heads, page, dim, fmt
        self.pages = sum(need) + spare
        size = dim // 2 if fmt == mx.E2M1 else dim
        top = 256 if fmt == mx.E2M1 else 127  # (0x7f is no code of a number)
        shape = (self.pages, heads, page)
        self.kq, self.vq = (rng.integers(0, top, shape + (size,), dtype=np.uint8) for _ in range(2))
        self.ks, self.vs = (np.full(shape + (dim // 32,), 255, np.uint8) for _ in range(2))
        ids = rng.permutation(self.pages)
        width = max(need + [1]) + 1 if width is None else width
        self.table = rng.choice(np.array([-1, -7, self.pages, 2 ** 31 - 1], np.int32), (len(lens), width))
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.k = [rng.standard_normal((n, heads, dim)).astype(np.float32) * 1.5 for n in lens] if k is None else k
        self.v = [rng.standard_normal((n, heads, dim)).astype(np.float32) for n in lens] if v is None else v
        for b in range(len(lens)):
            self.put(b, self.k[b], self.v[b])

    def put(self, b, k, v):
        p, at = self.where(b)
        for held, scales, x in ((self.kq, self.ks, k), (self.vq, self.vs, v)):
            if len(x):
                held[p, :, at], scales[p, :, at] = quantized(x, self.fmt)

    def where(self, b):
        t = np.arange(self.lens[b])
        return self.table[b, t // self.page].astype(np.int64), t % self.page

    def slots(self, b):
        p, at = self.where(b)
        return p * self.page + at

    def read(self, b):
        """float64 keys and values [tokens, heads, D] of sequence b."""
        p, at = self.where(b)
        return (values(self.kq[p, :, at], self.ks[p, :, at], self.fmt),
                values(self.vq[p, :, at], self.vs[p, :, at], self.fmt))

    def arrays(self):
        return self.kq, self.ks, self.vq, self.vs


def seen(n_q, n_k, causal, window):
    """[n_q, n_k]: which keys each query sees."""
    p = (n_k - n_q + np.arange(n_q))[:, None]
    j = np.arange(n_k)[None, :]
    m = (j <= p) if causal else np.ones((n_q, n_k), bool)
    return m & (j > p - window) if window else m


def attention(q, k, v, dt, scale, causal=True, window=0):
    """float64 q [n_q, heads, D], k and v [n_k, kv, D] -> (y, how far a kernel
    may be off).

    The bound, per output: with w the softmax weights and A = sum w |v|
      scores    a sum of D products in fp32, each and the sum's steps rounded,
                then times scale and log2(e) (three roundings): off by at most
                e = (D + 4) 2^-23 scale sum |q k|, so weights by exp(2 e) - 1
      weights   exp2 (2 2^-23), rounded to the type (half a step; in fp16 2^-25
                at least, against a sum of 1 at least), summed and multiplied
                in fp32 over n keys, rescaled and joined: (n + 64) 2^-23
      output    half a step of the type, 2^-25 at least in fp16
    (the matrix cores may keep one bit less than fp32 rounding: 2^-23)"""
    n_q, heads, D = q.shape
    n_k, kv, _ = k.shape
    group, u = heads // kv, HALF_STEP[dt]
    y, tol = np.zeros(q.shape), np.zeros(q.shape)
    see = seen(n_q, n_k, causal, window)
    least = 2.0 ** -25 if dt == "f16" else 0.0
    for h in range(heads):
        kh, vh = k[:, h // group], v[:, h // group]
        # (keys and values that a query does not see do not reach it)
        for i in range(n_q):
            m = see[i]
            if not m.any():
                continue
            ki, vi = kh[m], vh[m]
            s = (ki @ q[i, h]) * scale
            e = (D + 4) * 2.0 ** -23 * abs(scale) * (np.abs(ki) @ np.abs(q[i, h])).max()
            with np.errstate(invalid="ignore"):
                w = np.exp(s - s.max())
                w = w / w.sum()
                y[i, h] = w @ vi
                a = w @ np.abs(vi)
                tol[i, h] = (u + math.expm1(min(2 * e, 1.0)) + (len(s) + 64) * 2.0 ** -23) * a * (1 + u)
                tol[i, h] += u * np.abs(y[i, h]) + least + least * np.abs(vi).sum(axis=0)
    return y, tol
