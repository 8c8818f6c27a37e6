"""Plain numpy forms of the microscaled operators in 64 bits (test
infrastructure; include/sq_mx.h has the definitions).  fp32 roundings that
the definitions name are taken with numpy's float32; everything else is
float64, where each value here is exact."""
import numpy as np

E2M1, E4M3 = 0, 1
BLOCK = 32
GRID = {
    E2M1: np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64),
    # code 0x00 .. 0x7E of e4m3: 2^-9 m below 2^-6, else (8 + m) 2^(x - 10)
    E4M3: np.array([m * 2.0 ** -9 for m in range(8)]
                   + [(8 + m) * 2.0 ** (x - 10) for x in range(1, 16) for m in range(8)][:-1],
                   np.float64),
}
TOP_EXP = {E2M1: 2, E4M3: 8}


def to_f32(a):
    """A test array (uint16: bfloat16 bits) as float32."""
    if a.dtype == np.uint16:
        return (a.astype(np.uint32) << 16).view(np.float32)
    return a.astype(np.float32)


def nearest(z, fmt):
    """Codes (sign apart) of |z|: the nearest grid value, ties to the even
    code, beyond the largest to it.  z float64."""
    grid = GRID[fmt]
    mid = (grid[1:] + grid[:-1]) / 2
    lo = np.searchsorted(mid, z, side="left")    # midpoints below z
    hi = np.searchsorted(mid, z, side="right")   # midpoints up to z
    return np.where((lo != hi) & (hi % 2 == 0), hi, lo)


def quantize(v, fmt):
    """fp32 rows [R, K] -> (codes, scale bytes) as the library lays them out."""
    v = np.asarray(v, np.float32)
    R, K = v.shape
    b = v.reshape(R, K // BLOCK, BLOCK)
    bad = ~np.isfinite(b).all(axis=2)
    a = np.abs(np.where(bad[:, :, None], 0, b).astype(np.float64)).max(axis=2)
    _, p = np.frexp(a)                            # a = f 2^p, f in [0.5, 1)
    p = np.where(a >= 2.0 ** -126, p - 1, -127)
    e = np.maximum(p + 127 - TOP_EXP[fmt], 0)
    z = np.where(bad[:, :, None], 0, b).astype(np.float64) * np.exp2(127.0 - e)[:, :, None]
    code = nearest(np.abs(z), fmt)
    sign = np.signbit(np.where(bad[:, :, None], 0, b))
    code = (code + sign * (8 if fmt == E2M1 else 128)).astype(np.uint8).reshape(R, K)
    e = np.where(bad, 255, e).astype(np.uint8)
    if fmt == E2M1:
        code = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    return code, e


def decode(q, e, fmt):
    """float64 values of codes and scale bytes (NaN where e is 255)."""
    if fmt == E2M1:
        c = np.empty((q.shape[0], q.shape[1] * 2), np.int64)
        c[:, 0::2], c[:, 1::2] = q & 15, q >> 4
        v = GRID[fmt][c & 7] * np.where(c & 8, -1.0, 1.0)
    else:
        c = q.astype(np.int64)
        assert ((c & 127) < 127).all(), "NaN codes are never produced"
        v = GRID[fmt][c & 127] * np.where(c & 128, -1.0, 1.0)
    s = np.where(e == 255, np.nan, np.exp2(e.astype(np.float64) - 127))
    return (v.reshape(q.shape[0], -1, BLOCK) * s[:, :, None]).reshape(v.shape)


def smoothed(x, mul=None, row_mul=None):
    """fl(fl(x * row_mul[r]) * mul[k]) in fp32."""
    v = to_f32(x)
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        if row_mul is not None:
            v = v * row_mul[:, None].astype(np.float32)
        if mul is not None:
            v = v * mul[None, :].astype(np.float32)
    return v


def norm(x, gamma, beta, layer, eps):
    """The norm's fp32 output, statistics in float64 (two passes)."""
    x32 = to_f32(x)
    w = x32.astype(np.float64)
    mean = w.mean(axis=1, keepdims=True) if layer else np.zeros((len(w), 1))
    var = ((w - mean) ** 2).mean(axis=1, keepdims=True)
    rstd = (1.0 / np.sqrt(var + np.float64(np.float32(eps)))).astype(np.float32)
    y = x32 - mean.astype(np.float32) if layer else x32
    y = (y * rstd) * gamma[None, :]
    return y if beta is None else y + beta[None, :]


def product(xq, xs, x_fmt, wq, ws):
    """(y, sum of |terms|, sum over blocks of the largest |term|), float64."""
    x, w = decode(xq, xs, x_fmt), decode(wq, ws, E2M1)
    y, total = x @ w.T, np.abs(x) @ np.abs(w).T
    M, K = x.shape
    top = np.zeros_like(y)
    for b in range(0, K, BLOCK):
        xb, wb = np.abs(x[:, b:b + BLOCK]), np.abs(w[:, b:b + BLOCK])
        step = max(1, (1 << 22) // (BLOCK * len(wb)))
        for m in range(0, M, step):
            top[m:m + step] += (xb[m:m + step, None, :] * wb[None]).max(axis=2)
    return y, total, top
