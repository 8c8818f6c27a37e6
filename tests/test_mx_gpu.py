"""GPU parity of the microscaled operators (include/sq_mx.h) with their plain
64-bit forms (tests/mx_reference.py).

Codes and scale bytes are bit-exact: every step of the quantizer is exact or
one fp32 rounding that the definition names.  The norm's statistics are
double sums in another order; they reach the codes only through mu and rstd
rounded to fp32, so they may differ where a double result lies within about
2^-38 of an fp32 rounding border (chance 2^-14 a row at the very worst, and
inputs are fixed): codes are compared bit for bit.

Products: a scaled instruction adds up to 128 terms and rounds each to no
worse than c of the largest (c = 2^-20 with e2m1 activations, 2^-9 with e4m3);
its largest term is at most the sum over its blocks of their largest.  Each of
the at most K / 64 + 16 additions to an fp32 sum rounds by at most 2^-24 of
the sum of |terms|.  So
    |y - exact| <= c sum_blocks max|t| + (K / 64 + 16) 2^-24 sum|t|
                   + u_out |exact| (1 + 2^-8)
with u_out the output's half step (2^-24, 2^-11, 2^-8), and 2^-25 more for
fp16 (half its subnormal step).
"""
import ctypes

import numpy as np
import pytest

import synth
import w8a8_post_quantization_amd as sq
from tests import mx_reference as ref
from tests.gpu_util import assert_bits_equal, dev, host, log, to_bf16_bits

pytestmark = pytest.mark.gpu

FMT = {"e2m1": sq.SQ_MX_E2M1, "e4m3": sq.SQ_MX_E4M3}


@pytest.fixture(scope="module")
def torch():
    import torch as _t

    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    sq.lib()
    return _t


def _cast(a, dt):
    return a if dt == "f32" else a.astype(np.float16) if dt == "f16" else to_bf16_bits(a)


def _acts(seed, M, K, dt, special=True):
    """Normal rows with a few large channels; special rows at the front where
    there is room: zeros, tiny, one block of equal values, ties, powers of
    two and their neighbours, the type's largest, an infinity, a NaN."""
    a = synth.normal(seed, 1, (M, K)).astype(np.float32)
    cols = synth.choose(seed, 2, K, max(1, K // 500))
    a[:, cols] *= np.float32(40.0)
    if special and M >= 9:
        a[0] = 0
        a[0, ::2] = -0.0
        a[1] *= np.float32({"f32": 1e-42, "f16": 1e-7, "bf16": 1e-39}[dt])
        a[2] = 3.0
        a[3] = np.resize(np.array([5, 0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 7, 7.5, 4, 6, 1, 0.5],
                                  np.float32), K)
        a[4] = np.ldexp(1.0, np.arange(K) % 20 - 10)
        a[5] = np.nextafter(np.ldexp(np.float32(1.0), np.arange(K) % 12).astype(np.float32),
                            np.float32(0))
        top = 6e4 if dt == "f16" else 3e38
        a[6] = np.clip(a[6].astype(np.float64) * (top / 4), -top, top)
        a[7, K // 2] = np.inf
        a[8, K - 1] = np.nan
    return _cast(a, dt)


def _pos(seed, stream, n):
    return (np.abs(synth.normal(seed, stream, (n,))) * 2 + 0.05).astype(np.float32)


def _codes(seed, rows, K, fmt, spread=0, nan_at=None):
    """Random codes (every one of the format) and scale bytes 127 +- spread."""
    rng = np.random.default_rng(seed)
    if fmt == ref.E2M1:
        q = rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)
    else:
        q = rng.integers(0, 256, (rows, K), dtype=np.uint8)
        q[(q & 127) == 127] ^= 1
    e = (127 + rng.integers(-spread, spread + 1, (rows, K // 32))).astype(np.uint8)
    if nan_at is not None:
        e[nan_at] = 255
    return q, e


# ------------------------------------------------------------------ quantizer

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,K,dt,with_s", [
    (1, 32, "f16", True), (1, 8192, "f16", True), (9, 64, "f32", False), (17, 96, "bf16", True),
    (33, 480, "f16", False), (300, 512, "bf16", True), (256, 7168, "bf16", True),
    (1000, 2080, "f16", True), (4097, 1056, "f32", True), (70, 28672, "f16", False),
    (3, 65536, "bf16", False)])
def test_quantize_parity(torch, M, K, dt, with_s, fmt):
    x = _acts(M + K, M, K, dt)
    inv_s = _pos(M + K, 4, K) if with_s else None
    log(f"quantize_act_mx M={M} K={K} {dt} s={with_s} {fmt}")
    q, e = sq.quantize_act_mx(dev(x, torch), None if inv_s is None else dev(inv_s, torch), FMT[fmt])
    q_o, e_o = ref.quantize(ref.smoothed(x, inv_s), FMT[fmt])
    assert_bits_equal(host(e, torch), e_o, "x_scale")
    assert_bits_equal(host(q, torch), q_o, "xq")


@pytest.mark.parametrize("N,K,dt,with_s,fold", [
    (1, 32, "f32", True, True), (2100, 2048, "f16", True, False), (1000, 4096, "bf16", True, True),
    (37, 2080, "f16", False, True), (513, 96, "f32", True, True), (28672, 256, "f16", False, False),
    (9000, 4096, "f16", True, True)])   # above 64 MB: the streamed form
def test_smooth_weights_parity(torch, N, K, dt, with_s, fold):
    w = _cast(synth.normal(N + K, 1, (N, K)).astype(np.float32) * np.float32(0.03), dt)
    s = _pos(N + K, 3, K) if with_s else None
    r = _pos(N + K, 5, N) if fold else None
    log(f"smooth_weights_mxfp4 N={N} K={K} {dt} s={with_s} fold={fold}")
    q, e = sq.smooth_weights_mxfp4(dev(w, torch), None if s is None else dev(s, torch),
                                   None if r is None else dev(r, torch))
    q_o, e_o = ref.quantize(ref.smoothed(w, s, r), ref.E2M1)
    assert_bits_equal(host(e, torch), e_o, "w_scale")
    assert_bits_equal(host(q, torch), q_o, "wq")


def test_quantize_every_scale(torch):
    """Blocks whose largest value runs over every fp32 exponent (subnormals
    to infinity) with mantissas at and beside the borders."""
    mant = np.array([0, 1, 0x3fffff, 0x400000, 0x600000, 0x700000, 0x7fffff], np.uint32)
    tops = ((np.arange(256, dtype=np.uint32)[:, None] << 23) | mant[None, :]).reshape(-1)
    rng = np.random.default_rng(3)
    v = np.zeros((tops.size, 32), np.float32)
    with np.errstate(all="ignore"):
        v[:] = tops.view(np.float32)[:, None] * rng.uniform(-1, 1, v.shape).astype(np.float32)
    v[:, 13] = tops.view(np.float32)
    for fmt in ("e2m1", "e4m3"):
        log(f"quantize every scale {fmt}")
        q, e = sq.quantize_act_mx(dev(v, torch), None, FMT[fmt])
        q_o, e_o = ref.quantize(v, FMT[fmt])
        assert_bits_equal(host(e, torch), e_o, "scale")
        assert_bits_equal(host(q, torch), q_o, "codes")


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quantize_every_16_bit_value(torch, dt, fmt):
    """All 65536 bit patterns: signed zeros, subnormals, infinities, NaNs."""
    bits = np.arange(1 << 16, dtype=np.uint16).reshape(-1, 32)
    tdt = {"f16": torch.float16, "bf16": torch.bfloat16}[dt]
    x = torch.from_numpy(bits.view(np.int16)).cuda().view(tdt)
    f32 = bits.view(np.float16).astype(np.float32) if dt == "f16" else \
        (bits.astype(np.uint32) << 16).view(np.float32)
    q, e = sq.quantize_act_mx(x, None, FMT[fmt])
    q_o, e_o = ref.quantize(f32, FMT[fmt])
    assert_bits_equal(host(e, torch), e_o, "scales")
    assert_bits_equal(host(q, torch), q_o, "codes")


def test_rows_of_three_dimensions_and_out(torch):
    x = dev(_acts(5, 24, 96, "f16"), torch)
    q, e = sq.quantize_act_mx(x)
    out = (torch.full_like(q, 0xAA), torch.full_like(e, 0xAA))
    got = sq.quantize_act_mx(x.reshape(2, 12, 96), out=out)
    assert got[0] is out[0] and torch.equal(out[0], q) and torch.equal(out[1], e)
    for bad in ((q[:-1], e), (q, e[:, :-1].contiguous()), (q.to(torch.int8), e)):
        with pytest.raises(ValueError):
            sq.quantize_act_mx(x, out=bad)
    with pytest.raises(ValueError):
        sq.quantize_act_mx(x.t())
    with pytest.raises(ValueError):
        sq.quantize_act_mx(x, torch.ones(95, device="cuda"))
    with pytest.raises(ValueError):
        sq.quantize_act_mx(x[:, :80].contiguous())
    with pytest.raises(ValueError):
        sq.quantize_act_mx(x, fmt=3)


# -------------------------------------------------------------------- inverse

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("rows,K,ydt", [(1, 32, "f32"), (7, 96, "f16"), (300, 2080, "bf16"),
                                        (8192, 256, "f32"), (5000, 8192, "f16")])
def test_dequantize_parity(torch, rows, K, ydt, fmt):
    q, e = _codes(rows + K, rows, K, FMT[fmt], spread=30)
    e[0, 0] = 255
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[ydt]
    log(f"dequantize_mx rows={rows} K={K} {ydt} {fmt}")
    y = host(sq.dequantize_mx(dev(q, torch), dev(e, torch), FMT[fmt], tdt), torch)
    q0 = q.copy()
    q0[0, :(16 if fmt == "e2m1" else 32)] = 0
    want = ref.decode(q0, e, FMT[fmt])
    with np.errstate(over="ignore"):
        w32 = want.astype(np.float32)
        w = w32 if ydt == "f32" else w32.astype(np.float16) if ydt == "f16" else to_bf16_bits(w32)
    nan = np.isnan(want)
    assert np.isnan(ref.to_f32(y)[nan]).all() and nan.sum() == 32
    assert_bits_equal(np.where(nan, 0, y).astype(y.dtype), np.where(nan, 0, w).astype(w.dtype), "y")


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_dequantize_every_code_and_scale(torch, fmt):
    """Every code under every scale byte, fp32 and bf16, subnormals kept."""
    codes = np.arange(256, dtype=np.uint8)
    if fmt == "e4m3":
        codes[(codes & 127) == 127] ^= 1
    rows = 256
    per = 512 if fmt == "e2m1" else 256      # elements that 256 code bytes hold
    q = np.tile(codes, (rows, 1))
    e = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, per // 32))
    for tdt in (torch.float32, torch.bfloat16):
        y = ref.to_f32(host(sq.dequantize_mx(dev(q, torch), dev(e, torch), FMT[fmt], tdt), torch))
        want = ref.decode(q, e, FMT[fmt])
        with np.errstate(over="ignore"):
            w = want.astype(np.float32)
            if tdt == torch.bfloat16:
                w = ref.to_f32(to_bf16_bits(np.where(np.isnan(w), 0, w)))
        assert np.isnan(y[255]).all()
        assert_bits_equal(y[:255], w[:255], f"values {tdt}")


# ----------------------------------------------------------------------- norm

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,K,dt,layer,beta", [
    (1, 32, "f16", True, True), (8, 8192, "bf16", False, False), (3, 96, "f32", True, False),
    (65, 2080, "f16", True, True), (257, 1024, "bf16", True, False), (5, 16384, "f16", True, True),
    (7, 16384, "f32", False, True), (1030, 4096, "f16", False, False), (2050, 7168, "f16", True, True),
    (1500, 1056, "f32", True, True), (1100, 2048, "bf16", False, True), (4100, 512, "f16", True, False),
    (1025, 10240, "bf16", True, True), (4097, 4128, "f16", True, True), (4100, 8192, "bf16", False, True),
    (4096, 7168, "f16", True, False)])
def test_norm_parity(torch, M, K, dt, layer, beta, fmt):
    a = synth.normal(M + K, 1, (M, K)).astype(np.float32) * np.float32(2) + np.float32(0.25)
    a[:, synth.choose(M + K, 2, K, 2)] *= np.float32(60)
    a[0, 0] = 500.0                        # the pivot is an outlier
    if M > 4:
        a[1] += 3000.0                     # a mean far above the spread
        a[2] = 0.0
        a[3] = 1.5                         # a constant row
        a[4, 1:] = 0.0
    x = _cast(a, dt)
    g = (1 + 0.1 * synth.normal(M + K, 20, (K,))).astype(np.float32)
    b = (0.05 * synth.normal(M + K, 21, (K,))).astype(np.float32) if beta else None
    log(f"norm_quantize_act_mx M={M} K={K} {dt} layer={layer} beta={beta} {fmt}")
    q, e = sq.norm_quantize_act_mx(dev(x, torch), dev(g, torch), None if b is None else dev(b, torch),
                                   sq.SQ_NORM_LAYER if layer else sq.SQ_NORM_RMS, 1e-5, FMT[fmt])
    q_o, e_o = ref.quantize(ref.norm(x, g, b, layer, 1e-5), FMT[fmt])
    assert_bits_equal(host(e, torch), e_o, "x_scale")
    assert_bits_equal(host(q, torch), q_o, "xq")


def test_norm_rows_that_are_not_finite(torch):
    """A NaN or infinity in a row makes the row's statistics and with them all
    of its blocks NaN; the other rows keep their codes.  eps = 0 on a zero row
    divides 0 by 0."""
    K = 1056
    x = synth.normal(3, 1, (6, K)).astype(np.float16)
    g = dev(np.ones(K, np.float32), torch)
    q0, e0 = sq.norm_quantize_act_mx(dev(x, torch), g)
    x[1, 700] = np.nan
    x[3, 0] = np.inf
    x[5] = 0
    q, e = sq.norm_quantize_act_mx(dev(x, torch), g, eps=0.0)
    q1, e1 = sq.norm_quantize_act_mx(dev(x, torch), g)
    for r in (1, 3, 5):
        assert (host(e, torch)[r] == 255).all() and not host(q, torch)[r].any()
    for r in (0, 2, 4):
        assert_bits_equal(host(e1, torch)[r], host(e0, torch)[r], "scale of a finite row")
        assert_bits_equal(host(q1, torch)[r], host(q0, torch)[r], "codes of a finite row")


@pytest.mark.parametrize("M", [5, 700])
def test_rms_rows_with_an_infinity(torch, M):
    """sigma^2 is infinite and rstd 0: an infinity's block is NaN (inf * 0), the
    row's other elements are beta."""
    K = 1056
    x = synth.normal(4, 1, (M, K)).astype(np.float32)
    x[2, 700], x[4, 33], x[4, 64] = np.inf, -np.inf, np.inf
    g, b = np.ones(K, np.float32), np.linspace(-3, 5, K).astype(np.float32)
    log(f"norm_quantize_act_mx RMS with infinities M={M}")
    for beta in (None, b):
        q, e = sq.norm_quantize_act_mx(dev(x, torch), dev(g, torch), None if beta is None else dev(b, torch),
                                       sq.SQ_NORM_RMS, 1e-5)
        with np.errstate(invalid="ignore"):
            q_o, e_o = ref.quantize(ref.norm(x, g, beta, False, 1e-5), ref.E2M1)
        assert (e_o[2] == 255).sum() == 1 and (e_o[4] == 255).sum() == 2
        assert_bits_equal(host(e, torch), e_o, "x_scale")
        assert_bits_equal(host(q, torch), q_o, "xq")


# -------------------------------------------------------------------- product

UNIT = {ref.E2M1: 2.0 ** -20, ref.E4M3: 2.0 ** -9}
U_OUT = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _check_product(y, ydt, xq, xs, fmt, wq, ws):
    exact, total, top = ref.product(xq, xs, fmt, wq, ws)
    K = xs.shape[1] * 32
    got = ref.to_f32(y).astype(np.float64)
    nan = np.isnan(exact)
    assert np.array_equal(np.isnan(got), nan), "NaN where a scale is NaN, nowhere else"
    tol = UNIT[fmt] * top + (K / 64 + 16) * 2.0 ** -24 * total + U_OUT[ydt] * np.abs(exact) * (1 + 2.0 ** -8)
    if ydt == "f16":
        tol = tol + 2.0 ** -25
        over = np.abs(exact) + tol >= 65504    # may round to an infinity
        assert not over.any(), "the test's values stay inside fp16"
    err = np.abs(got - exact)[~nan]
    tol = tol[~nan]
    worst = float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0
    acc = float((np.abs(got - exact)[~nan] / np.maximum(top[~nan], 1e-300)).max()) if err.size else 0.0
    assert worst <= 1, f"worst error / bound {worst}"
    return worst, acc


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K,ydt,spread", [
    (1, 1, 32, "f32", 0), (1, 16, 128, "f32", 3), (5, 1001, 2080, "f16", 1), (8, 4096, 8192, "bf16", 2),
    (16, 520, 1024, "f32", 20), (17, 100, 96, "f32", 3), (32, 3000, 4096, "bf16", 2),
    (32, 11163, 1024, "f16", 0), (33, 1000, 256, "f32", 3), (77, 129, 160, "f32", 5),
    (64, 256, 128, "f32", 0), (100, 300, 512, "bf16", 3), (257, 384, 2048, "f32", 3),
    (300, 520, 1056, "f16", 1), (513, 640, 384, "f32", 3), (1030, 1100, 640, "f32", 2),
    (256, 2050, 7168, "bf16", 1), (2, 70000, 64, "f32", 3), (3000, 7, 224, "f32", 3)])
def test_product_parity(torch, M, N, K, ydt, spread, fmt):
    f = FMT[fmt]
    xq, xs = _codes(M * 3 + K, M, K, f, spread)
    if f == ref.E4M3:
        xs = (xs - 7).astype(np.uint8)       # values near the e2m1 ones
    wq, ws = _codes(N * 5 + K, N, K, ref.E2M1, spread)
    if ydt == "f16":
        ws = (ws - 6).astype(np.uint8)
    if M > 2 and N > 2:                      # a NaN scale in the last block of a row and a column
        xs[1, -1] = 255
        ws[2, 0] = 255
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[ydt]
    log(f"gemm_mxfp4 M={M} N={N} K={K} y={ydt} {fmt} spread={spread}")
    args = [dev(a, torch) for a in (xq, xs, wq, ws)]
    y = sq.gemm_mxfp4(*args, f, out_dtype=tdt)
    y2 = sq.gemm_mxfp4(*args, f, out_dtype=tdt)
    yh = host(y, torch)
    worst, acc = _check_product(yh, ydt, xq, xs, f, wq, ws)
    nan = np.isnan(ref.to_f32(yh))
    assert_bits_equal(np.where(nan, 0, host(y2, torch)), np.where(nan, 0, yh), "the same bits again")
    print(f"\ngemm_mxfp4 {fmt} M={M} N={N} K={K}: worst error / bound {worst:.3f}, error / largest terms {acc:.2g}")


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("tile", [0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K,ydt", [
    (40, 100, 256, "f32"), (300, 333, 384, "bf16"), (513, 520, 512, "f32"), (33, 260, 640, "f16"),
    (129, 1030, 1152, "f32"), (256, 256, 1280, "bf16"), (700, 130, 4224, "f32"),
    (200, 300, 288, "f32"), (65, 129, 800, "bf16"), (140, 270, 1056, "f16"), (300, 200, 2272, "f32")])
def test_product_tiles(torch, M, N, K, ydt, tile, fmt):
    """Every block shape of the pipelined kernel: fewer stages than its ring,
    as many and more, with and without a last partial stage, scale rows that
    start at any byte (K % 128 != 0), ragged edges."""
    f = FMT[fmt]
    xq, xs = _codes(M * 7 + K, M, K, f, 1)
    if f == ref.E4M3:
        xs = (xs - 7).astype(np.uint8)
    wq, ws = _codes(N * 9 + K, N, K, ref.E2M1, 1)
    if ydt == "f16":
        ws = (ws - 6).astype(np.uint8)
    xs[3, K // 32 - 1] = 255
    ws[N - 1, K // 32 - 5] = 255
    tdt = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[ydt]
    log(f"gemm_mxfp4 tile={tile} M={M} N={N} K={K} y={ydt} {fmt}")
    y = sq.gemm_mxfp4(*[dev(a, torch) for a in (xq, xs, wq, ws)], f, out_dtype=tdt, tile=tile)
    _check_product(host(y, torch), ydt, xq, xs, f, wq, ws)


# Decode (M <= 32): every window width, windows past K, several windows a
# wave, one to eight groups of rows a block and more than one round of blocks.
@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [
    (1, 5000, 992), (4, 20000, 544), (16, 33000, 1024), (31, 9000, 1056), (2, 13000, 1984),
    (9, 300, 4064), (20, 26000, 2080), (7, 70000, 352), (3, 7001, 6016), (32, 12345, 8224),
    (1, 100, 20000), (17, 40, 40000), (12, 4500, 16416)])
def test_product_decode(torch, M, N, K, fmt):
    f = FMT[fmt]
    xq, xs = _codes(M * 13 + K, M, K, f, 1)
    if f == ref.E4M3:
        xs = (xs - 7).astype(np.uint8)
    wq, ws = _codes(N * 17 + K, N, K, ref.E2M1, 1)
    xs[M - 1, K // 64] = 255 if M > 3 else xs[M - 1, K // 64]
    ws[N - 1, K // 32 - 1] = 255
    log(f"gemm_mxfp4 decode M={M} N={N} K={K} {fmt}")
    d = [dev(a, torch) for a in (xq, xs, wq, ws)]
    y = host(sq.gemm_mxfp4(*d, f, out_dtype=torch.float32), torch)
    n = np.unique(np.r_[0:min(N, 700), max(0, N - 700):N, N // 2:min(N, N // 2 + 300)])
    _check_product(y[:, n], "f32", xq, xs, f, wq[n], ws[n])


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(3, 50, 160), (40, 70, 96), (130, 140, 256)])
def test_product_writes_its_rows_only(torch, M, N, K, fmt):
    """Guard rows before and after y, and an odd first element (y needs only
    its element's alignment)."""
    f = FMT[fmt]
    xq, xs = _codes(7, M, K, f, 1)
    wq, ws = _codes(8, N, K, ref.E2M1, 1)
    L, P = sq.lib(), lambda t: t.data_ptr()  # noqa: E731
    args = [dev(a, torch) for a in (xq, xs, wq, ws)]
    for tdt, code in ((torch.float32, sq.SQ_F32), (torch.bfloat16, sq.SQ_BF16)):
        want = sq.gemm_mxfp4(*args, f, out_dtype=tdt)
        buf = torch.full((M * N + 2001,), 123.0, dtype=tdt, device="cuda")
        y = buf[1001:1001 + M * N]
        log(f"product guard M={M} N={N} K={K} {fmt} {tdt}")
        rc = L.sq_gemm_mxfp4(P(args[0]), P(args[1]), f, P(args[2]), P(args[3]), M, N, K, P(y), code,
                             ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
        assert rc == 0
        torch.cuda.synchronize()
        assert torch.equal(y.reshape(M, N), want)
        assert (buf[:1001] == 123).all() and (buf[1001 + M * N:] == 123).all()


@pytest.mark.parametrize("rows,K", [(5, 96), (3, 480), (130, 544)])
def test_quantizers_write_their_rows_only(torch, rows, K):
    L, P = sq.lib(), lambda t: t.data_ptr()  # noqa: E731
    x = dev(synth.normal(9, 1, (rows, K)).astype(np.float16), torch)
    g = torch.ones(K, device="cuda")
    sp = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    for fmt, per in ((0, 2), (1, 1)):
        nq, ns = rows * K // per, rows * K // 32
        for form in ("act", "norm"):
            q = torch.full((nq + 512,), 0xA5, dtype=torch.uint8, device="cuda")
            s = torch.full((ns + 512,), 0xA5, dtype=torch.uint8, device="cuda")
            log(f"quantizer guard {form} rows={rows} K={K} fmt={fmt}")
            if form == "act":
                rc = L.sq_quantize_act_mx(P(x), sq.SQ_F16, rows, K, P(g), fmt, P(q[256:]), P(s[256:]), sp)
            else:
                rc = L.sq_norm_quantize_act_mx(P(x), sq.SQ_F16, rows, K, 1, P(g), None, 1e-5, fmt,
                                               P(q[256:]), P(s[256:]), sp)
            assert rc == 0
            torch.cuda.synchronize()
            for t, n in ((q, nq), (s, ns)):
                assert (t[:256] == 0xA5).all() and (t[256 + n:] == 0xA5).all()
        y = torch.full((rows * K + 512,), 55.0, dtype=torch.float32, device="cuda")
        rc = L.sq_dequantize_mx(P(q[256:]), P(s[256:]), fmt, rows, K, P(y[256:]), sq.SQ_F32, sp)
        assert rc == 0
        torch.cuda.synchronize()
        assert (y[:256] == 55).all() and (y[256 + rows * K:] == 55).all()


# ---------------------------------------------------------------- a run of them

def _layer(torch, M, H, F, fmt, seed):
    """Weights and inputs of norm -> gate|up -> product of halves -> down."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (rnd(M, H) * 2).to(torch.float16)
    w1, w2 = (rnd(2 * F, H) * 0.03).to(torch.float16), (rnd(H, F) * 0.03).to(torch.float16)
    s1, s2 = rnd(H).abs() + 0.5, rnd(F).abs() + 0.5
    gamma, _ = sq.fold_norm(1 + 0.1 * rnd(H), s1)
    q1, q2 = sq.smooth_weights_mxfp4(w1, s1), sq.smooth_weights_mxfp4(w2, s2)
    inv2 = 1.0 / s2

    def run():
        a = sq.norm_quantize_act_mx(x, gamma, None, sq.SQ_NORM_RMS, 1e-5, fmt)
        h = sq.gemm_mxfp4(*a, *q1, fmt, out_dtype=torch.float32)
        h = h[:, :F] * h[:, F:]
        b = sq.quantize_act_mx(h, inv2, fmt)
        y = sq.gemm_mxfp4(*b, *q2, fmt, out_dtype=torch.bfloat16)
        return [*a, h, *b, y]

    return run, (x, gamma, q1, q2, inv2)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M", [1, 5, 32, 200])
def test_layer_eager_stream_and_graph(torch, M, fmt):
    """norm -> product -> quantize -> product as a layer calls them: each step
    against its plain form on the step's own inputs; the same bits on another
    stream and from a captured graph, replay after replay with eager work of
    the same layer between."""
    H, F = 512, 800
    f = FMT[fmt]
    run, (x, gamma, q1, q2, inv2) = _layer(torch, M, H, F, f, M)
    log(f"layer M={M} {fmt}")
    xq, xs, h, hq, hs, y = eager = run()
    torch.cuda.synchronize()
    hst = lambda t: host(t, torch)  # noqa: E731
    q_o, e_o = ref.quantize(ref.norm(hst(x), hst(gamma), None, False, 1e-5), f)
    assert_bits_equal(hst(xq), q_o, "xq")
    assert_bits_equal(hst(xs), e_o, "x_scale")
    q_o, e_o = ref.quantize(ref.smoothed(hst(h), hst(inv2)), f)
    assert_bits_equal(hst(hq), q_o, "hq")
    assert_bits_equal(hst(hs), e_o, "h_scale")
    _check_product(hst(y), "bf16", hst(hq), hst(hs), f, hst(q2[0]), hst(q2[1]))

    want = [hst(t).copy() for t in eager]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = run()
    s.synchronize()
    for t, w in zip(other, want):
        assert_bits_equal(hst(t), w, "another stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        outs = run()
    for r in range(4):
        for t in outs:
            t.zero_()
        again = run()                          # eager work between the replays
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for t, u, w in zip(outs, again, want):
            assert_bits_equal(hst(t), w, f"replay {r}")
            assert_bits_equal(hst(u), w, f"eager beside replay {r}")


def test_first_call_inside_a_capture(torch):
    """A variant that nothing before has launched (and whose grid size is asked
    of the runtime on its first call) captured before it ever ran eagerly."""
    M, K = 700, 2080
    x = dev(_cast(synth.normal(41, 1, (M, K)).astype(np.float32), "bf16"), torch)
    g = torch.rand(K, device="cuda") + 0.5
    b = torch.rand(K, device="cuda") - 0.5
    out = (torch.zeros((M, K), dtype=torch.uint8, device="cuda"),
           torch.zeros((M, K // 32), dtype=torch.uint8, device="cuda"))
    log("norm_quantize_act_mx first called in a capture")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        sq.norm_quantize_act_mx(x, g, b, sq.SQ_NORM_RMS, 1e-5, sq.SQ_MX_E4M3, out=out)
    q_o, e_o = ref.quantize(ref.norm(host(x, torch), host(g, torch), host(b, torch), False, 1e-5), ref.E4M3)
    for _ in range(3):
        out[0].zero_(), out[1].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert_bits_equal(host(out[1], torch), e_o, "x_scale")
        assert_bits_equal(host(out[0], torch), q_o, "xq")


def test_two_streams_at_once(torch):
    """No call has state of its own: the same and other calls interleaved on two
    streams give each the bits they give alone."""
    f = sq.SQ_MX_E4M3
    runs = [_layer(torch, M, 512, 800, f, M)[0] for M in (7, 200)]
    want = [[host(t, torch).copy() for t in run()] for run in runs]
    streams = [torch.cuda.Stream() for _ in runs]
    torch.cuda.synchronize()
    log("two streams at once")
    got = [[], []]
    for _ in range(5):
        for i, (run, s) in enumerate(zip(runs, streams)):
            with torch.cuda.stream(s):
                got[i].append(run())
    torch.cuda.synchronize()
    for i in range(2):
        for outs in got[i]:
            for t, w in zip(outs, want[i]):
                assert_bits_equal(host(t, torch), w, f"stream {i}")


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_short_inner_length_many_rows(torch, fmt):
    """K < 256 takes slabs of 32 tokens: more of them than a grid's second
    dimension could count."""
    f = FMT[fmt]
    M, N, K = 65536 * 32 + 5, 3, 32
    xq, xs = _codes(77, M, K, f, 1)
    wq, ws = _codes(78, N, K, ref.E2M1, 1)
    log(f"gemm_mxfp4 M={M} N={N} K={K} {fmt}")
    y = host(sq.gemm_mxfp4(*[dev(a, torch) for a in (xq, xs, wq, ws)], f, out_dtype=torch.float32), torch)
    rows = np.r_[0:100, M - 100:M, np.random.default_rng(1).integers(0, M, 500)]
    _check_product(y[rows], "f32", xq[rows], xs[rows], f, wq, ws)


def test_past_four_gigabytes(torch):
    """Codes, values and outputs whose offsets pass 2^32 bytes: the last rows
    against their plain forms."""
    K, M = 8192, 270000                       # bf16 x: 4.4 GB, e4m3 codes 2.2 GB
    log(f"quantize and decode M={M} K={K}")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    tail = dev(_acts(90, 64, K, "bf16"), torch)
    x[-64:] = tail
    q, e = sq.quantize_act_mx(x, None, sq.SQ_MX_E4M3)
    q_o, e_o = ref.quantize(ref.smoothed(host(tail, torch)), ref.E4M3)
    assert_bits_equal(host(q[-64:], torch), q_o, "codes")
    assert_bits_equal(host(e[-64:], torch), e_o, "scales")
    y = sq.dequantize_mx(q, e, sq.SQ_MX_E4M3, out_dtype=torch.bfloat16)
    want = sq.dequantize_mx(q[-64:].contiguous(), e[-64:].contiguous(), sq.SQ_MX_E4M3,
                            out_dtype=torch.bfloat16)
    assert torch.equal(y[-64:].view(torch.int16), want.view(torch.int16))
    nq, ne = sq.norm_quantize_act_mx(x, torch.ones(K, device="cuda"), None, sq.SQ_NORM_RMS, 1e-5)
    nq1, ne1 = sq.norm_quantize_act_mx(tail, torch.ones(K, device="cuda"), None, sq.SQ_NORM_RMS, 1e-5)
    assert torch.equal(nq[-64:], nq1) and torch.equal(ne[-64:], ne1)
    del x, y, nq, ne
    w = sq.smooth_weights_mxfp4(torch.randn(8200, K, device="cuda", dtype=torch.bfloat16))
    finite = torch.where((e == 255).any(dim=1, keepdim=True), torch.zeros_like(e), e)
    log(f"gemm_mxfp4 M={M} N=8200 K={K}")
    for tile in range(4):   # (a tile adds in one order, wherever its rows are)
        y = sq.gemm_mxfp4(q, finite, *w, sq.SQ_MX_E4M3, out_dtype=torch.bfloat16, tile=tile)  # 4.4 GB
        want = sq.gemm_mxfp4(q[-64:].contiguous(), finite[-64:].contiguous(), *w, sq.SQ_MX_E4M3,
                             out_dtype=torch.bfloat16, tile=tile)
        assert torch.equal(y[-64:].view(torch.int16), want.view(torch.int16))
        assert not y[:-64].any()


def test_explicit_stream(torch):
    x = dev(_acts(6, 40, 256, "f16"), torch)
    want = sq.quantize_act_mx(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = sq.quantize_act_mx(x, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_layer_error_against_the_unquantized_product(torch):
    """Smoothed 4-bit weights: with 8-bit activations the layer's error is the
    weights' alone (each off by at most 1/8 of its binade: normal weights come
    out near 0.11 relative), and 4-bit activations about double its square."""
    M, N, K = 64, 256, 2048
    X = synth.activations(3, 1, M, K, synth.choose(3, 3, K, 4), np.full(4, 30.0))
    W = synth.weights(3, 2, N, K, 0.03)
    x, w = dev(X, torch), dev(W, torch)
    s, inv = sq.compute_scales(sq.absmax_reduce(x), sq.absmax_reduce(w), 0.5)
    wq, ws = sq.smooth_weights_mxfp4(w, s)
    want = X.astype(np.float64) @ W.astype(np.float64).T
    err = {}
    for name, f in FMT.items():
        y = sq.gemm_mxfp4(*sq.quantize_act_mx(x, inv, f), wq, ws, f, out_dtype=torch.float32)
        err[name] = np.linalg.norm(host(y, torch) - want) / np.linalg.norm(want)
    print(f"\nlayer error against fp64: e4m3 {err['e4m3']:.3f}, e2m1 {err['e2m1']:.3f}")
    # a value is off by at most a quarter of the block's largest binade edge,
    # never by more than its block's largest value: well under one in the norm
    assert err["e4m3"] < 0.25 and err["e2m1"] < 0.5


def test_rows_are_never_copied(torch):
    """Inputs of more dimensions are viewed as rows; where that would take a copy
    (on the current stream, whatever the call's own) the call is refused."""
    g = torch.ones(64, device="cuda")
    x = torch.randn(4, 6, 64, device="cuda")
    q, e = sq.quantize_act_mx(x)
    q1, e1 = sq.quantize_act_mx(x.reshape(24, 64))
    assert torch.equal(q, q1) and torch.equal(e, e1)
    for bad in (x[:, ::2], x.transpose(0, 1), x[..., :32]):
        with pytest.raises(ValueError, match="contiguous"):
            sq.quantize_act_mx(bad)
        with pytest.raises(ValueError, match="contiguous"):
            sq.norm_quantize_act_mx(bad, g)


def test_empty_calls(torch):
    z = lambda *s: torch.empty(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    q, e = sq.quantize_act_mx(x)
    assert q.shape == (0, 32) and e.shape == (0, 2)
    q, e = sq.norm_quantize_act_mx(x, torch.ones(64, device="cuda"), fmt=sq.SQ_MX_E4M3)
    assert q.shape == (0, 64)
    assert sq.dequantize_mx(z(0, 32), z(0, 2)).shape == (0, 64)
    w = sq.smooth_weights_mxfp4(torch.randn(5, 64, device="cuda"))
    assert sq.gemm_mxfp4(z(0, 32), z(0, 2), *w).shape == (0, 5)
    assert sq.gemm_mxfp4(*w, z(0, 32), z(0, 2)).shape == (5, 0)
    with pytest.raises(sq.SQError):
        sq.gemm_mxfp4(z(3, 0), z(3, 0), z(4, 0), z(4, 0))
    with pytest.raises(ValueError):
        sq.gemm_mxfp4(z(3, 32), z(3, 2), z(4, 64), z(4, 4))
    with pytest.raises(ValueError):
        sq.gemm_mxfp4(z(3, 32), z(2, 2), *w)
