"""The sums of the microscaled product (include/sq_mx.h) are fp32 sums for both
activation formats: small terms beside large ones are kept.

Exactness.  With all scale bytes 127 every term is a multiple of 2^-10 (e4m3
2^-9 times e2m1 0.5).  Where the terms' magnitudes add up to less than 2^14
every partial sum is a multiple of 2^-10 below 2^14, so it fits fp32's 24 bits,
and an fp32 sum in any order is the exact value.

Scales that differ.  A step of the matrix cores (64 or 128 elements) rounds its
terms to no worse than 2^-20 of the largest; with e4m3 activations a step is two
instructions.  The largest term of a step is at most the sum over its blocks of
their largest, so all steps are off by at most 2^-19 sum_blocks max|t|.  Each
instruction adds to its fp32 sum in up to four pieces, each cut to the sum's
last place: at most 4 * 2^-23 of sum|t|, K / 32 instructions at the most (64
elements in two parts), and 16 more for the join of eight waves' sums:
    |y - exact| <= 2^-19 sum_blocks max|t| + (K / 32 * 8 + 16) 2^-24 sum|t|
                   + 2^-24 |exact|
"""
import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import mx_reference as ref
from tests.gpu_util import dev, host, log

pytestmark = pytest.mark.gpu

FMT = {"e2m1": sq.SQ_MX_E2M1, "e4m3": sq.SQ_MX_E4M3}


@pytest.fixture(scope="module")
def torch():
    import torch as _t

    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    sq.lib()
    return _t


def _small_and_large(seed, M, N, K):
    """e4m3 rows of magnitudes below 2 with few of up to 240 among them (about
    five a row), the first row's also in pairs of opposite sign that cancel;
    e2m1 weights; all scales 1."""
    rng = np.random.default_rng(seed)
    q = rng.integers(0, 64, (M, K)).astype(np.uint8)
    large = rng.random((M, K)) < 5 / K
    q[large] = rng.integers(64, 120, int(large.sum()))
    q |= (rng.integers(0, 2, (M, K)) << 7).astype(np.uint8)
    wq = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    q[0, 0:4], q[0, K - 6:K - 4] = (0x77, 0x01, 0xF7, 0x01), (0x77, 0xF7)
    wq[:, :2] = 0x17                  # weights 6, 0.5, 6, 0.5
    wq[:, K // 2 - 3] = 0x77
    one = lambda r: np.full((r, K // 32), 127, np.uint8)  # noqa: E731
    return q, one(M), wq, one(N)


@pytest.mark.parametrize("M,N,K", [
    # decode: both widths of activations, every window width, several passes
    (1, 100, 64), (1, 5000, 992), (4, 20000, 544), (16, 300, 1984), (9, 13000, 2048), (7, 300, 4064),
    (3, 9000, 4096), (5, 40, 8480), (2, 9000, 8192), (17, 300, 96), (32, 9000, 1056), (20, 40, 2080),
    (31, 9000, 2048), (18, 40, 8224), (32, 9000, 4096), (70, 50, 224)])
def test_small_terms_beside_large_ones(torch, M, N, K):
    _exact(torch, M, N, K, None)


@pytest.mark.parametrize("tile", [None, 0, 1, 2, 3])
@pytest.mark.parametrize("M,N,K", [(40, 100, 256), (130, 260, 384), (257, 300, 1152), (300, 130, 288),
                                   (66, 520, 1056), (129, 257, 4096)])
def test_small_terms_beside_large_ones_tiled(torch, M, N, K, tile):
    _exact(torch, M, N, K, tile)


def _exact(torch, M, N, K, tile):
    xq, xs, wq, ws = _small_and_large(M + 3 * N + K, M, N, K)
    want, total, _ = ref.product(xq, xs, ref.E4M3, wq, ws)
    assert total.max() < 2 ** 14, "the sums fit fp32"
    log(f"gemm_mxfp4 exact sums M={M} N={N} K={K} tile={tile}")
    y = host(sq.gemm_mxfp4(*[dev(a, torch) for a in (xq, xs, wq, ws)], sq.SQ_MX_E4M3,
                           out_dtype=torch.float32, tile=tile), torch)
    bad = np.nonzero(y != want)
    assert bad[0].size == 0, f"{bad[0].size} of {y.size}: {y[bad][:4]} for {want[bad][:4]}"


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("spread", [1, 3, 20])
@pytest.mark.parametrize("M,N,K", [(1, 700, 128), (5, 333, 1024), (16, 100, 4096), (32, 300, 2080), (30, 200, 96),
                                   (70, 300, 256), (200, 300, 1056), (300, 260, 640)])
def test_sums_over_scales_that_differ(torch, M, N, K, spread, fmt):
    f = FMT[fmt]
    rng = np.random.default_rng(M + K + spread)
    xq = rng.integers(0, 256, (M, K // 2 if fmt == "e2m1" else K), dtype=np.uint8)
    if fmt == "e4m3":
        xq[(xq & 127) == 127] ^= 1
    wq = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    xs, ws = ((127 + rng.integers(-spread, spread + 1, (r, K // 32))).astype(np.uint8) for r in (M, N))
    exact, total, top = ref.product(xq, xs, f, wq, ws)
    log(f"gemm_mxfp4 sums M={M} N={N} K={K} spread={spread} {fmt}")
    y = host(sq.gemm_mxfp4(*[dev(a, torch) for a in (xq, xs, wq, ws)], f, out_dtype=torch.float32), torch)
    tol = 2.0 ** -19 * top + (K / 32 * 8 + 16) * 2.0 ** -24 * total + 2.0 ** -24 * np.abs(exact)
    worst = float((np.abs(y - exact) / tol).max())
    print(f"\ngemm_mxfp4 {fmt} M={M} N={N} K={K} spread={spread}: worst error / bound {worst:.3f}")
    assert worst <= 1


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("M,N,K", [(33, 17, 32), (40, 512, 160), (1000, 1100, 64), (1030, 1000, 224), (4099, 300, 128),
                                   (70000, 16, 96), (65, 16500, 192), (2, 40, 224), (16, 33000, 128), (1, 17000, 160),
                                   (31, 17010, 32), (20, 3, 224)])
def test_short_inner_lengths(torch, M, N, K, fmt):
    """K < 256 with many rows: one and two windows, one and two groups of weight
    rows a block, ragged slabs.  All scales 1: e2m1 terms are multiples of 0.25
    and their sums below 36 * 224, so exact in any order, as the e4m3 ones."""
    if fmt == "e4m3":
        _exact(torch, M, N, K, None)
        return
    rng = np.random.default_rng(M + N + K)
    xq, wq = (rng.integers(0, 256, (r, K // 2), dtype=np.uint8) for r in (M, N))
    xs, ws = (np.full((r, K // 32), 127, np.uint8) for r in (M, N))
    want = ref.decode(xq, xs, ref.E2M1) @ ref.decode(wq, ws, ref.E2M1).T
    log(f"gemm_mxfp4 exact sums M={M} N={N} K={K} e2m1")
    y = host(sq.gemm_mxfp4(*[dev(a, torch) for a in (xq, xs, wq, ws)], out_dtype=torch.float32), torch)
    assert np.array_equal(y, want)
