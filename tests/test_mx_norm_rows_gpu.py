"""Rows at which the statistics of the norm -> MX kernels (sq_norm_quantize_act_mx)
change their form: rows of one value, and rows on both sides of the switch
between one pass over a row and two (mu^2 = 256 sigma^2).  Codes and scales bit
for bit against the 64-bit form, in the block- and the wave-per-row kernel and
with rows spread over several waves.
"""
import numpy as np
import pytest

import synth
import w8a8_post_quantization_amd as sq
from tests import mx_reference as ref
from tests.gpu_util import assert_bits_equal, dev, host, log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    import torch as _t

    if not _t.cuda.is_available():
        pytest.fail("GPU tests need a GPU")
    sq.lib()
    return _t


def _check(torch, x, K, beta, eps, what):
    g = (1 + 0.1 * synth.normal(K, 20, (K,))).astype(np.float32)
    b = (0.05 * synth.normal(K, 21, (K,))).astype(np.float32) if beta else None
    log(f"norm_quantize_act_mx {what} M={len(x)} K={K} beta={beta} eps={eps}")
    q, e = sq.norm_quantize_act_mx(dev(x, torch), dev(g, torch), None if b is None else dev(b, torch),
                                   sq.SQ_NORM_LAYER, eps)
    with np.errstate(divide="ignore", invalid="ignore"):
        q_o, e_o = ref.quantize(ref.norm(x, g, b, True, eps), ref.E2M1)
    assert_bits_equal(host(e, torch), e_o, "x_scale")
    assert_bits_equal(host(q, torch), q_o, "xq")
    return e_o


# (M, K, beta): few rows; a wave, two and four waves a row; the wave-per-row
# kernel (M >= 4096 with a beta, 4096 < K <= 8192)
SHAPES = [(9, 1568, False), (9, 5152, True), (600, 1568, True), (600, 3136, False), (600, 5152, False),
          (4100, 5152, True), (4100, 7168, True)]


@pytest.mark.parametrize("M,K,beta", SHAPES)
def test_rows_of_one_value(torch, M, K, beta):
    """sigma^2 is 0 whatever K: with eps = 0 every element is 0 * inf, a NaN."""
    x = synth.normal(M + K, 1, (M, K)).astype(np.float16)
    values = np.array([1.5, -0.1, 1000.0, 6e-8, 3.0, 0.7], np.float16)
    x[1:7] = values[:, None]
    x[-1] = 1.5
    e = _check(torch, x, K, beta, 0.0, "rows of one value")
    assert (e[1:7] == 255).all() and (e[-1] == 255).all() and not (e[7:-1] == 255).any()
    _check(torch, x, K, beta, 1e-5, "rows of one value")


@pytest.mark.parametrize("M,K,beta", SHAPES)
def test_rows_beside_the_switch(torch, M, K, beta):
    a = synth.normal(M + K, 2, (M, K)).astype(np.float64)
    a = (a - a.mean(axis=1, keepdims=True)) / a.std(axis=1, keepdims=True)
    ratio = np.resize(np.array([0.0, 200.0, 255.0, 255.99, 256.01, 257.0, 1e4, 1e6, 1e8]), M)
    x = (a + np.sqrt(ratio)[:, None]).astype(np.float32)
    if beta and M > 4096:
        x = x.astype(np.float16)             # (the wave-per-row kernel's type)
    _check(torch, x, K, beta, 1e-5, "rows beside the switch")
