"""The alpha sweep's microscaled modes: on the plain forms (CPU), and the same
sweep through the kernels against it (GPU)."""
import numpy as np
import pytest

import alpha_sweep
import oracle
import synth
from tests import mx_reference as ref


class PlainBackend:
    def absmax(self, a):
        return oracle.absmax_cols(a)

    def scales(self, x_amax, w_amax, alpha, static):
        return oracle.compute_scales(x_amax, w_amax, alpha, static=static)

    def mx_layer(self, x, w, s, inv_s, mode):
        fmt = ref.E4M3 if mode == alpha_sweep.MXFP8 else ref.E2M1
        wq = ref.quantize(ref.smoothed(w, s), ref.E2M1)
        xq = ref.quantize(ref.smoothed(x, inv_s), fmt)
        return (ref.product(*xq, fmt, *wq)[0], ref.decode(*xq, fmt), ref.decode(*wq, ref.E2M1))

    def rows(self, t, idx):
        return t[idx]


ALPHAS = [None, 0.0, 0.5, 1.0]


def _layer(M=64, K=256, N=192):
    X, W, _ = synth.linear_layer(11, M, N, K, 2, 25.0, 40.0, 0.03)
    return X, W


@pytest.mark.parametrize("mode", [alpha_sweep.MXFP8, alpha_sweep.MXFP4])
def test_plain_sweep(mode):
    rows = alpha_sweep.mx_sweep(*_layer(), ALPHAS, mode, PlainBackend(), sample_rows=64)
    assert [r["alpha"] for r in rows] == ["none", 0.0, 0.5, 1.0]
    by = {r["alpha"]: r for r in rows}
    assert by[0.0]["w_ratio"] == pytest.approx(1.0, rel=1e-5)
    assert by[1.0]["x_ratio"] == pytest.approx(1.0, rel=1e-5)
    for r in rows:
        # 0 is a value of both formats, so a nearest (or saturated) value is
        # never further from z than z is from 0: |q - z| <= |z|, element by
        # element, and so for any weighted norm.
        assert 0 < r["w_err"] <= 1 and 0 < r["x_err"] <= 1
        assert np.isfinite(r["y_err"]) and r["y_err"] > 0
    assert alpha_sweep.markdown(rows, "t").count("\n| ") == 5


@pytest.mark.gpu
@pytest.mark.parametrize("mode", [alpha_sweep.MXFP8, alpha_sweep.MXFP4])
def test_gpu_sweep_matches_plain_sweep(mode):
    """Codes are the same bits given the same factors; the factors may differ in
    their last places (a power in double on either side), which moves few codes:
    the errors agree to 1e-3."""
    X, W = _layer(M=128, K=1024, N=512)
    print(f"[gpu-case] mx sweep {mode}", flush=True)
    got = alpha_sweep.mx_sweep(X, W, ALPHAS, mode, alpha_sweep.GpuBackend(), sample_rows=64)
    want = alpha_sweep.mx_sweep(X, W, ALPHAS, mode, PlainBackend(), sample_rows=64)
    for g, w in zip(got, want):
        assert g["alpha"] == w["alpha"]
        for k in ("y_err", "x_err", "w_err", "x_zero", "w_zero", "x_ratio", "w_ratio"):
            assert g[k] == pytest.approx(w[k], rel=1e-3, abs=1e-6), (g["alpha"], k)


@pytest.mark.gpu
def test_command_runs():
    print("[gpu-case] alpha_sweep --mode mxfp4", flush=True)
    assert alpha_sweep.main(["--config", "single_1024", "--mode", "mxfp4", "--alphas", "0.5",
                             "--json"]) == 0
