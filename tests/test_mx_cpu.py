"""Microscaled operators on the CPU: the numpy reference against torch's own
e4m3 / E8M0 types and against values worked by hand, and every refusal of the
C ABI (include/sq_mx.h) and of the Python binding.  No kernel is launched."""
import os

import numpy as np
import pytest

import w8a8_post_quantization_amd as sq
from tests import mx_reference as ref

built = pytest.mark.skipif(not os.path.exists(sq.LIB_PATH),
                           reason="libsq.so not built (run __graft_entry__.build())")
OK, NULL, SHAPE, DTYPE, ALIGN, ARG, WORKSPACE, UNSUP, HIP = range(9)
FAKE = 0x100000  # a 256-aligned non-null address; never dereferenced on these paths


def test_reference_e2m1_by_hand():
    v = np.zeros((1, 32), np.float32)
    # largest 5 = 1.25 2^2: e = 127, codes are the values themselves
    v[0, :12] = [5.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, -0.24, 0.26, 4.9, -5.0, 1.0]
    q, e = ref.quantize(v, ref.E2M1)
    assert e.tolist() == [[127]]
    got = ref.decode(q, e, ref.E2M1)[0, :12].tolist()
    assert got == [4.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 0.0, 0.5, 4.0, -4.0, 1.0]
    # 7.9 = 1.975 2^2 saturates at 6; 8 starts the next exponent
    v[0, 0] = 7.9
    q, e = ref.quantize(v, ref.E2M1)
    assert e[0, 0] == 127 and ref.decode(q, e, ref.E2M1)[0, 0] == 6.0
    v[0, 0] = 8.0
    q, e = ref.quantize(v, ref.E2M1)
    assert e[0, 0] == 128 and ref.decode(q, e, ref.E2M1)[0, 0] == 8.0
    # packing: element 0 in the low nibble
    v[:] = 0
    v[0, 0], v[0, 1] = 6.0, -1.0
    q, _ = ref.quantize(v, ref.E2M1)
    assert q[0, 0] == (0xA << 4 | 0x7) and not q[0, 1:].any()


def test_reference_scale_range():
    for a, want2, want8 in ((0.0, 0, 0), (1e-45, 0, 0), (2.0 ** -126, 0, 0), (2.0 ** -124, 1, 0),
                            (2.0 ** -118, 7, 1), (3.4e38, 252, 246)):
        v = np.zeros((1, 32), np.float32)
        v[0, 7] = -a
        assert ref.quantize(v, ref.E2M1)[1][0, 0] == want2, a
        assert ref.quantize(v, ref.E4M3)[1][0, 0] == want8, a
    for bad in (np.inf, -np.inf, np.nan):
        v = np.ones((1, 64), np.float32)
        v[0, 40] = bad
        for fmt in (ref.E2M1, ref.E4M3):
            q, e = ref.quantize(v, fmt)
            assert e[0, 1] == 255 and e[0, 0] < 255
            d = ref.decode(q, e, fmt)
            assert np.isnan(d[0, 32:]).all() and (d[0, :32] == 1).all()


def test_reference_e4m3_matches_torch():
    torch = pytest.importorskip("torch")
    z = np.concatenate([np.linspace(-448, 448, 20001), np.ldexp(1.0, np.arange(-12, 9)),
                        ref.GRID[ref.E4M3], (ref.GRID[ref.E4M3][1:] + ref.GRID[ref.E4M3][:-1]) / 2])
    z = z.astype(np.float32)
    want = torch.from_numpy(z).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    got = ref.GRID[ref.E4M3][ref.nearest(np.abs(z.astype(np.float64)), ref.E4M3)] * np.sign(z)
    assert np.array_equal(got, want)
    e = np.arange(255, dtype=np.uint8)
    t = torch.from_numpy(e).view(torch.float8_e8m0fnu).to(torch.float32).numpy()
    assert np.array_equal(t.astype(np.float64), np.exp2(e.astype(np.float64) - 127))


def test_reference_relative_error():
    """In a block a value of the largest binade is off by at most a quarter
    (saturation: 8 to 6) in e2m1 and by 2^-4 plus saturation 512 to 448 in
    e4m3."""
    rng = np.random.default_rng(1)
    v = rng.normal(size=(64, 256)).astype(np.float32)
    for fmt, worst in ((ref.E2M1, 2.0 / 8), (ref.E4M3, 64.0 / 512)):
        q, e = ref.quantize(v, fmt)
        d = ref.decode(q, e, fmt)
        top = np.abs(v.reshape(64, 8, 32)).max(axis=2, keepdims=True)
        err = np.abs(d - v).reshape(64, 8, 32) / top
        assert err.max() <= worst


@built
def test_exports_every_declared_symbol():
    L = sq.lib()
    declared = sq.header_functions(sq.MX_HEADER)
    assert declared == ["sq_dequantize_mx", "sq_gemm_mxfp4", "sq_norm_quantize_act_mx",
                        "sq_quantize_act_mx", "sq_smooth_weights_mxfp4"]
    for name in declared:
        assert hasattr(L, name) and name in sq.SIGNATURES, name
    assert sq.header_functions(sq.MX_TEST_HEADER) == ["sq_gemm_mxfp4_tile"]
    assert hasattr(L, "sq_gemm_mxfp4_tile")


@built
def test_quantize_validation():
    f = sq.lib().sq_quantize_act_mx

    def call(x=FAKE, dt=sq.SQ_F16, M=8, K=64, inv=FAKE, fmt=0, q=FAKE, s=FAKE):
        return f(x, dt, M, K, inv, fmt, q, s, None)

    assert call(dt=5) == DTYPE
    assert call(fmt=2) == ARG and call(fmt=-1) == ARG
    for K in (16, 40, -32, 1 << 31):
        assert call(K=K) == SHAPE
    assert call(M=-1) == SHAPE and call(M=1 << 31) == SHAPE
    assert call(K=0, x=None) == SHAPE
    assert call(x=None) == NULL and call(q=None) == NULL and call(s=None) == NULL
    assert call(x=FAKE + 8) == ALIGN and call(q=FAKE + 8) == ALIGN
    assert call(inv=FAKE + 8) == ALIGN and call(s=FAKE + 2) == ALIGN
    assert call(M=0, x=None, q=None, s=None) == OK
    assert call(M=0, K=0, x=None, q=None, s=None) == OK


@built
def test_weights_validation():
    f = sq.lib().sq_smooth_weights_mxfp4

    def call(w=FAKE, dt=sq.SQ_BF16, N=8, K=64, r=FAKE, s=FAKE, q=FAKE, e=FAKE):
        return f(w, dt, N, K, r, s, q, e, None)

    assert call(dt=3) == DTYPE
    assert call(K=48) == SHAPE and call(N=-1) == SHAPE and call(K=0) == SHAPE
    assert call(w=None) == NULL and call(q=None) == NULL and call(e=None) == NULL
    assert call(w=FAKE + 4) == ALIGN and call(r=FAKE + 2) == ALIGN
    assert call(s=FAKE + 4) == ALIGN and call(q=FAKE + 4) == ALIGN and call(e=FAKE + 1) == ALIGN
    assert call(N=0, w=None, q=None, e=None) == OK


@built
def test_norm_validation():
    f = sq.lib().sq_norm_quantize_act_mx

    def call(x=FAKE, dt=sq.SQ_F16, M=8, K=64, norm=0, g=FAKE, b=None, eps=1e-5, fmt=0, q=FAKE,
             s=FAKE):
        return f(x, dt, M, K, norm, g, b, eps, fmt, q, s, None)

    assert call(dt=4) == DTYPE
    assert call(norm=2) == ARG and call(fmt=7) == ARG
    for eps in (-1.0, float("inf"), float("nan")):
        assert call(eps=eps) == ARG
    assert call(K=80) == SHAPE and call(K=0) == SHAPE and call(M=-1) == SHAPE
    assert call(K=16416) == UNSUP
    assert call(x=None) == NULL and call(g=None) == NULL and call(q=None) == NULL
    assert call(s=None) == NULL
    assert call(x=FAKE + 8) == ALIGN and call(g=FAKE + 4) == ALIGN and call(b=FAKE + 4) == ALIGN
    assert call(q=FAKE + 4) == ALIGN and call(s=FAKE + 2) == ALIGN
    assert call(M=0, x=None, g=None, q=None, s=None) == OK


@built
def test_dequantize_validation():
    f = sq.lib().sq_dequantize_mx

    def call(q=FAKE, s=FAKE, fmt=1, rows=8, K=64, y=FAKE, dt=sq.SQ_F32):
        return f(q, s, fmt, rows, K, y, dt, None)

    assert call(dt=9) == DTYPE and call(fmt=2) == ARG
    assert call(K=33) == SHAPE and call(rows=-1) == SHAPE and call(K=0) == SHAPE
    assert call(q=None) == NULL and call(s=None) == NULL and call(y=None) == NULL
    assert call(q=FAKE + 8) == ALIGN and call(s=FAKE + 2) == ALIGN and call(y=FAKE + 4) == ALIGN
    assert call(rows=0, q=None, s=None, y=None) == OK


@built
def test_gemm_validation():
    f = sq.lib().sq_gemm_mxfp4

    def call(x=FAKE, xs=FAKE, fmt=0, w=FAKE, ws=FAKE, M=4, N=4, K=64, y=FAKE, dt=sq.SQ_F32):
        return f(x, xs, fmt, w, ws, M, N, K, y, dt, None)

    assert call(dt=9) == DTYPE and call(fmt=2) == ARG
    assert call(K=48) == SHAPE and call(M=-1) == SHAPE and call(N=-1) == SHAPE
    assert call(K=0) == SHAPE and call(N=1 << 31) == SHAPE
    assert call(M=(1 << 31) - 1) == SHAPE and call(N=(1 << 31) - 1023) == SHAPE
    # tiles past a grid's 2^32 threads: slabs of 32 rows, and tiles of 64 to 256
    assert call(M=(1 << 31) - 1024, K=32) == UNSUP
    assert call(M=(1 << 31) - 1024, N=4096, K=256) == UNSUP
    for name in ("x", "xs", "w", "ws", "y"):
        assert call(**{name: None}) == NULL, name
    assert call(x=FAKE + 8) == ALIGN and call(w=FAKE + 8) == ALIGN
    assert call(xs=FAKE + 2) == ALIGN and call(ws=FAKE + 1) == ALIGN
    assert call(y=FAKE + 2) == ALIGN
    assert call(M=0, x=None, y=None) == OK and call(N=0, w=None, y=None) == OK
    assert call(K=(1 << 20) + 32) == UNSUP
    for bad in (-2, 4):
        assert sq.lib().sq_gemm_mxfp4_tile(FAKE, FAKE, 0, FAKE, FAKE, 64, 64, 256, FAKE, sq.SQ_F32,
                                           None, bad) == ARG


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64)
    u = torch.zeros(4, 32, dtype=torch.uint8)
    e = torch.zeros(4, 2, dtype=torch.uint8)
    for call in (lambda: sq.quantize_act_mx(x), lambda: sq.smooth_weights_mxfp4(x),
                 lambda: sq.norm_quantize_act_mx(x, torch.ones(64)),
                 lambda: sq.dequantize_mx(u, e), lambda: sq.gemm_mxfp4(u, e, u, e)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_a_stream_of_another_gpu(monkeypatch):
    """Refused before anything is asked of either GPU."""
    torch = pytest.importorskip("torch")

    class Operand:
        device = torch.device("cuda", 0)

        def get_device(self):
            return 0

    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    calls = []
    monkeypatch.setitem(sq._mx_fns, "sq_probe", lambda *a: calls.append(a) or 0)
    with pytest.raises(ValueError, match="stream on cuda:1"):
        sq._mx_call("sq_probe", (Operand(), None, Operand()), (), Stream())
    assert not calls
