"""MI355X (gfx950) W8A8 SmoothQuant linear-layer path - Python binding.

Thin ctypes marshalling over the C ABI in ``include/sq.h`` (``libsq.so``,
built from ``csrc/`` by ``build.py``).  Every step of the path runs in the
library's HIP kernels; this module only checks tensors, allocates outputs
with torch (device memory), passes raw pointers and the current HIP stream,
and raises on a non-zero status.  There is no CPU fallback: importing the
functions works anywhere, calling them needs the built library and a GPU.

Names follow the C ABI:
  absmax_reduce      a1  per-channel abs-max (calibration statistics)
  compute_scales     a2  smoothing factors s, 1/s and the static step
  smooth_weights     a3  W * s -> per-output-channel int8
  quantize_act       a4  fused X / s -> int8 (per-token or per-tensor)
  gemm_i8_dequant    a5  int8 GEMM with the outer-product dequant epilogue
  int8_mixed_matmul  a6  LLM.int8() mixed decomposition
  fold_norm          1/s folded into the preceding norm's gamma / beta
  norm_quantize_act  fused fp16 norm -> int8 (per-token or per-tensor)
Microscaled forms (``include/sq_mx.h``): quantize_act_mx,
smooth_weights_mxfp4, norm_quantize_act_mx, dequantize_mx, gemm_mxfp4; a
microscaled cache of keys and values (``include/sq_kv.h``): new_kv_cache_mx,
rope_frequencies, rope_quantize_kv_mx, dequantize_kv_mx, attention_kv_mx.
Their ``stream=`` gets the work and owns the outputs that the call makes; the
caller orders it behind the work that makes the operands.
"""
from __future__ import annotations

import ctypes
import math
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsq.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "sq.h")
MX_HEADER = os.path.join(os.path.dirname(HERE), "include", "sq_mx.h")
MX_TEST_HEADER = os.path.join(os.path.dirname(HERE), "include", "sq_mx_test.h")
TEST_HEADER = os.path.join(os.path.dirname(HERE), "include", "sq_test.h")
KV_HEADER = os.path.join(os.path.dirname(HERE), "include", "sq_kv.h")

SQ_F32, SQ_F16, SQ_BF16 = 0, 1, 2
SQ_PER_TENSOR_STATIC, SQ_PER_TOKEN_DYNAMIC = 0, 1
SQ_NORM_LAYER, SQ_NORM_RMS = 0, 1
SQ_MX_E2M1, SQ_MX_E4M3 = 0, 1
SQ_ROPE_HALF, SQ_ROPE_INTERLEAVED = 0, 1

_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float


class _KvCache(ctypes.Structure):
    """sq_kv_cache of include/sq_kv.h."""
    _fields_ = [("kq", _P), ("ks", _P), ("vq", _P), ("vs", _P), ("pages", _I64), ("heads", _I64),
                ("page", _I64), ("dim", _I64), ("fmt", _I)]


_CACHE_P = ctypes.POINTER(_KvCache)
_Strides2, _Strides6 = _I64 * 2, _I64 * 6
_MOST = (1 << 63) - 1

SIGNATURES = {
    "sq_status_str": (ctypes.c_char_p, [_I]),
    "sq_version": (_I, []),
    "sq_absmax_reduce": (_I, [_P, _I, _I64, _I64, _I, _P, _P]),
    "sq_compute_scales": (_I, [_P, _P, _I64, _F, _P, _P, _P, _P]),
    "sq_smooth_weights": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _P]),
    "sq_smooth_weights_folded": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _P, _P]),
    "sq_quantize_act": (_I, [_P, _I, _I64, _I64, _P, _I, _P, _P, _P, _P]),
    "sq_gemm_i8_dequant": (_I, [_P, _P, _I64, _I64, _I64, _P, _I, _P, _P, _I, _P, _P]),
    "sq_int8_mixed_matmul_workspace": (ctypes.c_size_t, [_I64, _I64, _I64]),
    "sq_int8_mixed_matmul": (_I, [_P, _I64, _I64, _P, _P, _P, _I64, _F, _P, ctypes.c_size_t,
                                  _P, _I, _P, _P, _P]),
    "sq_int8_mixed_matmul_noalloc": (_I, [_P, _I64, _I64, _P, _P, _P, _I64, _F, _P, _I, _P, _P,
                                          _P]),
    "sq_fold_norm": (_I, [_P, _P, _P, _I64, _P, _P, _P]),
    "sq_norm_quantize_act": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _F, _I, _P, _P, _P, _P]),
    "sq_norm_quantize_act_kernel": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _F, _I, _P, _P, _P, _P,
                                         _I]),
    "sq_static_scale": (_I, [_P, _P, _I64, _F, _P, _P]),
    "sq_smooth_weights_fp8": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _P]),
    "sq_quantize_act_fp8": (_I, [_P, _I, _I64, _I64, _P, _I, _P, _P, _P, _P]),
    "sq_gemm_fp8_dequant": (_I, [_P, _P, _I64, _I64, _I64, _P, _I, _P, _P, _I, _P]),
    # microscaled forms (include/sq_mx.h)
    "sq_quantize_act_mx": (_I, [_P, _I, _I64, _I64, _P, _I, _P, _P, _P]),
    "sq_smooth_weights_mxfp4": (_I, [_P, _I, _I64, _I64, _P, _P, _P, _P, _P]),
    "sq_norm_quantize_act_mx": (_I, [_P, _I, _I64, _I64, _I, _P, _P, _F, _I, _P, _P, _P]),
    "sq_dequantize_mx": (_I, [_P, _P, _I, _I64, _I64, _P, _I, _P]),
    "sq_gemm_mxfp4": (_I, [_P, _P, _I, _P, _P, _I64, _I64, _I64, _P, _I, _P]),
    # the microscaled cache (include/sq_kv.h)
    "sq_rope_quantize_kv_mx": (_I, [_P, _P, _P, _P, _P, _P, _I, _I64, _I64, _P,
                                    _P, _I64, ctypes.c_double, _I, _P, _P, _P, _CACHE_P, _P, _P]),
    "sq_dequantize_kv_mx": (_I, [_CACHE_P, _P, _I64, _I64, _P, _I64, _P, _P, _I, _P]),
    "sq_attention_kv_mx": (_I, [_P, _P, _I, _I64, _I64, _CACHE_P, _P, _I64, _I64, _P, _P, _I64,
                                _F, _I, _I64, _P, _P, ctypes.c_size_t, _P]),
    "sq_attention_kv_mx_workspace": (ctypes.c_size_t, [_I64, _I64, _CACHE_P, _I64, _I64, _I64]),
    # coverage entry point (include/sq_mx_test.h): the pipelined product's block shape forced
    "sq_gemm_mxfp4_tile": (_I, [_P, _P, _I, _P, _P, _I64, _I64, _I64, _P, _I, _P, _I]),
    # coverage entry points (include/sq_test.h): the tiled GEMM's block shape forced
    "sq_gemm_i8_dequant_tile": (_I, [_P, _P, _I64, _I64, _I64, _P, _I, _P, _P, _I, _P, _P, _I]),
    "sq_gemm_fp8_dequant_tile": (_I, [_P, _P, _I64, _I64, _I64, _P, _I, _P, _P, _I, _P, _I]),
    "sq_int8_mixed_matmul_tile": (_I, [_P, _I64, _I64, _P, _P, _P, _I64, _F, _P, ctypes.c_size_t,
                                       _P, _I, _P, _P, _P, _I]),
}


class SQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {lib().sq_status_str(status).decode()}")


def header_functions(path: str = HEADER, prefix: str = "sq_"):
    """Names of the functions a header declares (include/sq.h by default)."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(" + prefix + r"[a-z0-9_]+)\s*\(", text)))


def lib():
    """Load libsq.so; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m w8a8_post_quantization_amd.build` "
                              "(hipcc, gfx950) first; there is no CPU fallback")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


_torch_mod = None
_raw_stream = None  # torch's current-stream handle by device, where it has one
_current_gpu = None  # the current device's number
_dt_codes = {}


def _torch():
    global _torch_mod, _raw_stream, _current_gpu
    if _torch_mod is None:
        import torch

        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        # (torch.cuda.current_device asks this, 0.4 us later)
        _current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _dt_codes.update({torch.float32: SQ_F32, torch.float16: SQ_F16, torch.bfloat16: SQ_BF16})
        _torch_mod = torch
    return _torch_mod


def _dt(t) -> int:
    _torch()
    return _dt_codes[t.dtype]


def _tdt(code: int):
    torch = _torch()
    return {SQ_F32: torch.float32, SQ_F16: torch.float16, SQ_BF16: torch.bfloat16}[code]


def _check(t, name, dtypes=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must be {ndim}-D")
    return t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    torch = _torch()
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    # the current stream's handle alone costs 0.3 us, the Stream object 2.7 us
    if _raw_stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))


def _call(name, *args):
    status = getattr(lib(), name)(*args)
    if status != 0:
        raise SQError(name, status)


def absmax_reduce(x, out=None, accumulate=False, stream=None):
    """a1: out[c] = max_r |x[r, c]| (running max into `out` if accumulate)."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    _check(x2, "x", (torch.float32, torch.float16, torch.bfloat16))
    if out is None:
        out = torch.empty(x2.shape[1], dtype=torch.float32, device=x.device)
    _check(out, "out", (torch.float32,))
    _call("sq_absmax_reduce", x2.data_ptr(), _dt(x2), x2.shape[0], x2.shape[1],
          int(bool(accumulate)), out.data_ptr(), _stream(stream))
    return out


def compute_scales(act_amax, w_amax, alpha, static=False, stream=None):
    """a2: (s, inv_s) or (s, inv_s, static_scale[2])."""
    torch = _torch()
    _check(act_amax, "act_amax", (torch.float32,), 1)
    _check(w_amax, "w_amax", (torch.float32,), 1)
    K = act_amax.shape[0]
    s = torch.empty(K, dtype=torch.float32, device=act_amax.device)
    inv = torch.empty_like(s)
    st = torch.empty(2, dtype=torch.float32, device=act_amax.device) if static else None
    _call("sq_compute_scales", act_amax.data_ptr(), w_amax.data_ptr(), K, float(alpha),
          s.data_ptr(), inv.data_ptr(), _ptr(st), _stream(stream))
    return (s, inv, st) if static else (s, inv)


def smooth_weights(w, s=None, row_mul=None, stream=None):
    """a3: (wq int8 [N,K], w_scale fp32 [N]).  row_mul [N]: the next layer's
    inv_s folded into this layer's output channels (sq_smooth_weights_folded)."""
    torch = _torch()
    _check(w, "w", (torch.float32, torch.float16, torch.bfloat16), 2)
    if s is not None:
        _check(s, "s", (torch.float32,), 1)
    N, K = w.shape
    if row_mul is not None:
        _check(row_mul, "row_mul", (torch.float32,), 1)
        if row_mul.numel() != N:
            raise ValueError(f"row_mul has {row_mul.numel()} elements, w has {N} rows")
    if s is not None and s.numel() != K:
        raise ValueError(f"s has {s.numel()} elements, w has {K} columns")
    wq = torch.empty((N, K), dtype=torch.int8, device=w.device)
    ws = torch.empty(N, dtype=torch.float32, device=w.device)
    if row_mul is None:
        _call("sq_smooth_weights", w.data_ptr(), _dt(w), N, K, _ptr(s), wq.data_ptr(),
              ws.data_ptr(), _stream(stream))
    else:
        _call("sq_smooth_weights_folded", w.data_ptr(), _dt(w), N, K, _ptr(row_mul), _ptr(s),
              wq.data_ptr(), ws.data_ptr(), _stream(stream))
    return wq, ws


def quantize_act(x, inv_s=None, mode=SQ_PER_TOKEN_DYNAMIC, static_scale=None, out=None,
                 stream=None):
    """a4: (xq int8 [M,K], x_scale fp32 [M] or [1])."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    _check(x2, "x", (torch.float32, torch.float16, torch.bfloat16))
    if inv_s is not None:
        _check(inv_s, "inv_s", (torch.float32,), 1)
    if static_scale is not None:
        _check(static_scale, "static_scale", (torch.float32,), 1)
    M, K = x2.shape
    if out is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        xs = torch.empty(M if mode == SQ_PER_TOKEN_DYNAMIC else 1, dtype=torch.float32,
                         device=x.device)
    else:
        xq, xs = out
    _call("sq_quantize_act", x2.data_ptr(), _dt(x2), M, K, _ptr(inv_s), int(mode),
          _ptr(static_scale), xq.data_ptr(), xs.data_ptr(), _stream(stream))
    return xq, xs


def gemm_i8_dequant(xq, wq, x_scale, w_scale, out_dtype=None, with_acc=False, out=None,
                    stream=None, tile=None):
    """a5: y [M,N] (and acc int32 [M,N] if with_acc).  tile 0 | 1 | 2 | 3
    forces the tiled kernel's block shape (include/sq_test.h; same bits)."""
    torch = _torch()
    _check(xq, "xq", (torch.int8,), 2)
    _check(wq, "wq", (torch.int8,), 2)
    _check(x_scale, "x_scale", (torch.float32,), 1)
    _check(w_scale, "w_scale", (torch.float32,), 1)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError("xq and wq disagree on K")
    per_row = 1 if (x_scale.numel() == M and M != 1) else 0
    if x_scale.numel() not in (1, M):
        raise ValueError("x_scale must have 1 or M elements")
    if w_scale.numel() != N:
        raise ValueError("w_scale must have N elements")
    y = out if out is not None else torch.empty(
        (M, N), dtype=out_dtype or torch.float32, device=xq.device)
    acc = torch.empty((M, N), dtype=torch.int32, device=xq.device) if with_acc else None
    if tile is None:
        _call("sq_gemm_i8_dequant", xq.data_ptr(), wq.data_ptr(), M, N, K, x_scale.data_ptr(),
              per_row, w_scale.data_ptr(), y.data_ptr(), _dt(y), _ptr(acc), _stream(stream))
    else:
        _call("sq_gemm_i8_dequant_tile", xq.data_ptr(), wq.data_ptr(), M, N, K,
              x_scale.data_ptr(), per_row, w_scale.data_ptr(), y.data_ptr(), _dt(y), _ptr(acc),
              _stream(stream), int(tile))
    return (y, acc) if with_acc else y


SQ_MIXED_SIDE_COLS = 128


def int8_mixed_matmul_workspace(M, N, K) -> int:
    return int(lib().sq_int8_mixed_matmul_workspace(M, N, K))


def int8_mixed_workspace_parts(M, N, K):
    """Byte offsets of the parts the workspace holds on return (include/sq.h):
    xq [M,K] int8, x_scale [M], colmax [K], mask [K] fp32, idx [K] int32,
    count int32, then (written when |O| <= side_cols) the side operands
    x_side [side_cols, M] and w_side [side_cols, N] fp32."""
    r = lambda b: (b + 255) // 256 * 256  # noqa: E731
    cap = min(K, SQ_MIXED_SIDE_COLS)
    off = {"xq": 0, "side_cols": cap}
    off["x_scale"] = off["xq"] + r(M * K)
    off["colmax"] = off["x_scale"] + r(4 * M)
    off["mask"] = off["colmax"] + r(4 * K)
    off["idx"] = off["mask"] + r(4 * K)
    off["count"] = off["idx"] + r(4 * K)
    off["x_side"] = off["count"] + 256
    off["w_side"] = off["x_side"] + r(4 * cap * M)
    off["total"] = off["w_side"] + r(4 * cap * N)
    return off


def int8_mixed_matmul(x, wq, w_scale, w_f16, threshold=6.0, out_dtype=None, workspace=None,
                      with_count=False, with_acc=False, stream=None, tile=None):
    """a6: LLM.int8() y [M,N], then (if asked) acc int32 [M,N] and |O| as a
    1-element int32 tensor: y, (y, cnt), (y, acc) or (y, acc, cnt)."""
    torch = _torch()
    _check(x, "x", (torch.float16,), 2)
    _check(wq, "wq", (torch.int8,), 2)
    _check(w_scale, "w_scale", (torch.float32,), 1)
    _check(w_f16, "w_f16", (torch.float16,), 2)
    M, K = x.shape
    N = wq.shape[0]
    need = int8_mixed_matmul_workspace(M, N, K)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    y = torch.empty((M, N), dtype=out_dtype or torch.float16, device=x.device)
    cnt = torch.zeros(1, dtype=torch.int32, device=x.device) if with_count else None
    acc = torch.empty((M, N), dtype=torch.int32, device=x.device) if with_acc else None
    args = (x.data_ptr(), M, K, wq.data_ptr(), w_scale.data_ptr(), w_f16.data_ptr(), N,
            float(threshold), workspace.data_ptr(), workspace.numel(), y.data_ptr(), _dt(y),
            _ptr(acc), _ptr(cnt), _stream(stream))
    if tile is None:
        _call("sq_int8_mixed_matmul", *args)
    else:
        _call("sq_int8_mixed_matmul_tile", *args, int(tile))
    out = (y,) + ((acc,) if with_acc else ()) + ((cnt,) if with_count else ())
    return out if len(out) > 1 else y


def int8_mixed_matmul_noalloc(x, wq, w_scale, w_f16, threshold=6.0, out=None, acc=None,
                              count=None, stream=None):
    """a6 without a workspace (the library's per-GPU array): writes y into
    `out` (required, [M,N]), and acc / |O| into `acc` / `count` when given.
    Allocates nothing."""
    torch = _torch()
    _check(x, "x", (torch.float16,), 2)
    _check(wq, "wq", (torch.int8,), 2)
    _check(w_scale, "w_scale", (torch.float32,), 1)
    _check(w_f16, "w_f16", (torch.float16,), 2)
    _check(out, "out", (torch.float32, torch.float16, torch.bfloat16), 2)
    M, K = x.shape
    N = wq.shape[0]
    _call("sq_int8_mixed_matmul_noalloc", x.data_ptr(), M, K, wq.data_ptr(), w_scale.data_ptr(),
          w_f16.data_ptr(), N, float(threshold), out.data_ptr(), _dt(out), _ptr(acc), _ptr(count),
          _stream(stream))
    return out


def fold_norm(gamma, s, beta=None, stream=None):
    """(gamma / s, beta / s or None): the smoothing folded into the norm."""
    torch = _torch()
    _check(gamma, "gamma", (torch.float32,), 1)
    _check(s, "s", (torch.float32,), 1)
    if beta is not None:
        _check(beta, "beta", (torch.float32,), 1)
    g_out = torch.empty_like(gamma)
    b_out = None if beta is None else torch.empty_like(beta)
    _call("sq_fold_norm", gamma.data_ptr(), _ptr(beta), s.data_ptr(), gamma.numel(),
          g_out.data_ptr(), _ptr(b_out), _stream(stream))
    return g_out, b_out


def norm_quantize_act(x, gamma, beta=None, norm=SQ_NORM_LAYER, eps=1e-5,
                      mode=SQ_PER_TOKEN_DYNAMIC, static_scale=None, out=None, stream=None,
                      kernel=None):
    """Fused fp16 norm -> int8: (xq int8 [M,K], x_scale fp32 [M] or [1]).
    kernel (tests only): 0 or 1 forces the block- or wave-per-row kernel
    through the coverage entry point of sq_test.h."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    _check(x2, "x", (torch.float16,))
    _check(gamma, "gamma", (torch.float32,), 1)
    if beta is not None:
        _check(beta, "beta", (torch.float32,), 1)
    if static_scale is not None:
        _check(static_scale, "static_scale", (torch.float32,), 1)
    M, K = x2.shape
    if out is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
        xs = torch.empty(M if mode == SQ_PER_TOKEN_DYNAMIC else 1, dtype=torch.float32,
                         device=x.device)
    else:
        xq, xs = out
    args = (x2.data_ptr(), _dt(x2), M, K, int(norm), gamma.data_ptr(), _ptr(beta), float(eps),
            int(mode), _ptr(static_scale), xq.data_ptr(), xs.data_ptr(), _stream(stream))
    if kernel is None:
        _call("sq_norm_quantize_act", *args)
    else:
        _call("sq_norm_quantize_act_kernel", *args, int(kernel))
    return xq, xs


# ------------------------------------------------------------ FP8 (e4m3)

def static_scale(act_amax, inv_s=None, qmax=127.0, stream=None):
    """{step, 1/step} of a per-tensor static activation step (qmax 127 for
    int8, 448 for e4m3)."""
    torch = _torch()
    _check(act_amax, "act_amax", (torch.float32,), 1)
    if inv_s is not None:
        _check(inv_s, "inv_s", (torch.float32,), 1)
    out = torch.empty(2, dtype=torch.float32, device=act_amax.device)
    _call("sq_static_scale", act_amax.data_ptr(), _ptr(inv_s), act_amax.numel(), float(qmax),
          out.data_ptr(), _stream(stream))
    return out


def smooth_weights_fp8(w, s=None, stream=None):
    """a3 in e4m3: (wq uint8 [N,K] e4m3 codes, w_scale fp32 [N])."""
    torch = _torch()
    _check(w, "w", (torch.float32, torch.float16, torch.bfloat16), 2)
    if s is not None:
        _check(s, "s", (torch.float32,), 1)
    N, K = w.shape
    wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    ws = torch.empty(N, dtype=torch.float32, device=w.device)
    _call("sq_smooth_weights_fp8", w.data_ptr(), _dt(w), N, K, _ptr(s), wq.data_ptr(),
          ws.data_ptr(), _stream(stream))
    return wq, ws


def quantize_act_fp8(x, inv_s=None, mode=SQ_PER_TOKEN_DYNAMIC, static_scale=None, stream=None):
    """a4 in e4m3: (xq uint8 [M,K] e4m3 codes, x_scale fp32 [M] or [1])."""
    torch = _torch()
    x2 = x.reshape(-1, x.shape[-1])
    _check(x2, "x", (torch.float32, torch.float16, torch.bfloat16))
    if inv_s is not None:
        _check(inv_s, "inv_s", (torch.float32,), 1)
    if static_scale is not None:
        _check(static_scale, "static_scale", (torch.float32,), 1)
    M, K = x2.shape
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    xs = torch.empty(M if mode == SQ_PER_TOKEN_DYNAMIC else 1, dtype=torch.float32,
                     device=x.device)
    _call("sq_quantize_act_fp8", x2.data_ptr(), _dt(x2), M, K, _ptr(inv_s), int(mode),
          _ptr(static_scale), xq.data_ptr(), xs.data_ptr(), _stream(stream))
    return xq, xs


def gemm_fp8_dequant(xq, wq, x_scale, w_scale, out_dtype=None, out=None, stream=None,
                     tile=None):
    """f4: y [M,N] = fl(acc * fl(x_scale * w_scale)) with acc the fp32 sum of
    the e4m3 products (K % 128 == 0)."""
    torch = _torch()
    _check(xq, "xq", (torch.uint8,), 2)
    _check(wq, "wq", (torch.uint8,), 2)
    _check(x_scale, "x_scale", (torch.float32,), 1)
    _check(w_scale, "w_scale", (torch.float32,), 1)
    M, K = xq.shape
    N = wq.shape[0]
    if wq.shape[1] != K:
        raise ValueError(f"K mismatch: xq {tuple(xq.shape)}, wq {tuple(wq.shape)}")
    per_row = 1 if (x_scale.numel() == M and M != 1) else 0
    if not per_row and x_scale.numel() != 1:
        raise ValueError(f"x_scale has {x_scale.numel()} elements for M = {M}")
    if w_scale.numel() != N:
        raise ValueError(f"w_scale has {w_scale.numel()} elements for N = {N}")
    dt = out_dtype or torch.float16
    y = out if out is not None else torch.empty((M, N), dtype=dt, device=xq.device)
    if tile is None:
        _call("sq_gemm_fp8_dequant", xq.data_ptr(), wq.data_ptr(), M, N, K, x_scale.data_ptr(),
              int(per_row), w_scale.data_ptr(), y.data_ptr(), _dt(y), _stream(stream))
    else:
        _call("sq_gemm_fp8_dequant_tile", xq.data_ptr(), wq.data_ptr(), M, N, K,
              x_scale.data_ptr(), int(per_row), w_scale.data_ptr(), y.data_ptr(), _dt(y),
              _stream(stream), int(tile))
    return y


# ------------------------------------------------------- microscaled (MX)

_mx_fns = {}


def _mx_call(name, tensors, args, stream, *last):
    """Call `name` on the operands' own GPU.  `tensors` are all the operands
    (None allowed, the first present); `stream` (or that GPU's current stream)
    gets the work, and is one of that GPU (a kernel on another would read
    memory that it cannot); `last` are the arguments behind the stream."""
    fn = _mx_fns.get(name)
    if fn is None:
        fn = _mx_fns[name] = getattr(lib(), name)
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"operands on {tensors[0].device} and {t.device}")
    if stream is not None and stream.device.index != dev:
        raise ValueError(f"operands on {tensors[0].device}, stream on {stream.device}")
    if _current_gpu() == dev:
        if stream is None and _raw_stream is not None:
            status = fn(*args, _raw_stream(dev), *last)
        else:
            status = fn(*args, _stream(stream), *last)
    else:
        with _torch_mod.cuda.device(dev):
            status = fn(*args, _stream(stream), *last)
    if status != 0:
        raise SQError(name, status)


# The checks of these latency-bound calls are one expression each; the
# functions that name what is wrong run only where it fails.

def _mx_check(t, name, dtypes, ndim):
    if not (t.is_cuda and t.dtype in dtypes and t.dim() == ndim and t.is_contiguous()):
        _check(t, name, dtypes, ndim)


def _mx_codes(fmt, K):
    """Code bytes of a row of K elements."""
    if fmt not in (SQ_MX_E2M1, SQ_MX_E4M3):
        raise ValueError(f"unknown MX format {fmt}")
    return K // 2 if fmt == SQ_MX_E2M1 else K


def _mx_shapes(q, scale, fmt, name):
    """(rows, K) of codes [rows, K / 2] or [rows, K] and scales [rows, K / 32]."""
    u8 = _torch().uint8
    if not (q.is_cuda and q.dtype == u8 and q.is_contiguous() and scale.is_cuda
            and scale.dtype == u8 and scale.is_contiguous() and q.dim() == 2 == scale.dim()):
        _check(q, name, (u8,), 2)
        _check(scale, "the scales of codes", (u8,), 2)
    rows, codes = q.shape
    srows, blocks = scale.shape
    K = blocks * 32
    if codes != _mx_codes(fmt, K) or srows != rows:
        raise ValueError(f"{name} {tuple(q.shape)} and its scales {tuple(scale.shape)} disagree")
    return rows, K


def _mx_empty(rows, cols, dtype, device, stream):
    """A new output, allocated for the stream that writes it: memory of the
    current stream's pool may be a freed tensor's, whose last kernels another
    stream would not wait for."""
    if stream is not None:
        with _torch_mod.cuda.stream(stream):
            return _mx_empty(rows, cols, dtype, device, None)
    # (0.3 us less than empty, which works the strides out)
    return _torch_mod.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _mx_out(out, rows, K, fmt, device, stream):
    if K % 32:
        raise ValueError(f"rows of {K} elements: a multiple of 32 is needed")
    if out is None:
        u8 = _torch_mod.uint8
        return (_mx_empty(rows, _mx_codes(fmt, K), u8, device, stream),
                _mx_empty(rows, K // 32, u8, device, stream))
    q, scale = out
    if _mx_shapes(q, scale, fmt, "out") != (rows, K):
        raise ValueError(f"out {tuple(q.shape)} does not fit {rows} rows of {K} elements")
    return q, scale


def _mx_result(out, rows, cols, dtype, device, stream):
    """The values' tensor: `out`, checked, or a new one."""
    if out is None:
        if dtype not in _dt_codes:
            raise ValueError(f"out_dtype {dtype} not in {tuple(_dt_codes)}")
        return _mx_empty(rows, cols, dtype, device, stream)
    _mx_check(out, "out", _dt_codes, 2)
    if out.shape != (rows, cols):
        raise ValueError(f"out {tuple(out.shape)} is not {(rows, cols)}")
    return out


def _vector(t, name, n):
    """The pointer of an fp32 vector of n elements, or None."""
    if t is None:
        return None
    if not (t.is_cuda and t.dtype == _torch_mod.float32 and t.dim() == 1 and t.is_contiguous()):
        _check(t, name, (_torch_mod.float32,), 1)
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, not {n}")
    return t.data_ptr()


def _mx_rows(x, name):
    _torch()
    if x.dim() != 2:
        # (a view, never a copy: that would run on the current stream, the call
        # perhaps on another)
        _check(x, name, _dt_codes)
        x = x.reshape(-1, x.shape[-1])
    if not (x.is_cuda and x.dtype in _dt_codes and x.is_contiguous()):
        _check(x, name, _dt_codes, 2)
    return x


def quantize_act_mx(x, inv_s=None, fmt=SQ_MX_E2M1, out=None, stream=None):
    """a4 in MX: (xq uint8 [M, K/2] or [M, K], x_scale uint8 [M, K/32]) of
    fl(x * inv_s), a power-of-two scale for each 32 elements."""
    x2 = _mx_rows(x, "x")
    M, K = x2.shape
    inv = _vector(inv_s, "inv_s", K)
    xq, xs = _mx_out(out, M, K, fmt, x2.device, stream)
    _mx_call("sq_quantize_act_mx", (x2, inv_s, xq, xs),
             (x2.data_ptr(), _dt_codes[x2.dtype], M, K, inv, fmt, xq.data_ptr(), xs.data_ptr()), stream)
    return xq, xs


def smooth_weights_mxfp4(w, s=None, row_mul=None, out=None, stream=None):
    """a3 in MX: (wq uint8 [N, K/2] e2m1, w_scale uint8 [N, K/32]) of
    fl(fl(w * row_mul[n]) * s[k]); row_mul and s as in smooth_weights."""
    _torch()
    _mx_check(w, "w", _dt_codes, 2)
    N, K = w.shape
    sp, rp = _vector(s, "s", K), _vector(row_mul, "row_mul", N)
    wq, ws = _mx_out(out, N, K, SQ_MX_E2M1, w.device, stream)
    _mx_call("sq_smooth_weights_mxfp4", (w, s, row_mul, wq, ws),
             (w.data_ptr(), _dt_codes[w.dtype], N, K, rp, sp, wq.data_ptr(), ws.data_ptr()), stream)
    return wq, ws


def norm_quantize_act_mx(x, gamma, beta=None, norm=SQ_NORM_LAYER, eps=1e-5, fmt=SQ_MX_E2M1,
                         out=None, stream=None):
    """Fused norm -> MX codes: (xq, x_scale) as quantize_act_mx."""
    x2 = _mx_rows(x, "x")
    M, K = x2.shape
    if gamma is None:
        raise ValueError("gamma is needed")
    g, b = _vector(gamma, "gamma", K), _vector(beta, "beta", K)
    xq, xs = _mx_out(out, M, K, fmt, x2.device, stream)
    _mx_call("sq_norm_quantize_act_mx", (x2, gamma, beta, xq, xs),
             (x2.data_ptr(), _dt_codes[x2.dtype], M, K, norm, g, b, eps, fmt, xq.data_ptr(), xs.data_ptr()),
             stream)
    return xq, xs


def dequantize_mx(q, scale, fmt=SQ_MX_E2M1, out_dtype=None, out=None, stream=None):
    """The values [rows, K] (fp32 unless out_dtype says otherwise) that MX
    codes and scales stand for."""
    rows, K = _mx_shapes(q, scale, fmt, "q")
    y = _mx_result(out, rows, K, out_dtype or _torch_mod.float32, q.device, stream)
    _mx_call("sq_dequantize_mx", (q, scale, y),
             (q.data_ptr(), scale.data_ptr(), fmt, rows, K, y.data_ptr(), _dt_codes[y.dtype]), stream)
    return y


def gemm_mxfp4(xq, x_scale, wq, w_scale, x_fmt=SQ_MX_E2M1, out_dtype=None, out=None, stream=None,
               tile=None):
    """a5 in MX: y [M, N] (fp16 unless out_dtype says otherwise), the product
    of e2m1 weights with activations of x_fmt, summed in fp32.  tile (tests
    only) forces the block shape (include/sq_mx_test.h)."""
    M, K = _mx_shapes(xq, x_scale, x_fmt, "xq")
    N, Kw = _mx_shapes(wq, w_scale, SQ_MX_E2M1, "wq")
    if K != Kw:
        raise ValueError(f"K mismatch: xq has {K}, wq {Kw}")
    y = _mx_result(out, M, N, out_dtype or _torch_mod.float16, xq.device, stream)
    args = (xq.data_ptr(), x_scale.data_ptr(), x_fmt, wq.data_ptr(), w_scale.data_ptr(), M, N, K,
            y.data_ptr(), _dt_codes[y.dtype])
    if tile is None:
        _mx_call("sq_gemm_mxfp4", (xq, x_scale, wq, w_scale, y), args, stream)
    else:
        _mx_call("sq_gemm_mxfp4_tile", (xq, x_scale, wq, w_scale, y), args, stream, int(tile))
    return y


# ------------------------------- a microscaled cache of keys and values

def new_kv_cache_mx(pages, heads, page, dim, fmt=SQ_MX_E2M1, device="cuda"):
    """An empty cache of `pages` pages of `page` tokens: (kq, ks, vq, vs), codes
    uint8 [pages, heads, page, dim/2] or [.., dim] and scale bytes [.., dim/32]
    of keys and values."""
    if dim % 32:
        raise ValueError(f"heads of {dim} channels: a multiple of 32 is needed")
    torch = _torch()

    def zeros(n):
        return torch.zeros((pages, heads, page, n), dtype=torch.uint8, device=device)

    return (zeros(_mx_codes(fmt, dim)), zeros(dim // 32), zeros(_mx_codes(fmt, dim)), zeros(dim // 32))


def rope_frequencies(rotary, base=10000.0, scaling=None, factor=1.0, original=None, fast=32.0,
                     slow=1.0, device="cuda"):
    """(inv_freq fp64 [rotary/2], amplitude) of rotary positions for
    rope_quantize_kv_mx: base^(-2 i / rotary), for contexts `factor` times the
    `original` length by `scaling`
      None      as they are
      "linear"  positions divided by the factor
      "ntk"     the base raised so that the slowest frequency is divided by it
      "yarn"    frequencies that turn fewer than `slow` times in the original
                length divided by the factor, those that turn more than `fast`
                times kept, a ramp between that is linear in the number of
                turns; amplitude 0.1 ln(factor) + 1
    A model that was tuned with others (a ramp over i between the channels of
    `slow` and `fast` turns, say) passes its own: any fp64 tensor serves."""
    if rotary < 2 or rotary % 2:
        raise ValueError(f"{rotary} rotated channels: an even number is needed")
    if scaling not in (None, "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}")
    if not (base > 0 and factor >= 1):
        raise ValueError(f"base {base}, factor {factor}: base > 0 and factor >= 1 are needed")
    if scaling == "yarn" and not (original and original > 0 and fast > slow):
        raise ValueError("yarn needs the original length, and fast > slow")
    amplitude = 1.0
    if scaling == "ntk" and rotary > 2:
        base = base * factor ** (rotary / (rotary - 2.0))
    freq = [float(base) ** (-2.0 * i / rotary) for i in range(rotary // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    elif scaling == "yarn":
        amplitude = 0.1 * math.log(factor) + 1.0
        for i, f in enumerate(freq):
            turns = original * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - slow) / (fast - slow)))
            freq[i] = f * keep + f / factor * (1.0 - keep)
    torch = _torch()
    return torch.tensor(freq, dtype=torch.float64, device=device), amplitude


def _kv_cache(cache, fmt):
    """The C form of a cache (kq, ks, vq, vs)."""
    u8 = _torch().uint8
    kq, ks, vq, vs = cache
    shape, blocks = kq.shape, ks.shape
    if not (len(shape) == 4 == len(blocks) and vq.shape == shape and vs.shape == blocks
            and shape[:3] == blocks[:3] and shape[3] == _mx_codes(fmt, blocks[3] * 32)
            and kq.dtype == u8 == ks.dtype and vq.dtype == u8 == vs.dtype
            and kq.is_contiguous() and ks.is_contiguous() and vq.is_contiguous()
            and vs.is_contiguous() and kq.is_cuda):
        for t, name in ((kq, "cached keys"), (ks, "the keys' scales"), (vq, "cached values"),
                        (vs, "the values' scales")):
            _check(t, name, (u8,), 4)
        raise ValueError(f"cache of codes {tuple(shape)}, {tuple(vq.shape)} and scales "
                         f"{tuple(blocks)}, {tuple(vs.shape)}: they disagree")
    pages, heads, page, n = blocks
    return _KvCache(kq.data_ptr(), ks.data_ptr(), vq.data_ptr(), vs.data_ptr(), pages, heads, page,
                    n * 32, fmt)


def _kv_rows(x, name, dim, dtypes):
    """The token's and the head's stride of rows [T, heads, dim], each dense."""
    if not (x.dtype in dtypes and x.dim() == 3 and x.is_cuda):
        if not x.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
        if x.dtype not in dtypes:
            raise ValueError(f"{name}: dtype {x.dtype} not in {tuple(dtypes)}")
        raise ValueError(f"{name} must be [tokens, heads, {dim}]")
    token, head, one = x.stride()
    if x.shape[2] != dim:
        raise ValueError(f"{name} has rows of {x.shape[2]} channels, the cache of {dim}")
    if one != 1:
        raise ValueError(f"{name} must have dense rows")
    return token, head


def _kv_ints(t, name, dtype, shape):
    """The pointer of an integer tensor of this shape, or None."""
    if t is None:
        return None
    if not (t.dtype == dtype and t.shape == shape and t.is_contiguous() and t.is_cuda):
        _check(t, name, (dtype,), len(shape))
        raise ValueError(f"{name} {tuple(t.shape)} is not {tuple(shape)}")
    return t.data_ptr()


def _kv_mul(t, name, heads, dim):
    """The pointer of fp32 multipliers [heads, dim] (or as one vector), or None."""
    if t is None:
        return None
    if not (t.dtype == _torch_mod.float32 and t.is_contiguous() and t.is_cuda):
        _check(t, name, (_torch_mod.float32,))
    if t.shape != (heads, dim) and t.shape != (heads * dim,):
        raise ValueError(f"{name} {tuple(t.shape)} is not {(heads, dim)}")
    return t.data_ptr()


def _kv_result(out, name, shape, dtype, device, stream):
    """A dense output [tokens, heads, dim]: `out`, checked, or a new one."""
    if out is None:
        if stream is not None:  # (of that stream's memory: _mx_empty)
            with _torch_mod.cuda.stream(stream):
                return _kv_result(None, name, shape, dtype, device, None)
        return _torch_mod.empty_strided(shape, (shape[1] * shape[2], shape[2], 1), dtype=dtype, device=device)
    if not (out.is_cuda and out.dtype == dtype and out.is_contiguous() and out.shape == shape):
        _check(out, name, (dtype,), 3)
        raise ValueError(f"{name} {tuple(out.shape)} is not {tuple(shape)}")
    return out


def rope_quantize_kv_mx(q, k, v, slots, cache, fmt=SQ_MX_E2M1, positions=None, inv_freq=None,
                        amplitude=1.0, layout=SQ_ROPE_HALF, q_mul=None, k_mul=None, out=None,
                        stream=None):
    """Rotary positions, and keys and values quantized into the cache: rows of
    k and v [T, heads, dim] go to slots [T] int64 (page * page size + place;
    others, as -1, are not written), the rotated q [T, q_heads, dim] (None: keys
    and values alone) is returned, in `out` if given (which shares no memory with
    an input).  positions [T] int64 and inv_freq fp64 [rotary/2]
    (rope_frequencies; None: nothing is rotated), the first `rotary` channels;
    q_mul, k_mul fp32 [heads, dim]: smoothing, after the rotation."""
    c = _kv_cache(cache, fmt)
    heads, dim = c.heads, c.dim
    dt = k.dtype
    k_token, k_head = _kv_rows(k, "k", dim, _dt_codes)
    v_token, v_head = _kv_rows(v, "v", dim, (dt,))
    T = k.shape[0]
    if k.shape[1] != heads or v.shape != k.shape:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} do not fit a cache of {heads} heads")
    i64 = _torch_mod.int64
    if slots is None:
        raise ValueError("slots are needed")
    sp = _kv_ints(slots, "slots", i64, (T,))
    rotary, fp, pp = 0, None, None
    if inv_freq is not None:
        if positions is None:
            raise ValueError("positions are needed")
        pp = _kv_ints(positions, "positions", i64, (T,))
        _mx_check(inv_freq, "inv_freq", (_torch_mod.float64,), 1)
        rotary, fp = 2 * inv_freq.shape[0], inv_freq.data_ptr()
        if rotary > dim or rotary % 16:
            raise ValueError(f"{rotary} rotated channels: a multiple of 16 up to {dim} is needed")
    qp, yp, q_heads, y, q_token, q_head = None, None, 0, None, 0, 0
    if q is not None:
        q_token, q_head = _kv_rows(q, "q", dim, (dt,))
        q_tokens, q_heads, _ = q.shape
        if q_tokens != T:
            raise ValueError(f"q has {q_tokens} tokens, k {T}")
        qp = q.data_ptr()
        y = _kv_result(out, "out", (T, q_heads, dim), dt, q.device, stream)
        yp = y.data_ptr()
        if yp == qp and T:
            raise ValueError("out is q: a rotation in place is not supported")
    elif q_mul is not None or out is not None:
        raise ValueError("q_mul and out need q")
    qm, km = _kv_mul(q_mul, "q_mul", q_heads, dim), _kv_mul(k_mul, "k_mul", heads, dim)
    strides = _Strides6(q_token, q_head, k_token, k_head, v_token, v_head)
    at = ctypes.addressof(strides)
    _mx_call("sq_rope_quantize_kv_mx",
             (k, v, q, slots, positions if rotary else None, inv_freq, q_mul, k_mul, y, *cache),
             (qp, at, k.data_ptr(), at + 16, v.data_ptr(), at + 32, _dt_codes[dt], T, q_heads, pp, fp,
              rotary, amplitude, layout if 0 <= layout <= 1 else -1, qm, km, sp, c, yp), stream)
    return y


def dequantize_kv_mx(cache, table, cu, total, fmt=SQ_MX_E2M1, out_dtype=None, out=None, stream=None):
    """(k, v) [total, heads, dim]: the values (fp16 unless out_dtype says
    otherwise) of cached tokens, sequence after sequence.  table int32 [B,
    width]: each sequence's pages; cu int32 [B + 1]: where each begins in the
    result; rows from cu[B] on are left as they were."""
    c = _kv_cache(cache, fmt)
    i32 = _torch_mod.int32
    _mx_check(table, "table", (i32,), 2)
    B, width = table.shape
    if cu is None:
        raise ValueError("cu is needed")
    cp = _kv_ints(cu, "cu", i32, (B + 1,))
    dtype = out_dtype or _torch_mod.float16
    if dtype not in _dt_codes:
        raise ValueError(f"out_dtype {dtype} not in {tuple(_dt_codes)}")
    shape = (int(total), c.heads, c.dim)
    if shape[0] < 0:
        raise ValueError(f"total {total}")
    if out is not None:
        dtype = out[0].dtype if out_dtype is None else dtype
        if dtype not in _dt_codes:
            raise ValueError(f"out: dtype {dtype} not in {tuple(_dt_codes)}")
    k = _kv_result(None if out is None else out[0], "out", shape, dtype, table.device, stream)
    v = _kv_result(None if out is None else out[1], "out", shape, dtype, table.device, stream)
    _mx_call("sq_dequantize_kv_mx", (table, cu, k, v, *cache),
             (c, table.data_ptr(), B, width, cp, shape[0], k.data_ptr(), v.data_ptr(),
              _dt_codes[dtype]), stream)
    return k, v


def attention_kv_mx_workspace(T, q_heads, cache, B, width, max_q, fmt=SQ_MX_E2M1) -> int:
    """Bytes of workspace of such an attention_kv_mx call."""
    max_q = max(-1, min(max_q, T))  # (the C call's numbers have 64 bits)
    return int(lib().sq_attention_kv_mx_workspace(T, q_heads, _kv_cache(cache, fmt), B, width, max_q))


def attention_kv_mx(q, cache, table, seq_lens, cu_q=None, fmt=SQ_MX_E2M1, max_q=None, scale=None,
                    causal=True, window=0, out=None, workspace=None, stream=None):
    """Attention of q [T, q_heads, dim] (fp16 or bf16) over the cache: y of its
    shape.  seq_lens int32 [B]: each sequence's cached tokens, the queries' own
    keys among them; cu_q int32 [B + 1]: where each sequence's queries begin
    (None: one query a sequence).  table int32 [B, width].  max_q: an upper
    bound of a sequence's queries (T without it).  scale: 1 / sqrt(dim) unless
    given.  window > 0: a query sees that many keys at the most, itself the
    last.  A query that sees no key gets 0, one whose scores are all -inf NaN.
    workspace: attention_kv_mx_workspace bytes (uint8), used by this call alone
    while it runs; allocated without it."""
    c = _kv_cache(cache, fmt)
    dim = c.dim
    torch = _torch_mod
    strides = _Strides2(*_kv_rows(q, "q", dim, (torch.float16, torch.bfloat16)))
    T, q_heads, _ = q.shape
    if q_heads == 0 or q_heads % c.heads:
        raise ValueError(f"{q_heads} query heads do not share {c.heads} key heads evenly")
    i32 = torch.int32
    _mx_check(table, "table", (i32,), 2)
    B, width = table.shape
    if seq_lens is None:
        raise ValueError("seq_lens are needed")
    lp, cp = _kv_ints(seq_lens, "seq_lens", i32, (B,)), _kv_ints(cu_q, "cu_q", i32, (B + 1,))
    if cu_q is None:
        if T != B:
            raise ValueError(f"{T} queries for {B} sequences need cu_q")
        max_q = 1
    elif max_q is None:
        max_q = T
    elif max_q < 1:
        raise ValueError(f"max_q {max_q}")
    else:
        max_q = min(max_q, max(T, 1))  # (the C call's numbers have 64 bits)
    if scale is None:
        scale = dim ** -0.5
    if window < 0:
        raise ValueError(f"window {window}")
    window = min(window, _MOST)
    y = _kv_result(out, "out", (T, q_heads, dim), q.dtype, q.device, stream)
    if y.data_ptr() == q.data_ptr() and T:
        raise ValueError("out is q")
    need = lib().sq_attention_kv_mx_workspace(T, q_heads, c, B, width, max_q)
    if workspace is None:
        workspace = _mx_empty(1, need, torch.uint8, q.device, stream)
    else:
        _check(workspace, "workspace", (torch.uint8,))
    _mx_call("sq_attention_kv_mx", (q, table, seq_lens, cu_q, y, workspace, *cache),
             (q.data_ptr(), ctypes.addressof(strides), _dt_codes[q.dtype], T, q_heads, c,
              table.data_ptr(), B, width, lp, cp, max_q, scale, 1 if causal else 0, window,
              y.data_ptr(), workspace.data_ptr(), workspace.numel()), stream)
    return y
