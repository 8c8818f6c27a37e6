"""Outputs that a microscaled call makes belong to the stream that writes them:
a block of another stream's pool may still be in use by that stream's kernels."""
import pytest

import w8a8_post_quantization_amd as sq
from tests.gpu_util import log

pytestmark = pytest.mark.gpu


def _pool_of(torch, t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in any segment")


def test_new_outputs_belong_to_the_given_stream():
    import torch

    s = torch.cuda.Stream()
    x = torch.randn(40, 512, device="cuda", dtype=torch.float16)
    g = torch.ones(512, device="cuda")
    w = sq.smooth_weights_mxfp4(torch.randn(64, 512, device="cuda"))
    a = sq.quantize_act_mx(x)
    calls = {
        "quantize_act_mx": lambda st: sq.quantize_act_mx(x, stream=st),
        "smooth_weights_mxfp4": lambda st: sq.smooth_weights_mxfp4(x, stream=st),
        "norm_quantize_act_mx": lambda st: sq.norm_quantize_act_mx(x, g, stream=st),
        "dequantize_mx": lambda st: (sq.dequantize_mx(*a, stream=st),),
        "gemm_mxfp4": lambda st: (sq.gemm_mxfp4(*a, *w, stream=st),),
    }
    torch.cuda.synchronize()
    for name, call in calls.items():
        log(f"{name} on a given stream")
        # freed blocks of the current stream, of every size that follows
        freed = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (640, 10240, 20480, 40960, 81920)]
        del freed
        want = call(None)
        got = call(s)
        s.synchronize()
        for t, u in zip(got, want):
            assert _pool_of(torch, t) == s.cuda_stream, name
            assert _pool_of(torch, u) == torch.cuda.current_stream().cuda_stream, name
            assert torch.equal(t, u), name
