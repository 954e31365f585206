"""A launch that fails is reported by its own call and by no other."""

import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
RELAXED = 2


def test_a_failed_launch_is_forgotten_once_reported(bfp8, cuda_device):
    """While an ordinary stream is captured, a launch on the legacy stream is refused by the runtime. The call says so, and
    the next ones, which launch, do not."""
    dev, cu = cuda_device, ctypes.CDLL("libcuda.so.1")
    x = torch.randn(4, 2, 128, device=dev).to(torch.bfloat16)
    out, f, pos = torch.empty_like(x), torch.ones(64, device=dev), torch.arange(4, dtype=torch.int32, device=dev)
    y, codes, scales = x.view(4, 256), torch.empty(4, 256, dtype=torch.uint8, device=dev), torch.empty(4, 2, device=dev)
    calls = [lambda **kw: bfp8.bfp8_rotary(x, x, pos, f, out, out, **kw), lambda **kw: bfp8.bfp8_act_quant_group(y, codes, scales, **kw),
             lambda **kw: bfp8.bfp8_gated_norm(x, x, None, out, **kw)]
    for call in calls:
        call()
    torch.cuda.synchronize()
    for bad in calls:
        stream, graph = ctypes.c_void_p(), ctypes.c_void_p()
        assert cu.cuStreamCreate(ctypes.byref(stream), 0) == 0
        assert cu.cuStreamBeginCapture_v2(stream, RELAXED) == 0
        try:
            with pytest.raises(bfp8.Bfp8Error, match="CUDA"):
                bad(stream=0)
        finally:
            assert cu.cuStreamEndCapture(stream, ctypes.byref(graph)) != 0      # the capture ends with it
            assert cu.cuStreamDestroy_v2(stream) == 0
        for call in calls:
            call()
    torch.cuda.synchronize()
    assert bfp8.bfp8_device_status() == 0
