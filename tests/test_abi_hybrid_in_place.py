"""Outputs over their own input, without a GPU: with other strides than the input's, rows would be overwritten before they
are read, so the call is refused ahead of any CUDA call (which, without a GPU, is what a call that is not refused meets)."""

import pytest
import torch

from test_abi_hybrid_layer import INVAL, P, _gated, _rotary

CASES = [
    (_gated, dict(out_stride_token=512), True), (_gated, dict(out_stride_head=256, out_stride_token=512), True),
    (_gated, dict(x_bf16=2 * P, gate_stride_token=512), True), (_gated, dict(x_bf16=2 * P, gate_stride_head=136), True),
    (_gated, dict(tokens=1, out_stride_token=512), False), (_gated, dict(heads=1, ldq=128, out_stride_head=256), False),
    (_gated, dict(out_bf16=3 * P, out_stride_token=512), False), (_gated, dict(out_bf16=None, out_stride_token=512), False),
    (_gated, {}, False),
    (_rotary, dict(q_out_stride_token=512), True), (_rotary, dict(q_out_stride_head=136), True), (_rotary, dict(k_out_stride_token=512), True),
    (_rotary, dict(k_out_stride_head=256), False), (_rotary, dict(tokens=1, q_stride_token=512), False),
    (_rotary, dict(q_out_bf16=2 * P, q_out_stride_token=512), False), (_rotary, dict(k_heads=0, k_out_stride_token=512), False),
    (_rotary, {}, False),
]


@pytest.mark.parametrize("call,change,refused", CASES, ids=lambda v: getattr(v, "__name__", str(v)))
def test_an_output_over_its_input_has_its_strides(bfp8, call, change, refused):
    if torch.cuda.is_available() and not refused:
        pytest.skip("the placeholder addresses are looked at where there is a GPU")
    assert (call(bfp8, **change) == INVAL) == refused
