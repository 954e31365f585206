"""Calls whose dynamic shared memory is at or just below the 48 KB that a kernel gets without asking, of which the kernel's
own arrays take a part."""

import numpy as np
import pytest
import torch

from test_gpu_kv_cache import _check_plan, _random_plan
from test_gpu_residual_norm import _check, _inputs, _outputs, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [5121, 5128, 5632, 6137, 6144])
@pytest.mark.parametrize("gate", [None, "token"])
def test_residual_norm_of_many_rows(bfp8, cuda_device, H, gate):
    """Six warps a row with four vectors a thread keep 48 KB of factors."""
    t, out = _inputs(cuda_device, 1000, H, gate, torch.bfloat16, H), _outputs(cuda_device, 1000, H)
    _run(bfp8, t, out, residual_scale=0.75)
    _check(t, out)


@pytest.mark.parametrize("B", [6100, 6121, 6144, 6145])
def test_plans_of_some_thousand_requests(bfp8, cuda_device, B):
    """Eight bytes a request: 48 KB at 6144."""
    ctx, new, free, table = _random_plan(np.random.default_rng(B), B, 16, 2, 40)
    _check_plan(bfp8, cuda_device, ctx, new, free, table, 16, int(new.sum()) + 5)
