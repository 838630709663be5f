"""Linear attention on the GPU where its arguments leave the ordinary range: decays at the end of
fp32's range, non-finite values inside a sequence."""
from __future__ import annotations

import pytest
import torch

from tests import _operators as P
from tests.test_gpu_n_linear import DT, check, inputs, on_gpu, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,L", [("bf16", 30), ("f32", 30), ("f32", 200), ("bf16", 200)])
@pytest.mark.parametrize("row", [0, 3, 8])
def test_decays_below_the_normal_range_scale_nothing_behind_them(dtype, L, row):
    """exp(g) of -88 to -103.9 is subnormal in fp32 and holds few bits or one.  What it leaves of the state
    before it (below 1e-36 here) is nothing beside the rows behind it, which it must not touch."""
    x = inputs(dtype, 1, L, 6, 1, 64, 64, decay="none", epilogue=False)
    g = torch.full((1, L, 6), -0.01)
    g[:, row] = torch.tensor([-88.0, -95.0, -100.0, -103.0, -103.5, -103.9])
    x["log_decay"] = g
    x["v"] = x["v"].clone()
    x["v"][:, row:row + 3] *= 64
    o, S = prefill(on_gpu(x), 1, L, 6, 64, 64)
    check(x, o, S, dtype)
