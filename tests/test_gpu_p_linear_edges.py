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


@pytest.mark.parametrize("dtype,B,L,H,dk", [("bf16", 1, 300, 2, 64), ("bf16", 1, 30, 2, 64), ("f32", 1, 300, 2, 64),
                                            ("bf16", 1, 300, 2, 128)])
@pytest.mark.parametrize("name", ["log_decay", "in_scale", "q", "k", "gate"])
@pytest.mark.parametrize("t", [3, 7, 27])
def test_a_non_finite_value_reaches_no_row_before_its_own(name, t, dtype, B, L, H, dk):
    """NaN in the last of four rows, of the first sequence's first head: the rows before it and the other
    head, where it shares no row with the first, keep their bits."""
    x = inputs(dtype, B, L, H, H, dk, 64)
    clean, _ = prefill(on_gpu(x), B, L, H, 64, dk)
    for at in (t, L - 5):  # again in the last rows, which the last chunk holds
        bad = {**x, name: x[name].clone()}
        bad[name][0, at, 0] = float("nan")
        o, _ = prefill(on_gpu(bad), B, L, H, 64, dk)
        assert torch.equal(o[:, :at], clean[:, :at]) and torch.equal(o[:, :, 1:], clean[:, :, 1:])
        assert bool(o[0, at, 0].isnan().all())
        if name in ("log_decay", "in_scale", "k"):  # they reach the state
            assert bool(o[0, at:, 0].isnan().all())
        else:
            assert torch.equal(o[0, at + 1:], clean[0, at + 1:])
