"""Linear attention on the GPU where its arguments leave the ordinary range: decays at the end of
fp32's range, non-finite values inside a sequence."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
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


def test_a_long_chain_beside_short_sequences_keeps_a_low_wait_limit():
    """Six heads of 65536 rows, 180 of at most one: the segments of a chain (19 of 3456 rows) all start at
    once and the last one waits for the others, 18 * 3456 rows at 50 cycles, 3.1e6.  With the lowest
    limit, 1e5 cycles, the call grants its chains 500 cycles for each of their rows, 3.3e7."""
    B, L, H, dk, dv = 31, 65536, 6, 8, 8
    g = torch.Generator(device="cuda").manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    lengths = torch.tensor([L] + [1, 0] * 15, dtype=torch.int32, device="cuda")
    dev = dict(q=n(B, L, 1, dk), k=n(B, L, 1, dk), v=n(B, L, H, dv), lengths=lengths,
               log_decay=torch.full((1, 1, H), -0.01, device="cuda").expand(B, L, H))
    want = prefill(dev, B, L, H, dv, dk)
    try:
        assert hy.hymba_set_wait_limit(1) == 100000
        o, S = prefill(dev, B, L, H, dv, dk)
    finally:
        hy.hymba_set_wait_limit(0)
    assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    assert bool(torch.isfinite(S[0]).all()) and bool((S[0] != 0).any())


def test_another_device_or_a_host_workspace_is_refused():
    """Before any launch: a description of tensors of another GPU than the current one (one index further
    here), and a workspace on the host."""
    x = on_gpu(inputs("bf16", 1, 300, 2, 1, 16, 16))
    o, S = torch.zeros(1, 300, 2, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 16, 16, device="cuda")
    args = hy.make_linear_attention(o=o, state_out=S, **x)
    n = hy.hymba_linear_attention_workspace(args)
    with pytest.raises(ValueError, match="workspace is on cpu"):
        hy.hymba_linear_attention_prefill(args, torch.empty(n + 256, dtype=torch.uint8), n)
    assert args.device == o.device
    args.device, args.check_device = torch.device("cuda", o.device.index + 1), True
    with pytest.raises(ValueError, match="not the current device"):
        hy.hymba_linear_attention_prefill(args, torch.empty(n + 256, dtype=torch.uint8, device="cuda"), n)
    assert not bool(o.any())
