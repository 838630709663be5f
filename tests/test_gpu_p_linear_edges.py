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


@pytest.mark.parametrize("dtype,L", [("bf16", 150), ("bf16", 9), ("f32", 60)])
@pytest.mark.parametrize("order", [(2, 0, 1), (1, 0, 2), (1, 2, 0), (2, 1, 0)])
def test_any_order_of_sequences_rows_and_heads(dtype, L, order):
    """q, k, v, gate, o, log_decay and in_scale stored with their dimensions in another order give the bits
    of the dense call: a row's stride below its sequence's or its head's, or above both."""
    B, nh, K, dk, dv = 3, 4, 2, 40, 72
    x = inputs(dtype, B, L, nh, K, dk, dv, lengths=[L, 3, L - 1])
    dev = on_gpu(x)
    want = prefill(dev, B, L, nh, dv, dk)
    back = [order.index(i) for i in range(3)]

    def moved(t):
        rest = list(range(3, t.ndim))
        return t.permute(*order, *rest).contiguous().permute(*back, *rest)

    other = {n: moved(t) if n in ("q", "k", "v", "gate", "log_decay", "in_scale") else t for n, t in dev.items()}
    o = moved(torch.full((B, L, nh, dv), 7.0, dtype=DT[dtype], device="cuda"))
    got = prefill(other, B, L, nh, dv, dk, o=o)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("far", ["row", "batch", "head"])
def test_offsets_beyond_32_bits(dtype, far):
    """Rows, sequences or heads 2^27 .. 2^32 elements apart in one buffer (8.6 GB and more): the dense call's
    bits, from the whole sequences, a single token and the head norm/rotation."""
    B, L, nh, K, dk, dv = 2, 40, 2, 1, 64, 64
    x = inputs(dtype, B, L, nh, K, dk, dv, epilogue=True, start=True)
    dev = on_gpu(x)
    extent = {"row": L, "batch": B, "head": nh}[far]
    step = (1 << 32) // (extent - 1) // 8 * 8 + 8
    buf = torch.empty((extent - 1) * step + B * L * nh * dv * 8 + 65536, dtype=DT[dtype], device="cuda")
    at = 0

    def place(t):
        nonlocal at
        b, r, h, d = t.shape
        st = {"row": (h * d * 5, step, d * 5), "batch": (step, h * d, d), "head": (r * d, d, step)}[far]
        view = buf.as_strided((b, r, h, d), (*st, 1), at)
        at += sum((n - 1) * s for n, s, f in zip((b, r, h), st, ("batch", "row", "head")) if f != far) + d
        at = (at + 63) // 64 * 64
        view.copy_(t)
        return view

    assert (extent - 1) * step >= 1 << 32
    apart = {n: place(t) if n in ("q", "k", "v", "gate") else t for n, t in dev.items()}
    o = place(torch.full((B, L, nh, dv), 7.0, dtype=DT[dtype], device="cuda"))
    assert at <= B * L * nh * dv * 8 + 65536
    want, got = prefill(dev, B, L, nh, dv, dk), prefill(apart, B, L, nh, dv, dk, o=o)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for n in ("q", "k", "v", "gate"):
        assert torch.equal(apart[n], dev[n]), n
    last = lambda y: {n: t[:, -1:] if torch.is_tensor(t) and n not in ("skip", "state_in") else t for n, t in y.items()}  # noqa: E731
    for src, out in ((dev, want[0]), (apart, o)):
        state = torch.empty(B, nh, dv, dk, device="cuda")
        hy.hymba_linear_attention_decode_step(hy.make_linear_attention(o=out[:, -1:], state_out=state, **last(src)),
                                              torch.cuda.current_stream())
    qk = [hy.make_qk_norm_rope(y["v"], y["q"], y["v"], y["q"], rope=hy.make_rope(64, "halves")) for y in (dev, apart)]
    for a in qk:
        hy.hymba_qk_norm_rope(a, torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    assert torch.equal(o, want[0]) and torch.equal(apart["v"], dev["v"]) and torch.equal(apart["q"], dev["q"])
