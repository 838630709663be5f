"""Head norm and rotation on the GPU against the plain 64-bit form."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
from tests import _operators as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def bound(dtype, want, size):
    """fp32 arithmetic: the mean square (13 roundings at most), its root, two products of the norm,
    the factors' own roundings and angle (three steps of pi), and the rotation's two products and
    sum: under 32 half steps of the pair's size; then the rounding to storage."""
    return P.half_step(dtype) * want.abs() + 32 * P.F32_STEP * size + 1e-30


def run(q, k, qo, ko, **kw):
    hy.hymba_qk_norm_rope(hy.make_qk_norm_rope(q, k, qo, ko, **kw), torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())


CASES = [
    # dtype, B, R, Hq, Hk, d, rot, layout, scaling, norm, weights, given
    ("bf16", 2, 5, 25, 5, 64, 64, "pairs", "none", True, True, False),
    ("bf16", 3, 1, 25, 5, 64, 64, "halves", "none", True, True, False),
    ("bf16", 2, 131, 4, 2, 64, 64, "halves", "wavelength", True, True, True),
    ("bf16", 1, 9, 3, 1, 8, 8, "halves", "none", True, True, False),      # one lane per head
    ("bf16", 2, 7, 3, 3, 24, 24, "halves", "linear", True, False, True),  # halves 12 apart: through shared memory
    ("bf16", 2, 7, 5, 1, 40, 16, "halves", "linear", True, True, False),  # part of the head, halves 8 apart
    ("bf16", 2, 7, 5, 1, 96, 30, "pairs", "none", True, True, False),
    ("bf16", 1, 33, 2, 2, 256, 256, "halves", "wavelength", True, True, True),
    ("bf16", 1, 3, 2, 0, 256, 250, "halves", "none", False, False, False),
    ("bf16", 2, 3, 0, 5, 64, 0, "pairs", "none", True, True, False),      # norm alone, keys alone
    ("bf16", 2, 70, 3, 2, 16, 16, "halves", "none", True, True, False),   # one lane of 16 elements per head
    ("bf16", 2, 70, 3, 2, 48, 22, "pairs", "none", True, True, True),     # the last lanes idle, a pair border inside a lane
    ("bf16", 2, 7, 9, 4, 72, 72, "halves", "none", True, True, False),    # 8 elements a lane
    ("bf16", 2, 7, 9, 4, 88, 88, "pairs", "none", True, True, False),
    ("bf16", 3, 40, 11, 2, 240, 240, "halves", "linear", True, True, True),
    ("bf16", 2, 7, 9, 4, 80, 0, "pairs", "none", True, True, False),
    ("f32", 2, 5, 6, 3, 128, 40, "pairs", "linear", False, False, True),
    ("f32", 2, 17, 25, 5, 64, 64, "halves", "wavelength", True, True, False),
    ("f32", 1, 4, 3, 1, 256, 64, "pairs", "none", True, True, True),
    ("f32", 1, 4, 3, 1, 48, 44, "halves", "none", True, True, False),
]
SCALED = {"none": dict(base=10000.0), "linear": dict(base=10000.0, factor=8.0),
          "wavelength": dict(base=500000.0, factor=4.0, orig_len=2048.0, low_turns=1.0, high_turns=4.0)}


@pytest.mark.parametrize("dtype,B,R,Hq,Hk,d,rot,layout,scaling,norm,weights,given", CASES)
def test_heads_match_the_plain_form(dtype, B, R, Hq, Hk, d, rot, layout, scaling, norm, weights, given):
    g = torch.Generator().manual_seed(7)
    dt = DT[dtype]
    fused = (torch.randn(B, R, Hq + Hk + 2, d, generator=g) * torch.logspace(-2, 2, Hq + Hk + 2)[:, None]).to(dt)
    wq, wk = (1 + torch.randn(d, generator=g)) if weights else None, (1 + torch.randn(d, generator=g)) if weights else None
    given_pos = torch.randint(0, 1 << 20, (B, R), generator=g)
    pos0, m = 8191, 1.25
    dev = fused.cuda()
    q, k = dev[:, :, :Hq], dev[:, :, Hq:Hq + Hk]
    # keys go into slots of a [B, Hk, cap, d] store, queries into a dense buffer
    qo = torch.full((B, R, max(Hq, 1), d), 9.0, dtype=dt, device="cuda")
    store = torch.full((B, max(Hk, 1), R + 6, d), 9.0, dtype=dt, device="cuda")
    ko = store[:, :, 3:R + 3].transpose(1, 2)
    rope = hy.make_rope(rot, layout, scaling=scaling, attn_factor=m, **SCALED[scaling]) if rot else None
    run(q if Hq else None, k if Hk else None, qo if Hq else None, ko if Hk else None, norm=norm, eps=1e-5,
        q_weight=wq.cuda() if weights and Hq else None, k_weight=wk.cuda() if weights and Hk else None, rope=rope,
        pos0=0 if given else pos0, positions=given_pos.cuda() if given else None)
    pos = given_pos if given else (pos0 + torch.arange(R)).expand(B, R)
    freq = P.frequencies(rot, scaling=scaling, **SCALED[scaling])
    for name, x, w, out in (("q", fused[:, :, :Hq], wq, qo), ("k", fused[:, :, Hq:Hq + Hk], wk, ko)):
        if x.shape[2]:
            want, size = P.heads(x, w, norm, 1e-5, pos, rot, layout, m, freq)
            P.within(out, want, bound(dt, want, size), name)
    assert torch.equal(dev.cpu(), fused), "the inputs were written"
    if Hk:
        assert bool((store[:, :, :3] == 9).all()) and bool((store[:, :, R + 3:] == 9).all()), "other slots were written"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place_equals_out_of_place(dtype):
    g = torch.Generator().manual_seed(8)
    x = torch.randn(3, 11, 6, 64, generator=g).to(DT[dtype]).cuda()
    rope = hy.make_rope(48, "halves")
    out = torch.empty(3, 11, 6, 64, dtype=DT[dtype], device="cuda")
    run(x[:, :, :4], x[:, :, 4:], out[:, :, :4], out[:, :, 4:], rope=rope, pos0=5)
    y = x.clone()
    run(y[:, :, :4], y[:, :, 4:], None, None, rope=rope, pos0=5)
    assert torch.equal(y, out)


def test_zero_rows_and_non_finite_rows_stay_in_their_head():
    """A head of zeros normalises to zeros (eps > 0); a NaN or infinity spoils its own head only."""
    x = torch.randn(1, 2, 4, 64, generator=torch.Generator().manual_seed(9)).bfloat16().cuda()
    x[0, 0, 1] = 0
    ref = torch.empty_like(x)
    run(x, None, ref, None, rope=hy.make_rope(64))
    assert bool((ref[0, 0, 1] == 0).all())
    x[0, 0, 2, 5] = float("inf")
    x[0, 1, 0, 63] = float("nan")
    out = torch.empty_like(x)
    run(x, None, out, None, rope=hy.make_rope(64))
    keep = torch.ones(2, 4, dtype=torch.bool, device="cuda")
    keep[0, 2] = keep[1, 0] = False
    assert torch.equal(out[0][keep], ref[0][keep])
    assert bool(out[0, 1, 0].isnan().all())


def test_far_positions_keep_their_angles():
    """Positions up to 2^40: the angle is reduced in fp64, so the rotation stays a rotation by the
    right angle (fp64 position times fp64 frequency: 2^40 * 2^-53 turns)."""
    pos = torch.tensor([[0, 1, (1 << 24) + 1, (1 << 33) + 7, 1 << 40]])
    x = torch.randn(1, 5, 2, 64, generator=torch.Generator().manual_seed(10))
    out = torch.empty(1, 5, 2, 64, device="cuda")
    run(x.cuda(), None, out, None, norm=False, rope=hy.make_rope(64), positions=pos.cuda())
    want, size = P.heads(x, None, False, 0.0, pos, 64, "pairs", 1.0, P.frequencies(64, 10000.0))
    # the plain form's own angle p f carries 2^40 2^-53 radians as well
    P.within(out, want, bound(torch.float32, want, size) + 2.0 ** -10 * size, "far")
    P.within(out[:, :4], want[:, :4], bound(torch.float32, want[:, :4], size[:, :4]) + 2.0 ** -17 * size[:, :4], "nearer")


def test_captured_call_replays_on_new_inputs_and_another_stream():
    x = torch.randn(4, 1, 30, 64, generator=torch.Generator().manual_seed(11)).bfloat16()
    buf, out = x.cuda(), torch.empty(4, 1, 30, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([[5], [6], [7], [8]], device="cuda")
    args = hy.make_qk_norm_rope(buf[:, :, :25], buf[:, :, 25:], out[:, :, :25], out[:, :, 25:], rope=hy.make_rope(64),
                                positions=pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        hy.hymba_qk_norm_rope(args, torch.cuda.current_stream())
    for step in range(2):
        buf.copy_(x * (step + 1))
        pos.add_(1)
        graph.replay()
        torch.cuda.synchronize()
        want, size = P.heads((x * (step + 1)).bfloat16(), None, True, 1e-6, pos.cpu(), 64, "pairs", 1.0,
                             P.frequencies(64, 10000.0))
        P.within(out, want, bound(torch.bfloat16, want, size), f"replay {step}")
