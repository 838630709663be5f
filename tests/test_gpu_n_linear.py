"""Linear attention on the GPU (whole sequences and single tokens) against the plain 64-bit form."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
from tests import _operators as P

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def inputs(dtype, B, L, H, K, dk, dv, decay="token", epilogue=True, start=True, lengths=None, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DT[dtype]
    x = dict(q=(n(B, L, K, dk) * dk ** -0.5).to(dt), k=n(B, L, K, dk).to(dt), v=n(B, L, H, dv).to(dt))
    if decay == "token":
        delta = torch.nn.functional.softplus(n(B, L, H) - 2)
        x["log_decay"], x["in_scale"] = -(1 + 3 * torch.rand(H, generator=g)) * delta, delta
    elif decay == "head":
        x["log_decay"] = torch.log1p(-torch.exp2(-4 - 4 * torch.rand(H, generator=g))).expand(B, L, H)
    elif decay == "strong":  # steps of up to 30, so that a chunk spans hundreds
        x["log_decay"] = -30 * torch.rand(B, L, H, generator=g)
    if epilogue:
        x["skip"], x["gate"] = n(H, dv), n(B, L, H, dv).to(dt)
    if start:
        x["state_in"] = n(B, H, dv, dk)
    if lengths is not None:
        x["lengths"] = torch.tensor(lengths, dtype=torch.int32)
    x["scale"] = scale
    return x


def on_gpu(x):
    out = {}
    for k, v in x.items():
        if not torch.is_tensor(v):
            out[k] = v
        elif 0 in v.stride():
            out[k] = v[tuple(slice(0, 1) if st == 0 else slice(None) for st in v.stride())].cuda().expand(v.shape)
        else:
            out[k] = v.cuda()
    return out


def prefill(dev, B, L, H, dv, dk, o=None, state_out=None):
    o = torch.full((B, L, H, dv), 7.0, dtype=dev["q"].dtype, device="cuda") if o is None else o
    state_out = torch.full((B, H, dv, dk), 7.0, device="cuda") if state_out is None else state_out
    args = hy.make_linear_attention(o=o, state_out=state_out, **dev)
    ws = torch.empty(max(hy.hymba_linear_attention_workspace(args), 1), dtype=torch.uint8, device="cuda")
    hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    return o, state_out


def check(x, o, S, dtype, what=""):
    L, dk = x["q"].shape[1], x["q"].shape[3]
    base = torch.full(tuple(x["v"].shape), 7.0)
    want, Sw, size, Ssize = P.linear(o=base, **x)
    chunked = dtype == "bf16"
    bo, bs = P.linear_bounds(DT[dtype], L, dk, want, size, Sw, Ssize, chunked)
    P.within(o, want, bo, what + "o")
    P.within(S, Sw, bs, what + "state")


# dtype, B, L, H, K, dk, dv, decay, epilogue, start, lengths
CASES = [
    ("bf16", 2, 1, 4, 1, 64, 128, "token", True, True, None),
    ("bf16", 1, 2, 3, 3, 16, 64, "token", False, False, None),
    ("bf16", 2, 127, 4, 2, 64, 128, "token", True, True, None),
    ("bf16", 1, 128, 2, 1, 64, 128, "head", False, True, None),
    ("bf16", 2, 129, 2, 1, 128, 128, "token", True, False, None),
    ("bf16", 1, 300, 3, 1, 64, 128, "token", True, True, None),
    ("bf16", 1, 257, 4, 4, 128, 64, "head", True, True, None),
    ("bf16", 2, 140, 6, 2, 24, 40, "token", True, True, None),
    ("bf16", 1, 133, 2, 2, 72, 256, "token", False, True, None),
    ("bf16", 1, 200, 2, 1, 8, 8, "none", True, True, None),
    ("bf16", 1, 200, 2, 1, 104, 136, "strong", True, True, None),
    ("bf16", 5, 260, 2, 1, 64, 128, "token", True, True, [0, 1, 128, 200, 999]),
    ("bf16", 4, 37, 2, 2, 32, 32, "head", False, False, [37, -3, 36, 2]),
    # rows split over the SMs: segments' states first, then their outputs
    ("bf16", 2, 1000, 2, 1, 64, 128, "token", True, True, None),
    ("bf16", 3, 900, 2, 2, 128, 72, "head", True, True, [0, 130, 900]),
    ("bf16", 1, 1290, 1, 1, 16, 200, "strong", False, False, None),
    # more heads than SMs: chains of segments
    ("bf16", 30, 1030, 5, 1, 32, 64, "token", True, True, [0, 1, 128, 513, 1029] + [1030] * 25),
    # few rows: one after another
    ("bf16", 2, 9, 3, 1, 72, 40, "token", True, True, [9, 4]),
    ("f32", 2, 1, 4, 1, 64, 128, "token", True, True, None),
    ("f32", 2, 33, 4, 2, 64, 128, "token", True, True, None),
    ("f32", 1, 200, 3, 1, 128, 72, "head", True, True, None),
    ("f32", 2, 150, 4, 2, 80, 96, "head", True, True, [150, 77]),
    ("f32", 1, 700, 2, 1, 96, 24, "token", True, True, None),
    ("f32", 2, 70, 2, 2, 16, 256, "token", False, False, None),
    ("f32", 1, 50, 2, 1, 40, 8, "none", True, True, None),
    ("f32", 1, 90, 2, 1, 32, 64, "strong", True, True, None),
    ("f32", 4, 40, 2, 1, 24, 40, "token", True, True, [0, 1, 40, 17]),
]


@pytest.mark.parametrize("dtype,B,L,H,K,dk,dv,decay,epilogue,start,lengths", CASES)
def test_prefill_matches_the_plain_form(dtype, B, L, H, K, dk, dv, decay, epilogue, start, lengths):
    x = inputs(dtype, B, L, H, K, dk, dv, decay, epilogue, start, lengths, scale=0.75)
    o, S = prefill(on_gpu(x), B, L, H, dv, dk)
    check(x, o, S, dtype)
    if lengths is not None:  # rows behind a sequence's end are as they were
        for b, n in enumerate(lengths):
            assert bool((o[b, max(0, n):] == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_behind_a_sequence_hold_anything(dtype):
    """Infinities and NaN in the padding, in every input, change nothing."""
    B, L, H, K, dk, dv = 3, 150, 2, 1, 32, 64
    lengths = [0, 77, 130]
    x = inputs(dtype, B, L, H, K, dk, dv, lengths=lengths)
    clean = prefill(on_gpu(x), B, L, H, dv, dk)
    for name in ("q", "k", "v", "gate", "log_decay", "in_scale"):
        for b, n in enumerate(lengths):
            x[name][b, n::2] = float("nan")
            x[name][b, n + 1::2] = float("inf")
    dirty = prefill(on_gpu(x), B, L, H, dv, dk)
    assert torch.equal(clean[0], dirty[0]) and torch.equal(clean[1], dirty[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_decay_of_zero_forgets(dtype):
    """log decay -infinity (and the type's lowest value): two documents in one row of tokens equal the
    second alone from there on, also where a chunk holds the border."""
    B, L, H, K, dk, dv, cut = 1, 190, 2, 1, 32, 64, 70
    x = inputs(dtype, B, L, H, K, dk, dv)
    x["log_decay"] = x["log_decay"].clone()
    x["log_decay"][:, cut, 0] = -float("inf")
    x["log_decay"][:, cut, 1] = torch.finfo(torch.float32).min
    o, S = prefill(on_gpu(x), B, L, H, dv, dk)
    check(x, o, S, dtype)
    tail = {k: (v[:, cut:].contiguous() if torch.is_tensor(v) and k not in ("skip", "state_in") else v) for k, v in x.items()}
    tail.pop("state_in")
    o2, S2 = prefill(on_gpu(tail), B, L - cut, H, dv, dk)
    check(tail, o2, S2, dtype, "second document alone: ")
    assert bool(torch.isfinite(o).all()) and bool(torch.isfinite(S).all())


def test_no_decay_and_null_options():
    x = inputs("bf16", 1, 140, 2, 1, 64, 128, decay="none", epilogue=False, start=False)
    o, S = prefill(on_gpu(x), 1, 140, 2, 128, 64)
    check(x, o, S, "bf16")
    # without state_out only o is written
    o2 = torch.zeros_like(o)
    args = hy.make_linear_attention(o=o2, **on_gpu(x))
    ws = torch.empty(max(hy.hymba_linear_attention_workspace(args), 1), dtype=torch.uint8, device="cuda")
    hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    assert torch.equal(o, o2)


@pytest.mark.parametrize("dtype,L", [("bf16", 135), ("f32", 135), ("bf16", 1100)])
def test_strided_views_and_states_in_place(dtype, L):
    """q, k, v, gate as slices of one fused row, heads outermost in o, one state for every sequence,
    then the state continued in place (with 1100 rows by segments, whose first one reads it)."""
    B, H, K, dk, dv = 2, 4, 2, 32, 64
    x = inputs(dtype, B, L, H, K, dk, dv)
    x["state_in"] = x["state_in"][:1].expand(B, -1, -1, -1)
    width = 2 * K * dk + 2 * H * dv + 32
    fused = torch.zeros(B, L, width, dtype=DT[dtype], device="cuda")
    at, views = 0, {}
    for name, h, d in (("q", K, dk), ("k", K, dk), ("v", H, dv), ("gate", H, dv)):
        views[name] = fused[:, :, at:at + h * d].unflatten(2, (h, d))
        views[name].copy_(x[name])
        at += h * d
    dev = {**on_gpu(x), **views}
    o = torch.zeros(H, B, L, dv, dtype=DT[dtype], device="cuda").permute(1, 2, 0, 3)
    o, S = prefill(dev, B, L, H, dv, dk, o=o)
    check(x, o, S, dtype)
    first = S.clone()
    dev["state_in"] = S
    o2, S2 = prefill(dev, B, L, H, dv, dk, state_out=S)
    check({**x, "state_in": first.cpu()}, o2, S2, dtype, "continued in place: ")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_halves_equal_the_whole(dtype):
    B, L, H, K, dk, dv, cut = 2, 333, 2, 1, 64, 128, 150
    x = inputs(dtype, B, L, H, K, dk, dv, decay="head")
    dev = on_gpu(x)
    part = lambda lo, hi, st: {k: (v[:, lo:hi] if torch.is_tensor(v) and k not in ("skip", "state_in") else v)  # noqa: E731
                               for k, v in {**dev, "state_in": st}.items()}
    oa, Sa = prefill(part(0, cut, dev["state_in"]), B, cut, H, dv, dk)
    ob, Sb = prefill(part(cut, L, Sa), B, L - cut, H, dv, dk)
    check(x, torch.cat((oa, ob), 1), Sb, dtype)


@pytest.mark.parametrize("dtype,B,H,K,dk,dv,decay,epilogue,start,lengths", [
    ("bf16", 3, 25, 5, 64, 128, "token", True, True, None),
    ("bf16", 150, 4, 1, 64, 128, "head", True, True, None),
    ("bf16", 2, 4, 2, 8, 8, "token", False, True, None),
    ("bf16", 2, 4, 2, 104, 256, "none", True, False, None),
    ("f32", 2, 4, 2, 24, 40, "token", True, True, None),
    ("f32", 5, 3, 1, 128, 136, "head", True, True, [1, 0, 1, -1, 5]),
    ("bf16", 4, 2, 1, 72, 64, "token", True, True, [0, 0, 1, 0]),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_step_matches_the_plain_form(dtype, B, H, K, dk, dv, decay, epilogue, start, lengths, in_place):
    x = inputs(dtype, B, 1, H, K, dk, dv, decay, epilogue, start or in_place, lengths, scale=1.25)
    dev = on_gpu(x)
    o = torch.full((B, 1, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    out = dev["state_in"] if in_place else torch.full((B, H, dv, dk), 7.0, device="cuda")
    hy.hymba_linear_attention_decode_step(hy.make_linear_attention(o=o, state_out=out, **dev),
                                          torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    want, Sw, size, Ssize = P.linear(o=torch.full((B, 1, H, dv), 7.0), **x)
    bo, bs = P.linear_bounds(DT[dtype], 1, dk, want, size, Sw, Ssize, chunked=False)
    P.within(o, want, bo, "o")
    P.within(out, Sw, bs, "state")


def test_idle_rows_with_non_finite_inputs_keep_state_and_output():
    x = inputs("bf16", 2, 1, 2, 1, 64, 128, lengths=[0, 1])
    for name in ("q", "k", "v", "gate", "log_decay", "in_scale"):
        x[name][0] = float("nan")
    dev = on_gpu(x)
    o = torch.full((2, 1, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 2, 128, 64, device="cuda")
    hy.hymba_linear_attention_decode_step(hy.make_linear_attention(o=o, state_out=out, **dev), torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    assert torch.equal(out[0].cpu(), x["state_in"][0]) and bool((o[0] == 7).all())
    assert bool(torch.isfinite(out[1]).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_then_steps_equal_the_whole_prompt(dtype):
    """As a program uses them: rotate and norm, take a prompt, then single tokens on its state."""
    B, L, H, K, dk, dv, n = 2, 140, 4, 2, 64, 128, 5
    x = inputs(dtype, B, L + n, H, K, dk, dv)
    rope = hy.make_rope(dk, "halves")
    dev = on_gpu(x)
    qk = hy.make_qk_norm_rope(dev["q"], dev["k"], norm=True, rope=rope)
    hy.hymba_qk_norm_rope(qk, torch.cuda.current_stream())
    x["q"], x["k"] = dev["q"].cpu(), dev["k"].cpu()
    cut = lambda lo, hi: {k: (v[:, lo:hi] if torch.is_tensor(v) and k not in ("skip", "state_in") else v)  # noqa: E731
                          for k, v in dev.items()}
    o = torch.full((B, L + n, H, dv), 7.0, dtype=DT[dtype], device="cuda")
    _, S = prefill(cut(0, L), B, L, H, dv, dk, o=o[:, :L])
    for t in range(L, L + n):
        step = {**cut(t, t + 1), "state_in": S}
        hy.hymba_linear_attention_decode_step(hy.make_linear_attention(o=o[:, t:t + 1], state_out=S, **step),
                                              torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    check(x, o, S, dtype)


def test_long_sequence_keeps_a_slow_decay():
    """8320 rows of one decay near one: the state is a long sum whose weights must not drift.  Against
    the closed form sum_j a^(L-1-j) k_j v_j in fp64; the 2-norm is held to 2e-6 (fp32 roundings of the
    sum are independent: about sqrt(rows in memory) half steps)."""
    for dtype in ("bf16", "f32"):
        B, L, H, dk, dv = 1, 8320, 2, 32, 64
        x = inputs(dtype, B, L, H, 1, dk, dv, decay="none", epilogue=False, start=False)
        g = torch.tensor([-1 / 700.0, -1 / 1500.0])
        x["log_decay"] = g.expand(B, L, H)
        o, S = prefill(on_gpu(x), B, L, H, dv, dk)
        w = torch.exp(g.double()[:, None] * torch.arange(L - 1, -1, -1))
        want = torch.einsum("hl,lhv,lk->hvk", w, x["v"][0].double(), x["k"][0, :, 0].double())
        rel = float((S[0].cpu().double() - want).norm() / want.norm())
        assert rel <= 2e-6, (dtype, rel)
        last = torch.einsum("hvk,k->hv", want, x["q"][0, -1, 0].double())
        tol = 2 * P.half_step(DT[dtype]) + 2e-5
        assert float((o[0, -1].cpu().double() - last).norm() / last.norm()) <= tol


def test_captured_prefill_and_step_replay():
    B, L, H, K, dk, dv = 2, 260, 3, 1, 64, 128
    x = inputs("bf16", B, L, H, K, dk, dv)
    dev = on_gpu(x)
    o = torch.full((B, L, H, dv), 7.0, dtype=torch.bfloat16, device="cuda")
    S = torch.zeros(B, H, dv, dk, device="cuda")
    args = hy.make_linear_attention(o=o, state_out=S, **dev)
    one = {k: (v[:, :1] if torch.is_tensor(v) and k not in ("skip", "state_in") else v) for k, v in dev.items()}
    o1 = torch.zeros(B, 1, H, dv, dtype=torch.bfloat16, device="cuda")
    step = hy.make_linear_attention(o=o1, state_out=S, **{**one, "state_in": S})
    ws = torch.empty(max(hy.hymba_linear_attention_workspace(args), 1), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
        hy.hymba_linear_attention_decode_step(step, torch.cuda.current_stream())
    for rep in range(2):
        x["v"] = x["v"] * (1 + rep)
        dev["v"].copy_(x["v"])
        graph.replay()
        torch.cuda.synchronize()
        base = torch.full((B, L, H, dv), 7.0)
        want, Sw, size, Ssize = P.linear(o=base, **x)
        bo, _ = P.linear_bounds(torch.bfloat16, L, dk, want, size, Sw, Ssize, True)
        P.within(o, want, bo, f"replay {rep}")
        xs = {k: (v[:, :1] if torch.is_tensor(v) and k not in ("skip", "state_in") else v) for k, v in x.items()}
        want1, S1, size1, Ssize1 = P.linear(o=base[:, :1], **{**xs, "state_in": Sw})
        _, bs = P.linear_bounds(torch.bfloat16, L + 1, dk, want1, size1, S1, Ssize1 + Ssize, True)
        P.within(S, S1, bs, f"state after replay {rep}")


@pytest.mark.parametrize("dtype,B,L,H,K,dk,dv", [("bf16", 8, 1000, 25, 1, 64, 128), ("bf16", 4, 700, 9, 3, 128, 72),
                                                 ("f32", 4, 300, 6, 1, 64, 128)])
def test_repeated_calls_give_the_same_bits(dtype, B, L, H, K, dk, dv):
    """Many CTAs, every stage of their pipelines reused: 300 calls, bit for bit."""
    x = inputs(dtype, B, L, H, K, dk, dv)
    dev = on_gpu(x)
    o = torch.zeros(B, L, H, dv, dtype=DT[dtype], device="cuda")
    S = torch.zeros(B, H, dv, dk, device="cuda")
    args = hy.make_linear_attention(o=o, state_out=S, **dev)
    ws = torch.empty(max(hy.hymba_linear_attention_workspace(args), 1), dtype=torch.uint8, device="cuda")
    first = None
    for i in range(300):
        o.zero_()
        hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
        if first is None:
            first = o.clone(), S.clone()
        assert torch.equal(o, first[0]) and torch.equal(S, first[1]), i
    hy.hymba_stream_status(torch.cuda.current_stream())


@pytest.mark.parametrize("dk,dv,pad,off", [(64, 128, 8, 0), (64, 72, 0, 8), (128, 40, 8, 8), (16, 16, 8, 24)])
def test_outputs_off_sector_boundaries(dk, dv, pad, off):
    """Rows of o that start 16 but not 32 bytes into a sector: the dense call's bits, and nothing beside them."""
    B, L, H, K = 2, 300, 3, 1
    x = inputs("bf16", B, L, H, K, dk, dv, lengths=[300, 77])
    want, Sw = prefill(on_gpu(x), B, L, H, dv, dk)
    wide = torch.full((B, L, H * (dv + pad) + 32), 7.0, dtype=torch.bfloat16, device="cuda")
    o = wide[:, :, off:off + H * (dv + pad)].unflatten(2, (H, dv + pad))[..., :dv]
    got, S = prefill(on_gpu(x), B, L, H, dv, dk, o=o)
    assert torch.equal(got, want) and torch.equal(S, Sw)
    got.fill_(7.0)
    assert bool((wide == 7.0).all())


def test_chains_at_once_and_replayed():
    """More heads than SMs: two calls at a time on streams of their own, then as a graph's replays."""
    B, L, H, K, dk, dv = 6, 1030, 30, 2, 64, 64
    x = inputs("bf16", B, L, H, K, dk, dv, lengths=[1030, 0, 1, 513, 1030, 900])
    dev = on_gpu(x)
    want = prefill(dev, B, L, H, dv, dk)
    calls = []
    for _ in range(2):
        o = torch.full((B, L, H, dv), 7.0, dtype=torch.bfloat16, device="cuda")
        S = torch.empty(B, H, dv, dk, device="cuda")
        args = hy.make_linear_attention(o=o, state_out=S, **dev)
        ws = torch.full((hy.hymba_linear_attention_workspace(args),), 255, dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        calls.append((o, S, args, ws, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for o, S, args, ws, s in calls:
            hy.hymba_linear_attention_prefill(args, ws, ws.numel(), s)
    torch.cuda.synchronize()
    hy.hymba_stream_status(torch.cuda.current_stream())
    for o, S, *_ in calls:
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
    o, S, args, ws, s = calls[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
    for _ in range(3):
        o.fill_(7.0)
        S.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(S, want[1])
