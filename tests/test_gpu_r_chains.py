"""Linear attention in chains of segments (more heads than SMs): wide heads, several blocks of dv, states
in place, non-finite values, and inside the layer's batch chunks."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
import synth
from oracle import hymba_oracle as O
from synth.configs import DIMS_1P5B, Workload
from tests import _harness as H
from tests import _operators as P
from tests.test_gpu_n_linear import DT, inputs, on_gpu, prefill
from tests.test_gpu_o_layer_heads import set_heads, set_linear, state_close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,L,nh,K,dk,dv,decay,epilogue,lengths", [
    (40, 1030, 4, 2, 128, 128, "token", True, None),
    (30, 1100, 5, 1, 104, 72, "head", False, [0, 1, 128, 513, 1099] + [1100] * 25),
    (19, 1030, 4, 1, 64, 200, "token", True, [1030, 0, 600] + [1030] * 16),   # two blocks of dv
    (19, 1030, 4, 4, 128, 256, "strong", True, None),
    (150, 2070, 1, 1, 16, 8, "head", False, None),
])
@pytest.mark.parametrize("in_place", [False, True])
def test_chains_match_the_plain_form(B, L, nh, K, dk, dv, decay, epilogue, lengths, in_place):
    x = inputs("bf16", B, L, nh, K, dk, dv, decay, epilogue, True, lengths, scale=0.75)
    dev = on_gpu(x)
    o, S = prefill(dev, B, L, nh, dv, dk, state_out=dev["state_in"] if in_place else None)
    some = [0, 2, B - 1]
    part = {k: (v[some] if torch.is_tensor(v) and k != "skip" else v) for k, v in x.items()}
    want, Sw, size, Ssize = P.linear(o=torch.full((len(some), L, nh, dv), 7.0), **part)
    bo, bs = P.linear_bounds(DT["bf16"], L, dk, want, size, Sw, Ssize, True)
    P.within(o[some], want, bo, "o")
    P.within(S[some], Sw, bs, "state")
    if lengths is not None:
        for b, n in enumerate(lengths):
            assert bool((o[b, n:] == 7).all())


def test_repeated_chains_of_wide_heads_give_the_same_bits():
    B, L, nh, dk, dv = 19, 1030, 4, 128, 256
    x = inputs("bf16", B, L, nh, 1, dk, dv)
    dev = on_gpu(x)
    first = prefill(dev, B, L, nh, dv, dk)
    o, S = (torch.empty_like(t) for t in first)
    args = hy.make_linear_attention(o=o, state_out=S, **dev)
    ws = torch.empty(hy.hymba_linear_attention_workspace(args), dtype=torch.uint8, device="cuda")
    for i in range(60):
        o.zero_()
        hy.hymba_linear_attention_prefill(args, ws, ws.numel(), torch.cuda.current_stream())
        assert torch.equal(o, first[0]) and torch.equal(S, first[1]), i
    hy.hymba_stream_status(torch.cuda.current_stream())


def test_layer_batch_chunks_inside_a_chain():
    """Seven sequences of 25 linear heads (175 heads, chains of segments; a projection of 153 columns): in
    three batch chunks the serial call's bits, and one sequence against the oracle."""
    w = Workload("chain_layer", DIMS_1P5B, "bf16", 7, 128, 1000, 256)
    d, B, L, N = w.dims, w.batch, w.seq_rows, 64
    out = []
    for chunks in (0, 3):
        lay = H.GpuLayer(w, 0, branch_chunks=chunks)
        ow = H.oracle_weights(lay.cpu)
        ow["heads"], ow["linear"] = set_heads(lay, "halves"), set_linear(lay, N)
        x = synth.configs.x_tilde(w).cuda()
        k, v, kv = H.alloc_kv_seq(w, B, L)
        kc, vc, kvc = H.alloc_kv_cache(w, B, w.n_meta + w.window)
        h = torch.zeros(B, d.d_inner, N, device="cuda")
        c = torch.zeros(B, d.d_conv - 1, d.d_inner, dtype=torch.bfloat16, device="cuda")
        ssm = hy.hymba_ssm_cache(h.data_ptr(), c.data_ptr())
        y, _ = H.run_prefill(lay, x, kv, kvc, ssm)
        h1 = h.clone()
        xt = x[:, -1].contiguous()
        yt = torch.empty_like(xt)
        dws = H.workspace(hy.hymba_layer_decode_workspace(lay.handle, B, L))
        s = torch.cuda.current_stream()
        hy.hymba_layer_decode_step(lay.handle, B, L, xt, yt, kvc, ssm, dws, dws.numel(), s)
        hy.hymba_stream_status(s)
        out.append((y, k, h1, yt, h))
        if not chunks:
            b = B - 1
            r = O.layer_prefill(H.to64(x[b]), ow, lay.spec, capacity=w.n_meta + w.window)
            H.close_bf16(H.to64(y[b]), r["Y"], "Y")
            state_close(w, H.to64(h1[b]), r["h"], "state")
            got, cache = O.layer_decode(H.to64(xt[b]), L, ow, lay.spec,
                                        dict(k=r["k_cache"], v=r["v_cache"], ssm=r["h"], conv=r["conv"]))
            H.close_bf16(H.to64(yt[b]), got, "decode")
            state_close(w, H.to64(h[b]), cache["ssm"], "state after the decode step")
        lay.close()
    for a, b, name in zip(*out, ("Y", "K", "state", "decode", "decoded state")):
        H.assert_bits_equal(a, b, name)
