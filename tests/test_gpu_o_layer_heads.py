"""The layer with its head operators on: per-head norm and rotation of Q and K, linear heads in the
SSM branch, and both, through prefill, meta cache, K/V sharing, blocks and decode, against the fp64
oracle on the same inputs."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
import synth
from oracle import hymba_oracle as O
from synth.configs import STRESS_STD, LayerDims, Workload
from tests import _harness as H

pytestmark = pytest.mark.gpu

DIMS = LayerDims(d_model=256, n_heads=4, n_kv_heads=2, head_dim_qk=64, d_inner=512)
ROPES = {"pairs": dict(layout="pairs", rope_dim=64, base=10000.0),
         "halves": dict(layout="halves", rope_dim=48, base=500.0, scaling="wavelength", factor=4.0, orig_len=64.0,
                        low_turns=1.0, high_turns=8.0, attn_factor=1.1)}


def set_heads(lay, rope="pairs", weights=True, seed=5):
    d = lay.workload.dims
    w = {n: 1 + 0.3 * synth.gen.normal_tensor((d.head_dim_qk,), seed, f"heads/{n}") for n in ("q_weight", "k_weight")}
    lay.dev.update({f"heads_{n}": t.cuda() for n, t in w.items()})
    r = ROPES[rope]
    hy.hymba_layer_set_heads(lay.handle, hy.make_layer_heads(
        True, 1e-6, lay.dev["heads_q_weight"] if weights else None, lay.dev["heads_k_weight"] if weights else None,
        hy.make_rope(r["rope_dim"], r["layout"], **{k: v for k, v in r.items() if k not in ("rope_dim", "layout")})))
    return dict(norm=True, eps=1e-6, **({n: H.to64(t) for n, t in w.items()} if weights else {}), **r)


def set_linear(lay, d_state, seed=6):
    d, dt = lay.workload.dims, H.torch_dt(lay.workload)
    E, nh = d.d_inner, d.n_heads
    g = synth.gen.normal_tensor
    w = dict(w_x=torch.cat([g((2 * d_state, E), seed, "lin/bc", E ** -0.5), g((nh, E), seed, "lin/d", E ** -0.5)]).to(dt),
             b_dt=g((nh,), seed, "lin/b", 0.5, -2.0), a_log=synth.gen.uniform_tensor((nh,), seed, "lin/a", -1.0, 2.0),
             d_skip=g((E,), seed, "lin/skip"))
    lay.dev.update({f"lin_{n}": t.cuda().contiguous() for n, t in w.items()})
    hy.hymba_layer_set_linear_heads(lay.handle, hy.make_linear_heads(
        {n: lay.dev[f"lin_{n}"] for n in w}, d_state))
    return {n: H.to64(t) for n, t in w.items()}


def state_close(w, g, o, what):
    """bf16 storage: B, C, u and the projection are rounded once each (four half steps of 2^-8 along
    a term at most); fp32: the layer's own 1e-4."""
    H.close_rel_l2(g, o, 4 * 2.0 ** -8 if w.dtype == "bf16" else 1e-4, what)


@pytest.mark.parametrize("dtype,glob,rope,d_state,chunks", [
    ("bf16", False, "pairs", None, 4), ("bf16", False, None, 64, 4), ("bf16", True, "halves", 128, 4),
    ("bf16", False, "halves", 24, 0), ("f32", False, "halves", 64, 4), ("f32", True, None, 16, 0)])
def test_prefill_consumer_and_decode(dtype, glob, rope, d_state, chunks):
    dims = DIMS if dtype == "bf16" else synth.configs.DIMS_SMALL
    w = Workload(f"lh_{dtype}_{glob}_{rope}_{d_state}", dims, dtype, 3, 16, 200, 0 if glob else 64)
    prod = H.GpuLayer(w, 0, is_global=glob, std=STRESS_STD, branch_chunks=chunks)
    cons = H.GpuLayer(w, 1, consumer=True, is_global=glob, std=STRESS_STD, branch_chunks=chunks)
    hy.hymba_kv_share_bind(cons.handle, prod.handle)
    wp, wc = H.oracle_weights(prod.cpu), H.oracle_weights(cons.cpu)
    for lay, ow in ((prod, wp), (cons, wc)):
        if rope:
            ow["heads"] = set_heads(lay, rope)
        if d_state:
            ow["linear"] = set_linear(lay, d_state, seed=6 + lay.consumer)
    N = d_state or dims.d_state
    B, L, steps = w.batch, w.seq_rows, 3
    cap = L + steps if glob else w.n_meta + w.window
    x = synth.configs.x_tilde(w).cuda()
    x2 = synth.gen.normal_tensor(tuple(x.shape), 0, f"{w.name}/x2", device="cuda").to(H.torch_dt(w))
    k, v, kv = H.alloc_kv_seq(w, B, L)
    kc, vc, kvc = H.alloc_kv_cache(w, B, cap)
    hs = [torch.zeros(B, dims.d_inner, N, device="cuda") for _ in range(2)]
    cs = [torch.zeros(B, dims.d_conv - 1, dims.d_inner, dtype=H.torch_dt(w), device="cuda") for _ in range(2)]
    ssm = [hy.hymba_ssm_cache(h.data_ptr(), c.data_ptr()) for h, c in zip(hs, cs)]
    y1, ws = H.run_prefill(prod, x, kv, kvc, ssm[0])
    y2, ws = H.run_prefill(cons, x2, kv, None, ssm[1], ws=ws)
    refs = []
    for b in range(B):
        r1 = O.layer_prefill(H.to64(x[b]), wp, prod.spec, capacity=cap)
        r2 = O.layer_prefill(H.to64(x2[b]), wc, cons.spec, kv_from=r1)
        H.close(w, H.to64(y1[b]), r1["Y"], f"producer Y b={b}")
        H.close(w, H.to64(k[b]), r1["k"], f"K b={b}")
        H.close(w, H.to64(y2[b]), r2["Y"], f"consumer Y b={b}")
        state_close(w, H.to64(hs[0][b]), r1["h"], f"state b={b}")
        refs.append((dict(k=r1["k_cache"], v=r1["v_cache"], ssm=r1["h"], conv=r1["conv"]),
                     dict(ssm=r2["h"], conv=r2["conv"])))
    dws = H.workspace(max(hy.hymba_layer_decode_workspace(lay.handle, B, L + steps) for lay in (prod, cons)))
    s = torch.cuda.current_stream()
    for i in range(steps):
        xn = [synth.gen.normal_tensor((B, dims.d_model), 0, f"{w.name}/xn{i}{j}", device="cuda").to(H.torch_dt(w)) for j in (0, 1)]
        yt = [torch.empty_like(t) for t in xn]
        for lay, j in ((prod, 0), (cons, 1)):
            hy.hymba_layer_decode_step(lay.handle, B, L + i, xn[j], yt[j], kvc, ssm[j], dws, dws.numel(), s)
        hy.hymba_stream_status(s)
        for b in range(B):
            o1, c1 = O.layer_decode(H.to64(xn[0][b]), L + i, wp, prod.spec, refs[b][0])
            o2, c2 = O.layer_decode(H.to64(xn[1][b]), L + i, wc, cons.spec, refs[b][1], kv_cache=c1)
            H.close(w, H.to64(yt[0][b]), o1, f"decode {i} b={b}")
            H.close(w, H.to64(yt[1][b]), o2, f"consumer's decode {i} b={b}")
            state_close(w, H.to64(hs[0][b]), c1["ssm"], f"state after decode {i} b={b}")
            refs[b] = (c1, c2)
    prod.close()
    cons.close()


def test_operators_are_really_applied_and_can_be_taken_off():
    w = Workload("lh_off", DIMS, "bf16", 2, 16, 100, 64)
    lay = H.GpuLayer(w, 0, std=STRESS_STD)
    x = synth.configs.x_tilde(w).cuda()

    def run():
        k, v, kv = H.alloc_kv_seq(w, w.batch, w.seq_rows)
        return H.run_prefill(lay, x, kv)[0]

    plain = run()
    set_heads(lay)
    headed = run()
    set_linear(lay, 64)
    both = run()
    assert float((headed - plain).abs().max()) > 0.05 and float((both - headed).abs().max()) > 0.05
    hy.hymba_layer_set_heads(lay.handle, None)
    hy.hymba_layer_set_linear_heads(lay.handle, None)
    H.assert_bits_equal(run(), plain, "as before")
    lay.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_side_by_side_branches_give_the_serial_bits(dtype):
    """The batch chunks of the concurrent prefill and the side-stream decode step, bit for bit."""
    dims = DIMS if dtype == "bf16" else synth.configs.DIMS_SMALL
    w = Workload(f"lh_bits_{dtype}", dims, dtype, 5, 16, 1300, 64)
    out = []
    for chunks in (0, 3):
        lay = H.GpuLayer(w, 0, std=STRESS_STD, branch_chunks=chunks)
        set_heads(lay, "halves")
        set_linear(lay, 32)
        x = synth.configs.x_tilde(w).cuda()
        k, v, kv = H.alloc_kv_seq(w, w.batch, w.seq_rows)
        kc, vc, kvc = H.alloc_kv_cache(w, w.batch, w.n_meta + w.window)
        h = torch.zeros(w.batch, dims.d_inner, 32, device="cuda")
        c = torch.zeros(w.batch, dims.d_conv - 1, dims.d_inner, dtype=H.torch_dt(w), device="cuda")
        ssm = hy.hymba_ssm_cache(h.data_ptr(), c.data_ptr())
        y, _ = H.run_prefill(lay, x, kv, kvc, ssm)
        h1 = h.clone()
        xt = x[:, -1].contiguous()
        yt = torch.empty_like(xt)
        dws = H.workspace(hy.hymba_layer_decode_workspace(lay.handle, w.batch, w.seq_rows))
        s = torch.cuda.current_stream()
        hy.hymba_layer_decode_step(lay.handle, w.batch, w.seq_rows, xt, yt, kvc, ssm, dws, dws.numel(), s)
        hy.hymba_stream_status(s)
        out.append((y, k, h1, yt, h))
        lay.close()
    for a, b, name in zip(*out, ("Y", "K", "state", "decode", "decoded state")):
        H.assert_bits_equal(a, b, name)


def test_meta_cache_starts_linear_heads_and_rotated_keys():
    w = Workload("lh_meta", DIMS, "bf16", 2, 128, 200, 128)
    lay = H.GpuLayer(w, 0, std=STRESS_STD)
    ow = H.oracle_weights(lay.cpu)
    ow["heads"], ow["linear"] = set_heads(lay, "halves"), set_linear(lay, 64)
    B, L, m, d = w.batch, w.seq_rows, w.n_meta, w.dims
    xt = synth.configs.x_tilde(w).cuda()
    bufs = dict(k=torch.zeros(m, d.n_kv_heads * 64, dtype=torch.bfloat16, device="cuda"),
                v=torch.zeros(m, d.n_kv_heads * 128, dtype=torch.bfloat16, device="cuda"),
                h=torch.zeros(d.d_inner, 64, device="cuda"),
                conv=torch.zeros(3, d.d_inner, dtype=torch.bfloat16, device="cuda"),
                y=torch.zeros(m, d.d_model, dtype=torch.bfloat16, device="cuda"))
    mc = hy.hymba_meta_cache(*[bufs[n].data_ptr() for n in ("k", "v", "h", "conv", "y")], 0)
    mws = H.workspace(hy.hymba_layer_meta_workspace(lay.handle))
    s = torch.cuda.current_stream()
    hy.hymba_layer_meta_precompute(lay.handle, xt[0, :m].contiguous(), mc, None, mws, mws.numel(), s)
    k, v, kv = H.alloc_kv_seq(w, B, L)
    h = torch.zeros(B, d.d_inner, 64, device="cuda")
    c = torch.zeros(B, 3, d.d_inner, dtype=torch.bfloat16, device="cuda")
    ssm = hy.hymba_ssm_cache(h.data_ptr(), c.data_ptr())
    xr = xt[:, m:].contiguous()
    y = torch.empty_like(xr)
    ws = H.workspace(hy.hymba_layer_prefill_cached_workspace(lay.handle, B, w.n_tokens))
    hy.hymba_layer_prefill_cached(lay.handle, B, w.n_tokens, xr, y, mc, kv, None, ssm, ws, ws.numel(), s)
    hy.hymba_stream_status(s)
    for b in range(B):
        r = O.layer_prefill(H.to64(xt[b]), ow, lay.spec)
        H.close_bf16(H.to64(y[b]), r["Y"][m:], f"cached prefill b={b}")
        H.close_bf16(H.to64(k[b]), r["k"], f"K b={b}")
        state_close(w, H.to64(h[b]), r["h"], f"state b={b}")
    lay.close()


def test_captured_decode_steps_replay():
    """Two decode steps with both operators captured as one graph, replayed from the same state, equal
    the eager steps bit for bit."""
    w = Workload("lh_graph", DIMS, "bf16", 3, 16, 60, 64)
    lay = H.GpuLayer(w, 0, std=STRESS_STD)
    set_heads(lay)
    set_linear(lay, 64)
    B, L, d = w.batch, w.seq_rows, w.dims
    x = synth.configs.x_tilde(w).cuda()
    k, v, kv = H.alloc_kv_seq(w, B, L)
    kc, vc, kvc = H.alloc_kv_cache(w, B, w.n_meta + w.window)
    h = torch.zeros(B, d.d_inner, 64, device="cuda")
    c = torch.zeros(B, 3, d.d_inner, dtype=torch.bfloat16, device="cuda")
    ssm = hy.hymba_ssm_cache(h.data_ptr(), c.data_ptr())
    H.run_prefill(lay, x, kv, kvc, ssm)
    saved = [t.clone() for t in (kc, vc, h, c)]
    xt = [x[:, -1 - i].contiguous() for i in range(2)]
    yt = [torch.empty_like(t) for t in xt]
    dws = H.workspace(hy.hymba_layer_decode_workspace(lay.handle, B, L + 2))

    def steps():
        for i in range(2):
            hy.hymba_layer_decode_step(lay.handle, B, L + i, xt[i], yt[i], kvc, ssm, dws, dws.numel(),
                                       torch.cuda.current_stream())

    steps()
    torch.cuda.synchronize()
    want = [t.clone() for t in (*yt, kc, vc, h, c)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        steps()
    for _ in range(2):
        for t, o in zip((kc, vc, h, c), saved):
            t.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        for t, o in zip((*yt, kc, vc, h, c), want):
            H.assert_bits_equal(t, o, "replay")
    hy.hymba_stream_status(torch.cuda.current_stream())
    lay.close()


def test_block_with_both_operators():
    w = Workload("lh_block", DIMS, "bf16", 2, 16, 90, 64)
    lay = H.GpuLayer(w, 0, std=STRESS_STD)
    ow = H.oracle_weights(lay.cpu)
    ow["heads"], ow["linear"] = set_heads(lay), set_linear(lay, 16)
    d, F = w.dims, 192
    bw = synth.configs.block_weights(w, 0, F)
    dev = {n: t.cuda().contiguous() for n, t in bw.items()}
    ow.update({n: H.to64(t) for n, t in bw.items()})
    gu = ow["w_gate_up"]
    ow["w_gate"], ow["w_up"] = gu[0::2], gu[1::2]
    x = synth.configs.x_tilde(w).cuda()
    y = torch.empty_like(x)
    k, v, kv = H.alloc_kv_seq(w, w.batch, w.seq_rows)
    ws = H.workspace(hy.hymba_block_prefill_workspace(lay.handle, F, w.batch, w.n_tokens))
    s = torch.cuda.current_stream()
    hy.hymba_block_prefill(lay.handle, hy.make_block_weights(dev), w.batch, w.n_tokens, x, y, kv, None, None, ws,
                           ws.numel(), s)
    hy.hymba_stream_status(s)
    for b in range(w.batch):
        out, _ = O.block_prefill(H.to64(x[b]), ow, lay.spec)
        H.close_bf16(H.to64(y[b]), out, f"block b={b}")
    lay.close()


def test_consumer_must_rotate_as_its_producer():
    w = Workload("lh_rot", DIMS, "bf16", 1, 16, 40, 64)
    prod, cons = H.GpuLayer(w, 0), H.GpuLayer(w, 1, consumer=True)
    hy.hymba_kv_share_bind(cons.handle, prod.handle)
    set_heads(prod, "pairs")
    x = synth.configs.x_tilde(w).cuda()
    k, v, kv = H.alloc_kv_seq(w, 1, w.seq_rows)
    H.run_prefill(prod, x, kv)
    for other in (None, "halves"):
        if other:
            set_heads(cons, other)
        with pytest.raises(hy.HymbaError) as e:
            H.run_prefill(cons, x, kv)
        assert e.value.status == hy.HYMBA_ERR_NOT_BOUND
    set_heads(cons, "pairs", weights=False)
    y, _ = H.run_prefill(cons, x, kv)
    assert bool(torch.isfinite(y).all())
    prod.close()
    cons.close()
