"""The operators' argument checks: every refusal comes before any launch (CPU only)."""
from __future__ import annotations

import ctypes as C

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
from tests import _operators as P

A = 1 << 44  # aligned fake device addresses: never dereferenced


def _heads(**kw):
    row = 30 * 64
    q = hy.hymba_head_rows(A, A, None, 7 * row, row, 64, 7 * row, row, 64, 25)
    k = hy.hymba_head_rows(A + 25 * 128, A + 25 * 128, None, 7 * row, row, 64, 7 * row, row, 64, 5)
    a = hy.hymba_qk_norm_rope_args(dtype=hy.HYMBA_BF16, batch=2, n_rows=7, head_dim=64, q=q, k=k, norm=1, eps=1e-6,
                                   rope=hy.make_rope(64), pos0=0, positions=None)
    for name, v in kw.items():
        obj = a
        *path, last = name.split("__")
        for p in path:
            obj = getattr(obj, p)
        setattr(obj, last, v)
    return a


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), hy.HYMBA_ERR_INVALID_ARG),
    (dict(batch=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(n_rows=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(head_dim=60), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(head_dim=264), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(q__n_heads=0, k__n_heads=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__n_heads=-1), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__in_=None), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__in_=A + 8), hy.HYMBA_ERR_INVALID_ARG),
    (dict(k__out=None), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__in_row=30 * 64 + 4), hy.HYMBA_ERR_INVALID_ARG),    # not 16 bytes
    (dict(q__in_head=0, q__out_head=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__out=A + (1 << 30), q__out_head=32), hy.HYMBA_ERR_INVALID_ARG),  # written heads overlap
    (dict(q__out_row=31 * 64), hy.HYMBA_ERR_INVALID_ARG),       # in place with other strides
    (dict(q__weight=A + 4), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q__weight=A, norm=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(eps=-1.0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(eps=float("nan")), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__dim=63), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__dim=66), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__dim=-2), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__layout=2), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__base=1.0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__base=float("inf")), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__scaling=3), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__scaling=1, rope__factor=0.0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__scaling=2, rope__factor=4.0), hy.HYMBA_ERR_INVALID_ARG),  # no trained length
    (dict(rope__scaling=2, rope__factor=4.0, rope__orig_len=2048.0, rope__low_turns=4.0, rope__high_turns=4.0),
     hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope__attn_factor=0.0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(positions=A + 4), hy.HYMBA_ERR_INVALID_ARG),
])
def test_qk_norm_rope_refuses(kw, status):
    with pytest.raises(hy.HymbaError) as e:
        hy.hymba_qk_norm_rope(_heads(**kw))
    assert e.value.status == status, e.value
    assert hy.hymba_last_error()


def test_null_descriptions_are_refused():
    lib = hy.lib()
    n = C.c_size_t()
    assert lib.hymba_qk_norm_rope(None, None) == hy.HYMBA_ERR_INVALID_ARG
    assert lib.hymba_linear_attention_workspace(None, C.byref(n)) == hy.HYMBA_ERR_INVALID_ARG
    assert lib.hymba_linear_attention_prefill(None, None, 0, None) == hy.HYMBA_ERR_INVALID_ARG
    assert lib.hymba_linear_attention_decode_step(None, None) == hy.HYMBA_ERR_INVALID_ARG
    assert lib.hymba_linear_attention_workspace(C.byref(_linear()), None) == hy.HYMBA_ERR_INVALID_ARG


def _linear(L=9, **kw):
    a = hy.hymba_linear_attention(
        dtype=hy.HYMBA_BF16, batch=2, n_rows=L, n_heads=6, n_qk_heads=2, dk=64, dv=128, scale=1.0,
        q=A, q_batch=L * 128, q_row=128, q_head=64, k=A + (1 << 24), k_batch=L * 128, k_row=128, k_head=64,
        v=A + (2 << 24), v_batch=L * 768, v_row=768, v_head=128, o=A + (3 << 24), o_batch=L * 768, o_row=768, o_head=128,
        log_decay=A + (4 << 24), decay_batch=0, decay_row=0, decay_head=1, state_in=A + (5 << 24),
        state_in_batch=6 * 128 * 64, state_out=A + (6 << 24))
    for n, v in kw.items():
        setattr(a, n, v)
    return a


LINEAR_REFUSALS = [
    (dict(dtype=3), hy.HYMBA_ERR_INVALID_ARG),
    (dict(batch=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(n_rows=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(n_qk_heads=4), hy.HYMBA_ERR_INVALID_ARG),
    (dict(dk=20), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(dk=136), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(dv=264), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(dv=-8), hy.HYMBA_ERR_INVALID_ARG),
    (dict(batch=70000), hy.HYMBA_ERR_UNSUPPORTED),
    (dict(scale=float("inf")), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q=None), hy.HYMBA_ERR_INVALID_ARG),
    (dict(k=A + 2), hy.HYMBA_ERR_INVALID_ARG),
    (dict(v_head=0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(q_head=68), hy.HYMBA_ERR_INVALID_ARG),
    (dict(v_batch=1 << 39), hy.HYMBA_ERR_INVALID_ARG),
    (dict(o=None), hy.HYMBA_ERR_INVALID_ARG),
    (dict(o_head=64), hy.HYMBA_ERR_INVALID_ARG),        # written heads overlap
    (dict(o=A + (2 << 24)), hy.HYMBA_ERR_INVALID_ARG),  # o is v
    (dict(gate=A + 8), hy.HYMBA_ERR_INVALID_ARG),
    (dict(gate=A, gate_head=128, gate_row=768), hy.HYMBA_ERR_INVALID_ARG),  # gate's batch stride 0
    (dict(log_decay=A + 2), hy.HYMBA_ERR_INVALID_ARG),
    (dict(decay_head=-1), hy.HYMBA_ERR_INVALID_ARG),
    (dict(in_scale=A, scale_row=-4), hy.HYMBA_ERR_INVALID_ARG),
    (dict(skip=A + 4), hy.HYMBA_ERR_INVALID_ARG),
    (dict(lengths=A + 2), hy.HYMBA_ERR_INVALID_ARG),
    (dict(state_in=A + 4), hy.HYMBA_ERR_INVALID_ARG),
    (dict(state_in_batch=64), hy.HYMBA_ERR_INVALID_ARG),
    (dict(state_out=A + 8), hy.HYMBA_ERR_INVALID_ARG),
    (dict(state_out=A + (5 << 24) + 4096), hy.HYMBA_ERR_INVALID_ARG),     # overlaps state_in
    (dict(state_out=A + (5 << 24), state_in_batch=0), hy.HYMBA_ERR_INVALID_ARG),  # one state, in place
]


@pytest.mark.parametrize("kw,status", LINEAR_REFUSALS)
def test_linear_attention_refuses(kw, status):
    for L, call in ((9, lambda a: hy.hymba_linear_attention_prefill(a, A, 1 << 40)),
                    (1, lambda a: hy.hymba_linear_attention_decode_step(a))):
        with pytest.raises(hy.HymbaError) as e:
            call(_linear(L, **kw))
        assert e.value.status == status, (kw, e.value)


def test_linear_step_needs_one_row_and_a_state():
    for a in (_linear(2), _linear(1, state_out=None)):
        with pytest.raises(hy.HymbaError) as e:
            hy.hymba_linear_attention_decode_step(a)
        assert e.value.status == hy.HYMBA_ERR_INVALID_ARG


def test_description_helpers_check_what_the_library_cannot_see():
    B, L, H, K, dk, dv = 2, 5, 4, 2, 16, 24
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    good = dict(q=t(B, L, K, dk), k=t(B, L, K, dk), v=t(B, L, H, dv), o=t(B, L, H, dv))
    a = hy.make_linear_attention(**good, log_decay=torch.zeros(H).expand(B, L, H))
    assert (a.decay_batch, a.decay_row, a.decay_head) == (0, 0, 1) and a.v_head == dv and a.scale == 1.0
    for bad in (dict(k=t(B, L, K, dk + 8)), dict(o=torch.zeros(B, L, H, dv)), dict(v=t(B, L, dv, H).transpose(2, 3)),
                dict(log_decay=torch.zeros(B, L, H, dtype=torch.float64)), dict(lengths=torch.zeros(B, dtype=torch.int64)),
                dict(state_out=torch.zeros(B, H, dk, dv)), dict(skip=torch.zeros(H))):
        with pytest.raises(ValueError):
            hy.make_linear_attention(**{**good, **bad})
    r = hy.make_qk_norm_rope(t(B, L, H, dk), t(B, L, K, dk), rope=hy.make_rope(8, "halves"))
    assert r.q.in_ == r.q.out and r.k.n_heads == K and r.rope.layout == hy.HYMBA_ROPE_HALVES
    for bad in (dict(q_out=t(B, L, K, dk)), dict(q_weight=torch.zeros(dk + 1)), dict(positions=torch.zeros(B, L))):
        with pytest.raises(ValueError):
            hy.make_qk_norm_rope(t(B, L, H, dk), t(B, L, K, dk), **bad)


def test_plain_linear_form_equals_the_sum_over_earlier_rows():
    """The tests' recurrence against o_i = sum_j<=i exp(g_j+1 + .. + g_i) s_j (q_i . k_j) v_j."""
    r = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=r, dtype=torch.float64)  # noqa: E731
    L, H, dk, dv = 7, 2, 4, 3
    q, k, v = n(1, L, 1, dk), n(1, L, 1, dk), n(1, L, H, dv)
    g, s = -n(1, L, H).abs(), n(1, L, H).abs()
    o, S, _, _ = P.linear(q, k, v, torch.zeros(1, L, H, dv), g, s, scale=0.5)
    for h in range(H):
        for i in range(L):
            want = sum(torch.exp(g[0, j + 1:i + 1, h].sum()) * s[0, j, h] * (q[0, i, 0] @ k[0, j, 0]) * v[0, j, h]
                       for j in range(i + 1)) * 0.5
            torch.testing.assert_close(o[0, i, h], want, rtol=1e-12, atol=1e-14)
        want = sum(torch.exp(g[0, j + 1:, h].sum()) * s[0, j, h] * torch.outer(v[0, j, h], k[0, j, 0]) for j in range(L))
        torch.testing.assert_close(S[0, h], want, rtol=1e-12, atol=1e-14)


def test_plain_rotation_is_a_complex_product():
    x = torch.randn(1, 3, 2, 8, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    pos = torch.tensor([[0, 5, 70000]])
    f = P.frequencies(6, 100.0)
    for layout in ("pairs", "halves"):
        y, _ = P.heads(x, None, False, 0.0, pos, 6, layout, 1.5, f)
        for i in range(3):
            a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + 3)
            turn = 1.5 * torch.exp(1j * pos.double() * f[i])[..., None]
            z = torch.complex(x[..., a], x[..., b]) * turn
            torch.testing.assert_close(torch.complex(y[..., a], y[..., b]), z, rtol=1e-12, atol=1e-12)
        torch.testing.assert_close(y[..., 6:], x[..., 6:], rtol=0, atol=0)


def _layer(**kw):
    base = dict(d_model=256, n_heads=4, n_kv_heads=2, head_dim_qk=64, d_inner=512, d_state=16, d_conv=4, dt_rank=16,
                n_meta=16, window=64, is_global=False, dtype="bf16")
    base.update(kw)
    return hy.hymba_layer_create(hy.make_config(**base), hy.hymba_layer_weights(*[A + 4096 * i for i in range(11)]))


@pytest.mark.parametrize("heads,cfg,status", [
    (dict(rope=hy.make_rope(66)), {}, hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope=hy.make_rope(64, base=0.5)), {}, hy.HYMBA_ERR_INVALID_ARG),
    (dict(rope=hy.make_rope(64)), dict(rope_base=10000.0), hy.HYMBA_ERR_INVALID_ARG),
    (dict(eps=-1.0), {}, hy.HYMBA_ERR_INVALID_ARG),
    (dict(norm=False, q_weight=A), {}, hy.HYMBA_ERR_INVALID_ARG),
    (dict(k_weight=A + 4), {}, hy.HYMBA_ERR_INVALID_ARG),
    ({}, dict(dtype="f32", head_dim_qk=20), hy.HYMBA_ERR_UNSUPPORTED),
])
def test_layer_heads_refuse(heads, cfg, status):
    h = _layer(**cfg)
    with pytest.raises(hy.HymbaError) as e:
        hy.hymba_layer_set_heads(h, hy.make_layer_heads(**heads))
    assert e.value.status == status
    hy.hymba_layer_set_heads(h, None)
    hy.hymba_layer_destroy(h)
    with pytest.raises(hy.HymbaError):
        hy.hymba_layer_set_heads(None, None)


@pytest.mark.parametrize("d_state,missing,status", [
    (0, None, hy.HYMBA_ERR_UNSUPPORTED), (20, None, hy.HYMBA_ERR_UNSUPPORTED), (136, None, hy.HYMBA_ERR_UNSUPPORTED),
    (64, "b_dt", hy.HYMBA_ERR_INVALID_ARG), (64, "w_x", hy.HYMBA_ERR_INVALID_ARG)])
def test_linear_heads_refuse(d_state, missing, status):
    h = _layer()
    before = hy.hymba_layer_prefill_workspace(h, 2, 100), hy.hymba_layer_decode_workspace(h, 2, 100)
    w = {n: A + 4096 * i for i, n in enumerate(("w_x", "b_dt", "a_log", "d_skip"))}
    if missing:
        w[missing] = None
    with pytest.raises(hy.HymbaError) as e:
        hy.hymba_layer_set_linear_heads(h, hy.make_linear_heads(w, d_state))
    assert e.value.status == status
    assert before == (hy.hymba_layer_prefill_workspace(h, 2, 100), hy.hymba_layer_decode_workspace(h, 2, 100))
    good = {n: A + 4096 * i for i, n in enumerate(("w_x", "b_dt", "a_log", "d_skip"))}
    hy.hymba_layer_set_linear_heads(h, hy.make_linear_heads(good, 128))
    assert hy.hymba_layer_decode_workspace(h, 2, 100) > before[1]
    hy.hymba_layer_set_linear_heads(h, None)
    assert before == (hy.hymba_layer_prefill_workspace(h, 2, 100), hy.hymba_layer_decode_workspace(h, 2, 100))
    hy.hymba_layer_destroy(h)


def test_oracle_heads_and_linear_heads_against_the_plain_forms():
    """The layer oracle's versions of both operators agree with the ones written for the operators'
    tests, and its rotation with the configuration's own where they overlap."""
    import numpy as np
    from oracle import hymba_oracle as O
    from tests import _small as T
    r = np.random.default_rng(2)
    x, pos = r.normal(size=(5, 3 * 8)), np.array([0, 1, 7, 300, 8191])
    np.testing.assert_allclose(O.heads_norm_rope(x, pos, 8, dict(rope_dim=8, base=100.0, layout="pairs"), None),
                               O.rope(x, pos, 8, 100.0), rtol=1e-12, atol=1e-12)
    wl = dict(scaling="wavelength", factor=4.0, orig_len=512.0, low_turns=1.0, high_turns=4.0)
    w = r.normal(size=8)
    got = O.heads_norm_rope(x, pos, 8, dict(norm=True, eps=1e-5, rope_dim=6, base=50.0, layout="halves", attn_factor=1.2, **wl), w)
    want, _ = P.heads(torch.tensor(x).view(1, 5, 3, 8), torch.tensor(w), True, 1e-5, torch.tensor(pos)[None], 6, "halves",
                      1.2, P.frequencies(6, 50.0, **wl))
    np.testing.assert_allclose(got, want.view(5, 24).numpy(), rtol=1e-11, atol=1e-12)
    s = T.spec()
    E, nh, n, L = s.d_inner, s.n_heads, 6, 9
    u = r.normal(size=(L, E))
    lw = dict(w_x=r.normal(size=(2 * n + nh, E)) / 4, b_dt=r.normal(size=nh), a_log=r.normal(size=nh), d_skip=r.normal(size=E))
    spread, Bm, Cm, A_, D = O._ssm_terms(u, dict(linear=lw), s)
    y, h = O.selective_scan(u, spread, A_, Bm, Cm, D)
    proj = torch.tensor(u @ lw["w_x"].T)
    delta = torch.nn.functional.softplus(proj[:, 2 * n:] + torch.tensor(lw["b_dt"]))
    t = lambda a: a[None, :, None]  # noqa: E731
    o, S, _, _ = P.linear(t(proj[:, n:2 * n]), t(proj[:, :n]), torch.tensor(u).view(1, L, nh, E // nh),
                          torch.zeros(1, L, nh, E // nh), (-torch.tensor(lw["a_log"]).exp() * delta)[None], delta[None],
                          skip=torch.tensor(lw["d_skip"]).view(nh, -1))
    np.testing.assert_allclose(y, o.view(L, E).numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(h, S.view(E, n).numpy(), rtol=1e-10, atol=1e-12)
