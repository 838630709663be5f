"""What the layer's head operators and the operators' descriptions check before any launch (CPU only)."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
from tests.test_operators_host import A, _layer


def _status(call, *args) -> int:
    try:
        call(*args)
    except hy.HymbaError as e:
        return e.status
    return hy.HYMBA_OK


def _consumer_status(cons, owner: int) -> int:
    """A consumer's prefill on K/V stamped `owner`.  It passes a decode store too, so that an accepted
    stamp is refused as INVALID_ARG, before any launch."""
    kv = hy.hymba_kv_seq(A, A, 1, 116, owner)
    store = hy.hymba_kv_cache(A, A, 1, 200, 0)
    return _status(hy.hymba_layer_prefill, cons, 1, 100, A, A, kv, store, None, A, 1 << 40)


def _stamp(status, *args) -> int:
    """The only stamp that is not refused as another handle's."""
    hits = [i for i in range(1, 4000) if status(*args, i) != hy.HYMBA_ERR_NOT_BOUND]
    assert len(hits) == 1, hits
    return hits[0]


def test_a_consumer_outlives_its_producer():
    """The K/V are the caller's: a consumer goes on accepting what its producer stamped when that handle
    is gone, whatever has taken its memory."""
    prod, cons = _layer(), _layer()
    hy.hymba_kv_share_bind(cons, prod)
    stamp = _stamp(_consumer_status, cons)
    hy.hymba_layer_destroy(prod)
    others = [_layer() for _ in range(16)]
    for h in others:
        hy.hymba_layer_set_heads(h, hy.make_layer_heads(rope=hy.make_rope(64, "halves")))
    assert hy.hymba_layer_is_consumer(cons)
    assert _consumer_status(cons, stamp) == hy.HYMBA_ERR_INVALID_ARG
    assert _stamp(_consumer_status, cons) == stamp
    for h in (cons, *others):
        hy.hymba_layer_destroy(h)


def _meta_status(layer, owner: int) -> int:
    """A prefill from a meta cache stamped `owner`, with a workspace that an accepted stamp finds too small."""
    meta = hy.hymba_meta_cache(A, A, A, A, A, owner)
    kv = hy.hymba_kv_seq(A, A, 0, 0, 0)
    return _status(hy.hymba_layer_prefill_cached, layer, 1, 100, A, A, meta, kv, None, None, A, 256)


def _store_status(layer, owner: int) -> int:
    """A decode step on a store stamped `owner`, likewise."""
    store = hy.hymba_kv_cache(A, A, 1, 200, owner)
    return _status(hy.hymba_layer_decode_step, layer, 1, 150, A, A, store, hy.hymba_ssm_cache(A, A), A, 256)


LINEAR = {n: A + 4096 * i for i, n in enumerate(("w_x", "b_dt", "a_log", "d_skip"))}
SETTERS = {
    "heads": (hy.hymba_layer_set_heads, lambda: hy.make_layer_heads(), lambda: hy.make_layer_heads(rope=hy.make_rope(64))),
    "linear": (hy.hymba_layer_set_linear_heads, lambda: hy.make_linear_heads(LINEAR, 16),
               lambda: hy.make_linear_heads(LINEAR, 128)),
}


@pytest.mark.parametrize("which", SETTERS)
def test_data_of_another_head_setting_is_refused(which):
    """A meta cache, K/V and decode store written before a head operator was set, changed or taken off hold
    other keys, or a state of another size: NOT_BOUND.  Setting the same again keeps them, and the
    plain heads accept what plain heads wrote."""
    put, one, two = SETTERS[which]
    lay, cons = _layer(), _layer()
    hy.hymba_kv_share_bind(cons, lay)
    uses = ((_meta_status, lay), (_store_status, lay), (_consumer_status, cons))

    def stamps():
        return {_stamp(f, h) for f, h in uses}

    plain = stamps()
    assert len(plain) == 1
    put(lay, one())
    first = stamps()
    assert len(first) == 1 and first != plain
    put(lay, one())
    assert stamps() == first
    put(lay, two())
    second = stamps()
    assert len(second) == 1 and second != first and second != plain
    put(lay, one())
    assert not stamps() & (first | second | plain)
    with pytest.raises(hy.HymbaError):  # a refused setting changes nothing
        now = stamps()
        put(lay, hy.make_layer_heads(eps=-1.0) if which == "heads" else hy.make_linear_heads(LINEAR, 12))
    assert stamps() == now
    put(lay, None)
    assert stamps() == plain
    # the consumer's own setting concerns its own meta cache, not its producer's K/V
    put(cons, two())
    assert _stamp(_consumer_status, cons) in plain and _stamp(_meta_status, cons) not in plain
    for h in (lay, cons):
        hy.hymba_layer_destroy(h)


def _linear_tensors(B=2, L=3, nh=2, dk=8, dv=8):
    t = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    return dict(q=t(B, L, 1, dk), k=t(B, L, 1, dk), v=t(B, L, nh, dv), o=t(B, L, nh, dv))


def test_host_tensors_are_not_launched_on():
    """A kernel that got a host address would fault."""
    x = _linear_tensors()
    one = {n: v[:, :1] for n, v in x.items()}
    state = torch.zeros(2, 2, 8, 8)
    calls = ((hy.hymba_linear_attention_prefill, hy.make_linear_attention(**x), A, 1 << 30),
             (hy.hymba_linear_attention_decode_step, hy.make_linear_attention(**one, state_out=state)),
             (hy.hymba_qk_norm_rope, hy.make_qk_norm_rope(x["q"], x["k"])))
    for call, *args in calls:
        with pytest.raises(ValueError, match="not on a GPU"):
            call(*args)


def test_tensors_of_one_description_are_on_one_device():
    x = _linear_tensors()
    other = dict(lengths=torch.zeros(2, dtype=torch.int32, device="meta"), skip=torch.zeros(2, 8, device="meta"),
                 state_in=torch.zeros(2, 2, 8, 8, device="meta"), log_decay=torch.zeros(2, 3, 2, device="meta"),
                 v=x["v"].to("meta"), gate=x["v"].to("meta"))
    for n, t in other.items():
        with pytest.raises(ValueError, match="different devices"):
            hy.make_linear_attention(**{**x, n: t})
    for kw in (dict(q_weight=torch.zeros(8, device="meta")), dict(k_out=x["k"].to("meta")),
               dict(positions=torch.zeros(2, 3, dtype=torch.int64, device="meta"))):
        with pytest.raises(ValueError, match="different devices"):
            hy.make_qk_norm_rope(x["q"], x["k"], **kw)


def test_head_weights_are_checked_for_what_the_library_cannot_see():
    nh, E, n = 4, 32, 8
    good = dict(w_x=torch.zeros(2 * n + nh, E, dtype=torch.bfloat16), b_dt=torch.zeros(nh), a_log=torch.zeros(nh),
                d_skip=torch.zeros(E))
    lh = hy.make_linear_heads(good, n)
    assert lh.w_x == good["w_x"].data_ptr() and lh.d_state == n
    for bad in (dict(w_x=torch.zeros(E, 2 * n + nh).t()), dict(w_x=torch.zeros(2 * n, E)), dict(w_x=torch.zeros(E)),
                dict(b_dt=torch.zeros(nh, dtype=torch.bfloat16)), dict(a_log=torch.zeros(nh + 1)),
                dict(a_log=torch.zeros(2 * nh)[::2]), dict(d_skip=torch.zeros(E, dtype=torch.bfloat16)),
                dict(d_skip=torch.zeros(nh))):
        with pytest.raises(ValueError):
            hy.make_linear_heads({**good, **bad}, n)
    w = torch.zeros(64)
    assert hy.make_layer_heads(q_weight=w, k_weight=A).q_weight == w.data_ptr()
    for bad in (w.bfloat16(), torch.zeros(128)[::2]):
        with pytest.raises(ValueError):
            hy.make_layer_heads(k_weight=bad)
