"""Handles and stored data of the layer's head operators, checked before any launch (CPU only)."""
from __future__ import annotations

import pytest

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
