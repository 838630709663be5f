"""Head norm and rotation on the GPU: sides without heads, and the parts of a head that go through
shared memory."""
from __future__ import annotations

import pytest
import torch

import hybrid_attention_ssm_head_b200 as hy
from tests import _operators as P
from tests.test_gpu_m_heads import DT, bound, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("H", [1, 25])
def test_a_side_without_heads_is_not_looked_at(side, dtype, H):
    """25 heads of 64 leave slots of the last load empty.  Whatever the other side's fields hold, they
    change nothing (its pointers are host addresses and odd ones here)."""
    B, R, d = 2, 5, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, R, H, d, generator=g).to(DT[dtype])
    w = 1 + torch.randn(d, generator=g)
    dev, wd, out = x.cuda(), w.cuda(), torch.full((B, R, H, d), 9.0, dtype=DT[dtype], device="cuda")
    args = hy.make_qk_norm_rope(*((dev, None, out, None) if side == "q" else (None, dev, None, out)),
                                rope=hy.make_rope(d, "halves"), pos0=11,
                                **{"q_weight" if side == "q" else "k_weight": wd})
    setattr(args, "k" if side == "q" else "q", hy.hymba_head_rows(8191, 8191, 8191, -3, 7, 5, -3, 7, 5, 0))
    hy.hymba_qk_norm_rope(args, torch.cuda.current_stream())
    hy.hymba_stream_status(torch.cuda.current_stream())
    pos = (11 + torch.arange(R)).expand(B, R)
    want, size = P.heads(x, w, True, 1e-6, pos, d, "halves", 1.0, P.frequencies(d, 10000.0))
    P.within(out, want, bound(DT[dtype], want, size), side)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,rot", [(72, 44), (24, 12), (128, 70), (256, 254), (16, 2)])
def test_halves_of_a_part_of_the_head(dtype, d, rot):
    """Halves that end inside a lane's eight elements."""
    B, R, H, K = 2, 9, 5, 2
    g = torch.Generator().manual_seed(4)
    q, k = (torch.randn(B, R, n, d, generator=g).to(DT[dtype]) for n in (H, K))
    wq, wk = 1 + torch.randn(d, generator=g), 1 + torch.randn(d, generator=g)
    qo, ko = torch.empty_like(q, device="cuda"), torch.empty_like(k, device="cuda")
    run(q.cuda(), k.cuda(), qo, ko, q_weight=wq.cuda(), k_weight=wk.cuda(), rope=hy.make_rope(rot, "halves"), pos0=100)
    pos = (100 + torch.arange(R)).expand(B, R)
    for name, x, w, out in (("q", q, wq, qo), ("k", k, wk, ko)):
        want, size = P.heads(x, w, True, 1e-6, pos, rot, "halves", 1.0, P.frequencies(rot, 10000.0))
        P.within(out, want, bound(DT[dtype], want, size), name)
