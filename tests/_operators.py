"""Plain 64-bit forms of the operators (head norm/rotation, linear attention), with the magnitudes
their error bounds are built from.  Torch on the CPU, float64, one row at a time."""
from __future__ import annotations

import math

import torch

F32_STEP = 2.0 ** -24   # half a step of fp32, relative to the value
BF16_STEP = 2.0 ** -8   # half a step of bf16


def half_step(dtype: torch.dtype) -> float:
    return torch.finfo(dtype).eps / 2


def frequencies(rot, base, scaling="none", factor=1.0, orig_len=0.0, low_turns=0.0, high_turns=0.0):
    out = []
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "wavelength":
            turns = orig_len * f / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low_turns) / (high_turns - low_turns)))
            f = keep * f + (1 - keep) * f / factor
        out.append(f)
    return out


def heads(x, weight, norm, eps, pos, rot, layout, m, freq):
    """x [B, R, H, d], pos [B, R] integers.  Returns (y, size): size bounds |y|'s terms."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if weight is not None:
            y = y * weight.double()
    y = y.clone()
    size = y.abs().clone()
    for i, f in enumerate(freq):
        a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + rot // 2)
        angle = (pos.double() * f)[..., None]
        c, s = torch.cos(angle) * m, torch.sin(angle) * m
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = ya * c - yb * s, ya * s + yb * c
        size[..., a] = size[..., b] = m * (ya.abs() + yb.abs())
    return y, size


def linear(q, k, v, o, log_decay=None, in_scale=None, skip=None, gate=None, state_in=None, lengths=None, scale=1.0):
    """Row by row.  Returns (o, state, o_size, state_size): the sizes are the same sums with every
    term's absolute value, what a sum's rounding errors are relative to."""
    B, L, K, dk = q.shape
    H, dv = v.shape[2:]
    head = torch.arange(H) // (H // K)
    S = torch.zeros(B, H, dv, dk, dtype=torch.float64)
    if state_in is not None:
        S = S + state_in.double()
    A = S.abs()
    out, size = o.double().clone(), torch.zeros(o.shape, dtype=torch.float64)
    for b in range(B):
        n = L if lengths is None else max(0, min(L, int(lengths[b])))
        for t in range(n):
            a = torch.ones(H, dtype=torch.float64) if log_decay is None else log_decay[b, t].double().exp()
            s = torch.ones(H, dtype=torch.float64) if in_scale is None else in_scale[b, t].double()
            kk, qq, vv = k[b, t].double()[head], q[b, t].double()[head], v[b, t].double()
            x = s[:, None, None] * vv[:, :, None] * kk[:, None, :]
            # a decay of zero forgets, whatever was there
            S[b] = torch.where(a[:, None, None] > 0, a[:, None, None] * S[b], 0.0) + x
            A[b] = torch.where(a[:, None, None] > 0, a[:, None, None] * A[b], 0.0) + x.abs()
            y = scale * (S[b] @ qq[:, :, None])[..., 0]
            z = abs(scale) * (A[b] @ qq.abs()[:, :, None])[..., 0]
            if skip is not None:
                y, z = y + skip.double() * vv, z + (skip.double() * vv).abs()
            if gate is not None:
                y, z = y * gate[b, t].double(), z * gate[b, t].double().abs()
            out[b, t], size[b, t] = y, z
    return out, S, size, A


def linear_bounds(dtype, L, dk, want, size, state, state_size, chunked):
    """Elementwise bounds of o and of the state.

    fp32 sums: a row's product, its addition into the state and the decay's multiplication round
    once each, as does the decay itself, so behind L rows a state is within (4 L + 8) half steps of
    its size; the dot product over dk columns adds dk + 8.  bf16 storage rounds o once more
    (half a bf16 step of o).  The chunked form, where one is used, rounds each score to bf16 once
    (half a bf16 step of the size) and multiplies with states split in two bf16 parts, which leaves
    2^-16 of each term, and with keys split in three, which leaves 2^-24."""
    rho = (4 * L + dk + 16) * F32_STEP
    if chunked:
        return (BF16_STEP * want.abs() + (BF16_STEP + 2 * 2.0 ** -16 + rho) * size + 1e-30,
                rho * state_size + 1e-30)
    return half_step(dtype) * want.abs() + rho * size + 1e-30, rho * state_size + 1e-30


def within(got, want, bound, what):
    got, want = got.detach().cpu().double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    err = (got - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; first at {i}: "
                             f"{float(got[tuple(i)])} against {float(want[tuple(i)])}, bound {float(bound[tuple(i)]):.3g}")
