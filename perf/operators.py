"""What is measured of the attention heads' and the linear heads' operators, with their plain forms.

Three operators of the hybrid layer's two branches:

* `heads`: the norm of every query and key head and the rotation to its position, in one pass
  (hymba_qk_norm_rope).
* `prompt`: linear attention with a decay for each head over whole sequences
  (hymba_linear_attention_prefill).
* `step`: the same recurrence for one token per sequence, on the stored state
  (hymba_linear_attention_decode_step).

Definitions, per sequence and head h (query/key head h // (n_heads / n_qk_heads)):

    S_t = exp(g_t) S_{t-1} + s_t v_t k_t^T             S: [dv, dk], fp32
    o_t = (scale S_t q_t + skip * v_t) * gate_t

with g the log decay, s the input scale, and skip, gate, s optional.  Rows from a sequence's
length on do not change the state, and their o is left as it was.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of a few sequences: the call's latency
        dict(name="heads 3 tokens", op="heads", dtype="bf16", batch=3, rows=1, heads=25, kv_heads=5, dim=64,
             norm=True, rot=64, layout="pairs", scaling="none", pos0=8319, given=False),
        # one decode step of the 128-sequence batch of the 1.5B widths
        dict(name="heads decode 128", op="heads", dtype="bf16", batch=128, rows=1, heads=25, kv_heads=5, dim=64,
             norm=True, rot=64, layout="halves", scaling="none", pos0=8320, given=False),
        # a prompt batch of 4096 tokens behind 128 meta rows, positions stretched by wavelength
        dict(name="heads prompt", op="heads", dtype="bf16", batch=8, rows=4224, heads=25, kv_heads=5, dim=64,
             norm=True, rot=64, layout="halves", scaling="wavelength", pos0=0, given=False),
        # fp32 storage, part of a wide head rotated, every row at a position of its own
        dict(name="heads part f32", op="heads", dtype="f32", batch=2, rows=1021, heads=6, kv_heads=3, dim=128,
             norm=False, rot=40, layout="pairs", scaling="linear", pos0=0, given=True),
        # the linear heads of one layer over the same prompt batch, with gate, skip and input scale
        dict(name="prompt 8 x 4224", op="prompt", dtype="bf16", batch=8, rows=4224, heads=25, qk_heads=1, dk=64,
             dv=128, decay="token", epilogue=True, start=False, ragged=False),
        # one long sequence continued from a stored state: few heads, the time axis has to be split
        dict(name="prompt 1 x 8320 wide", op="prompt", dtype="bf16", batch=1, rows=8320, heads=25, qk_heads=5, dk=128,
             dv=128, decay="head", epilogue=False, start=True, ragged=False),
        # sequences of unequal lengths in one padded batch, small heads
        dict(name="prompt ragged", op="prompt", dtype="bf16", batch=7, rows=517, heads=4, qk_heads=2, dk=16,
             dv=64, decay="token", epilogue=False, start=True, ragged=True),
        # fp32 storage
        dict(name="prompt f32", op="prompt", dtype="f32", batch=2, rows=1031, heads=4, qk_heads=1, dk=64,
             dv=128, decay="token", epilogue=True, start=False, ragged=False),
        # a prefill batch of the headline length
        dict(name="prompt 16 x 8320", op="prompt", dtype="bf16", batch=16, rows=8320, heads=25, qk_heads=1, dk=64,
             dv=128, decay="token", epilogue=True, start=False, ragged=False),
        # one new token of one sequence: latency
        dict(name="step 1", op="step", dtype="bf16", batch=1, heads=25, qk_heads=1, dk=64, dv=128,
             decay="token", epilogue=True, ragged=False),
        # one decode step of 128 sequences: the state is read and written once
        dict(name="step 128", op="step", dtype="bf16", batch=128, heads=25, qk_heads=1, dk=64, dv=128,
             decay="token", epilogue=True, ragged=False),
        # fp32 storage, a batch with idle rows, odd head sizes
        dict(name="step f32 odd", op="step", dtype="f32", batch=13, heads=4, qk_heads=2, dk=24, dv=40,
             decay="head", epilogue=False, ragged=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, round(math.exp(rng.uniform(math.log(low), math.log(high))))))


def draw(rng):
    op = rng.choice(["heads", "prompt", "prompt", "step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    group = rng.choice([1, 2, 3, 5, 8])
    shared = rng.randint(1, 5)
    if op == "heads":
        dim = 8 * _log(rng, 2, 32)
        rows = _log(rng, 1, 4224)
        width = (shared * group + shared) * dim
        batch = _log(rng, 1, max(1, min(256, (64 << 20) // (rows * width))))
        return dict(op=op, dtype=dtype, batch=batch, rows=rows, heads=shared * group, kv_heads=shared, dim=dim,
                    norm=rng.random() < 0.7, rot=2 * rng.randint(1, dim // 2), layout=rng.choice(["pairs", "halves"]),
                    scaling=rng.choice(["none", "linear", "wavelength"]), pos0=_log(rng, 1, 1 << 20),
                    given=rng.random() < 0.3)
    dk, dv = 8 * rng.randint(1, 16), 8 * rng.randint(1, 16)
    case = dict(op=op, dtype=dtype, heads=shared * group, qk_heads=shared, dk=dk, dv=dv,
                decay=rng.choice(["token", "head"]), epilogue=rng.random() < 0.5, ragged=rng.random() < 0.4)
    per = shared * group * max(dk, 32) * max(dv, 32)
    if op == "step":
        return dict(case, batch=_log(rng, 1, max(1, min(256, (32 << 20) // per))))
    rows = _log(rng, 1, 8320)
    case["batch"] = _log(rng, 1, max(1, min(64, (3 << 30) // (per * rows))))
    return dict(case, rows=rows, start=rng.random() < 0.5)


# ---------------------------------------------------------------------------------------- inputs

ROPE = {  # base, scaling and its numbers: none; positions divided by 4; long wavelengths divided by 4
    "none": dict(base=10000.0),
    "linear": dict(base=10000.0, factor=4.0),
    "wavelength": dict(base=500000.0, factor=4.0, orig_len=2048.0, low_turns=1.0, high_turns=4.0, attn_factor=1.1),
}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    c = dict(case)
    dt = DTYPES[c["dtype"]]
    B = c["batch"]
    if c["op"] == "heads":
        R, H, K, d = c["rows"], c["heads"], c["kv_heads"], c["dim"]
        # Q, K (and V) rows as the input projection lays them side by side
        fused = normal(B, R, H + 2 * K, d).mul_(torch.rand(H + 2 * K, 1, generator=gen, device="cuda") * 3 + 0.1).to(dt)
        c["q"], c["k"] = fused[:, :, :H], fused[:, :, H:H + K]
        c["q_out"], c["k_out"] = torch.zeros(B, R, H, d, dtype=dt, device="cuda"), torch.zeros(B, R, K, d, dtype=dt, device="cuda")
        c["wq"] = 1 + 0.2 * normal(d) if c["norm"] else None
        c["wk"] = 1 + 0.2 * normal(d) if c["norm"] else None
        c["positions"] = torch.randint(0, 1 << 20, (B, R), generator=gen, device="cuda") if c["given"] else None
        return c
    L, H, K, dk, dv = c.get("rows", 1), c["heads"], c["qk_heads"], c["dk"], c["dv"]
    c["rows"] = L
    c["q"] = (normal(B, L, K, dk) * dk ** -0.5).to(dt)
    c["k"] = normal(B, L, K, dk).to(dt)
    c["v"] = torch.nn.functional.silu(normal(B, L, H, dv)).to(dt)
    if c["decay"] == "token":  # a rate for each head times the token's step, as the step sizes come out of a softplus
        rate = 1 + 15 * torch.rand(H, generator=gen, device="cuda")
        delta = torch.nn.functional.softplus(normal(B, L, H) - 4)
        c["g"], c["s"] = -rate * delta, delta
    else:  # one decay for each head, from about 30 to about 1000 tokens long
        c["g"] = torch.log1p(-torch.exp2(-5 - 5 * torch.rand(H, generator=gen, device="cuda"))).expand(B, L, H)
        c["s"] = None
    c["skip"] = 1 + 0.1 * normal(H, dv) if c["epilogue"] else None
    c["gate"] = torch.nn.functional.silu(normal(B, L, H, dv)).to(dt) if c["epilogue"] else None
    c["state"] = normal(B, H, dv, dk) if c["op"] == "step" or c["start"] else None
    c["state_out"] = torch.zeros(B, H, dv, dk, device="cuda")
    c["lengths"] = None
    if c["ragged"]:
        c["lengths"] = torch.randint(0, L + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    c["o"] = torch.zeros(B, L, H, dv, dtype=dt, device="cuda")
    return c


# ---------------------------------------------------------------------------------------- plain forms

def _frequencies(rot, base, factor=1.0, orig_len=0.0, low_turns=0.0, high_turns=0.0, attn_factor=1.0, device="cuda"):
    """Radians per position of each pair, in 64 bits."""
    f = base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    if not orig_len:
        return f / factor
    turns = orig_len * f / (2 * math.pi)
    keep = ((turns - low_turns) / (high_turns - low_turns)).clamp(0, 1)
    return keep * f + (1 - keep) * f / factor


def _heads_plain(c):
    opt = ROPE[c["scaling"]]
    if c["given"]:
        pos = c["positions"].double()
    else:
        pos = (c["pos0"] + torch.arange(c["rows"], device="cuda")).double().expand(c["batch"], -1)
    angle = pos[:, :, None, None] * _frequencies(c["rot"], **opt)
    m = opt.get("attn_factor", 1.0)
    cos, sin = (angle.cos() * m).float(), (angle.sin() * m).float()
    rot = c["rot"]

    def one(x, w):
        y = x.float()
        if c["norm"]:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w
        if c["layout"] == "pairs":
            a, b = y[..., 0:rot:2], y[..., 1:rot:2]
            r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        else:
            a, b = y[..., :rot // 2], y[..., rot // 2:rot]
            r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        return torch.cat((r, y[..., rot:]), -1).to(x.dtype)

    return one(c["q"], c["wq"]), one(c["k"], c["wk"])


CHUNK = 64


def _prompt_plain(c):
    """Chunks of 64 rows: inside a chunk by the masked scores, between chunks by the states at their ends."""
    B, L, H, K, dk, dv = (c[n] for n in ("batch", "rows", "heads", "qk_heads", "dk", "dv"))
    n = -(-L // CHUNK)
    pad = n * CHUNK - L
    valid = torch.ones(B, L, dtype=torch.bool, device="cuda")
    if c["lengths"] is not None:
        valid = torch.arange(L, device="cuda") < c["lengths"][:, None]

    def rows(x, heads):  # [B, L, heads, d] -> [B, heads, n, CHUNK, d]
        x = x.float() * valid[:, :, None, None]
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad))
        return x.view(B, n, CHUNK, heads, -1).permute(0, 3, 1, 2, 4)

    q, k, v = rows(c["q"], K), rows(c["k"], K), rows(c["v"], H)
    g = rows(c["g"][..., None], H)[..., 0].double().cumsum(-1)  # [B, H, n, CHUNK]
    if c["s"] is not None:
        v = v * rows(c["s"][..., None], H)
    end = g[..., -1]
    # states at the start of each chunk
    w = (end[..., None] - g).exp().float()
    own_state = (v * w[..., None]).transpose(-1, -2).view(B, K, H // K, n, dv, CHUNK) @ k[:, :, None]
    own_state = own_state.reshape(B, H, n, dv * dk)
    total = torch.cat((torch.zeros_like(end[..., :1]), end.cumsum(-1)), -1)  # before each chunk, and at the end
    step = total[..., :, None] - total[..., None, 1:]
    live = torch.arange(n + 1, device="cuda")[:, None] > torch.arange(n, device="cuda")
    carry = torch.where(live, step, -math.inf).exp().float()
    states = carry @ own_state
    if c["state"] is not None:
        states = states + total.exp().float()[..., None] * c["state"].reshape(B, H, 1, dv * dk)
    states = states.view(B, H, n + 1, dv, dk)
    # outputs
    tri = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device="cuda").tril()
    decay = torch.where(tri, g[..., :, None] - g[..., None, :], -math.inf).float().exp()
    p = (q @ k.transpose(-1, -2))[:, :, None] * decay.view(B, K, H // K, n, CHUNK, CHUNK)
    o = p.view(B, H, n, CHUNK, CHUNK) @ v
    qs = q[:, :, None] @ states[:, :, :n].reshape(B, K, H // K, n, dv, dk).transpose(-1, -2)
    o = o + g.exp().float()[..., None] * qs.view(B, H, n, CHUNK, dv)
    o = o.permute(0, 2, 3, 1, 4).reshape(B, n * CHUNK, H, dv)[:, :L]
    return _epilogue(c, o, valid), states[:, :, n].contiguous()


def _epilogue(c, o, valid):
    if c["epilogue"]:
        o = (o + c["skip"] * c["v"].float()) * c["gate"].float()
    return torch.where(valid[:, :, None, None], o, c["o"].float()).to(c["o"].dtype)


def _step_plain(c):
    B, H, K = c["batch"], c["heads"], c["qk_heads"]
    on = torch.ones(B, dtype=torch.bool, device="cuda") if c["lengths"] is None else c["lengths"] > 0
    q, k = (c[n][:, 0].float().repeat_interleave(H // K, 1) for n in "qk")
    v = c["v"][:, 0].float()
    x = v if c["s"] is None else v * c["s"][:, 0, :, None]
    new = c["g"][:, 0].exp()[..., None, None] * c["state"] + x[..., None] * k[:, :, None]
    o = (new * q[:, :, None]).sum(-1)
    state = torch.where(on[:, None, None, None], new, c["state"])
    return _epilogue(c, o[:, None], on[:, None]), state


# ---------------------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _run_own(state)
    return {"heads": _heads_plain, "prompt": _prompt_plain, "step": _step_plain}[state["op"]](state)


def _run_own(c):
    import hybrid_attention_ssm_head_b200 as hy
    stream = torch.cuda.current_stream()
    if c["op"] == "heads":
        if "call" not in c:  # the description of its buffers and of the rotation that a program fills in once
            rope = hy.make_rope(c["rot"], c["layout"], scaling=c["scaling"], **ROPE[c["scaling"]])
            c["call"] = hy.make_qk_norm_rope(c["q"], c["k"], c["q_out"], c["k_out"], norm=c["norm"], eps=1e-6,
                                             q_weight=c["wq"], k_weight=c["wk"], rope=rope,
                                             pos0=0 if c["given"] else c["pos0"], positions=c["positions"])
        hy.hymba_qk_norm_rope(c["call"], stream)
        return c["q_out"], c["k_out"]
    if "call" not in c:  # the description of its buffers and the workspace that a program keeps
        args = hy.make_linear_attention(c["q"], c["k"], c["v"], c["o"], c["g"], in_scale=c["s"], skip=c["skip"],
                                        gate=c["gate"], state_in=c["state"], state_out=c["state_out"],
                                        lengths=c["lengths"])
        ws = torch.empty(max(1, hy.hymba_linear_attention_workspace(args)), dtype=torch.uint8, device="cuda")
        c["call"] = (args, ws)
    args, ws = c["call"]
    if c["op"] == "prompt":
        hy.hymba_linear_attention_prefill(args, ws, ws.numel(), stream)
    else:
        hy.hymba_linear_attention_decode_step(args, stream)
    return c["o"], c["state_out"]


# ---------------------------------------------------------------------------------------- work

def work(case):
    c = case
    es = 2 if c["dtype"] == "bf16" else 4
    B, R = c["batch"], c.get("rows", 1)
    if c["op"] == "heads":
        n = B * R * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 2 * n * es + (8 * B * R if c["given"] else 0) + 8 * c["dim"], "flops": 8 * n}
    H, K, dk, dv = c["heads"], c["qk_heads"], c["dk"], c["dv"]
    epi, per = c["epilogue"], c["decay"] == "token"
    row = 2 * K * dk * es + (3 if epi else 2) * H * dv * es + (8 * H if per else 0)
    state = 4 * B * H * dk * dv
    reads = 1 + (1 if c["op"] == "step" or c.get("start") else 0)
    return {"bytes": B * R * row + reads * state + (4 * H * dv if epi else 0) + (0 if per else 4 * H),
            "flops": B * R * H * (5 * dk * dv + (3 * dv if epi else 0))}


# ---------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definitions of the head of this file, step by step in 64 bits."""
    c = prepare(case, seed)
    B, L = c["batch"], c["rows"]
    if c["op"] == "heads":
        return _heads_exact(c)
    H, K = c["heads"], c["qk_heads"]
    lengths = torch.full((B,), L, device="cuda") if c["lengths"] is None else c["lengths"]
    head = torch.arange(H, device="cuda") // (H // K)
    S = torch.zeros(B, H, c["dv"], c["dk"], dtype=torch.float64, device="cuda")
    if c["state"] is not None:
        S += c["state"]
    o = c["o"].double()
    for t in range(L):
        on = (t < lengths)[:, None, None]
        q, k, v = (c[n][:, t].double() for n in "qkv")
        v = torch.where(on, v, 0)
        x = v if c["s"] is None else v * c["s"][:, t, :, None]
        S *= torch.where(on[..., 0], c["g"][:, t].double(), 0).exp()[..., None, None]
        S += x[..., :, None] * torch.where(on, k, 0)[:, head][..., None, :]
        y = (S @ q[:, head][..., None])[..., 0]
        if c["epilogue"]:
            y = (y + c["skip"].double() * v) * c["gate"][:, t].double()
        o[:, t] = torch.where(on, y, o[:, t])
    return o, S


def _heads_exact(c):
    opt = dict(ROPE[c["scaling"]])
    rot, m = c["rot"], opt.get("attn_factor", 1.0)
    pos = c["positions"] if c["given"] else (c["pos0"] + torch.arange(c["rows"], device="cuda"))[None].expand(c["batch"], -1)
    i = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    theta = torch.pow(torch.tensor(opt["base"], dtype=torch.float64, device="cuda"), -2 * i / rot)
    if c["scaling"] == "linear":
        theta = theta / opt["factor"]
    elif c["scaling"] == "wavelength":
        r = opt["orig_len"] / (2 * math.pi / theta)
        lo, hi = opt["low_turns"], opt["high_turns"]
        mix = torch.where(r <= lo, torch.zeros_like(r), torch.where(r >= hi, torch.ones_like(r), (r - lo) / (hi - lo)))
        theta = theta * (mix + (1 - mix) / opt["factor"])
    turn = torch.polar(torch.full_like(pos, m, dtype=torch.float64)[..., None] + 0 * theta, pos.double()[..., None] * theta)

    def one(x, w):
        y = x.double()
        if c["norm"]:
            y = y / torch.sqrt(y.square().sum(-1, keepdim=True) / y.shape[-1] + 1e-6) * w.double()
        y = y.clone()
        first = slice(0, rot, 2) if c["layout"] == "pairs" else slice(0, rot // 2)
        second = slice(1, rot, 2) if c["layout"] == "pairs" else slice(rot // 2, rot)
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * turn[:, :, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    return one(c["q"], c["wq"]), one(c["k"], c["wk"])
