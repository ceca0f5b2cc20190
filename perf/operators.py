"""Measured cases of the token-level operators: rotary positions over (time, height, width),
attention with one decay per head in its chunked form, its form for single tokens, and its
backward pass.

Layouts are the library's: Q, K, V, O [B, H, T, U, d] (the token sequence of a (batch, head) pair is
its T * U tokens in order), states [B, H, d_v, d_k] float32.

  rotary     y = R(pos) x: on each axis a, channel pair i turns by pos_a * scale_a * theta^(-2 i / dim_a)
  attention  S_i = exp(g_h) S_{i-1} + v_i k_i^T,  o_i = S_i q_i   (g_h <= 0 one value per head)
  backward   dq_i = S_i^T do_i,  Z_i = exp(g_h) Z_{i+1} + do_i q_i^T (Z_n = dS_out / exp(g_h)),
             dk_i = Z_i^T v_i,  dv_i = Z_i k_i,  dS_in = exp(g_h) Z_0
"""
import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases
def listed():
    return [
        # one denoising pass: the rotary positions of Q and K of the whole clip (102 latent frames of a
        # 24 x 42 token grid)
        dict(name="rotary_clip", op="rotary", B=1, H=24, T=102, gh=24, gw=42, d=128, dtype="bf16", dim_t=44, dim_h=42,
             dim_w=42, interleaved=True, inverse=False, layout="head", positions="grid", frame0=0, theta=10000.0,
             scale=1.0),
        # a live stream far into its run: one five-frame segment straight from the QKV projection
        # (token-major), with V brought into the head-major layout by the same call
        dict(name="rotary_stream_qkv", op="rotary", B=1, H=24, T=5, gh=24, gw=42, d=128, dtype="bf16", dim_t=16,
             dim_h=56, dim_w=56, interleaved=False, inverse=False, layout="qkv", positions="grid", frame0=1234567,
             theta=256.0, scale=0.5),
        # the gradient's way back through the rotation in float32, on an odd grid
        dict(name="rotary_inverse_f32", op="rotary", B=2, H=4, T=19, gh=15, gw=17, d=64, dtype="f32", dim_t=20,
             dim_h=20, dim_w=20, interleaved=False, inverse=True, layout="head", positions="grid", frame0=0,
             theta=10000.0, scale=1.0),
        # one generated token per sequence, at positions that the caller gives
        dict(name="rotary_tokens", op="rotary", B=16, H=24, T=1, gh=1, gw=1, d=128, dtype="bf16", dim_t=44, dim_h=42,
             dim_w=42, interleaved=True, inverse=False, layout="qkv", positions="given", frame0=0, theta=10000.0,
             scale=1.0),
        # a whole clip as one token sequence, few heads and a long axis
        dict(name="attn_clip", op="attn", B=1, H=24, T=102, U=1008, d=128, dtype="bf16", ragged=False, state_in=True),
        # text prompts
        dict(name="attn_text", op="attn", B=4, H=24, T=1, U=512, d=128, dtype="bf16", ragged=False, state_in=False),
        # a padded batch of prompts of unequal length, one of them empty
        dict(name="attn_ragged", op="attn", B=8, H=16, T=1, U=4099, d=64, dtype="bf16", ragged=True, state_in=True),
        # the float32 form at the small configuration's size
        dict(name="attn_f32", op="attn", B=1, H=4, T=20, U=256, d=64, dtype="f32", ragged=False, state_in=True),
        # one token of one sequence: latency
        dict(name="step_one", op="step", B=1, H=24, d=128, dtype="bf16", idle=False),
        # one token of each of a serving batch's sequences, some slots idle
        dict(name="step_batch", op="step", B=96, H=24, d=128, dtype="bf16", idle=True),
        # the backward pass over twenty frames
        dict(name="backward_frames", op="backward", B=1, H=24, T=20, U=1008, d=128, dtype="bf16", ragged=False,
             state_in=True),
        # the backward pass of a short padded float32 batch
        dict(name="backward_f32", op="backward", B=3, H=4, T=1, U=777, d=32, dtype="f32", ragged=True, state_in=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "attn", "attn", "attn", "step", "backward", "backward"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "rotary":
        d = rng.choice([32, 64, 128])
        while True:
            B, H, T = _log(rng, 1, 8), _log(rng, 1, 32), _log(rng, 1, 150)
            gh, gw = _log(rng, 1, 48), _log(rng, 1, 84)
            if B * H * T * gh * gw * d * (2 if dtype == "f32" else 1) <= 24 * 102 * 1008 * 128 // 2:
                break
        pairs = d // 2
        pt = rng.randint(0, pairs)
        ph = rng.randint(0, pairs - pt)
        pw = rng.randint(0, pairs - pt - ph)
        if pt + ph + pw == 0:
            pt = pairs
        return dict(op="rotary", B=B, H=H, T=T, gh=gh, gw=gw, d=d, dtype=dtype, dim_t=2 * pt, dim_h=2 * ph, dim_w=2 * pw,
                    interleaved=rng.random() < 0.5, inverse=rng.random() < 0.3, layout=rng.choice(["head", "qkv"]),
                    positions=rng.choice(["grid", "grid", "given"]), frame0=rng.choice([0, _log(rng, 1, 4000000)]),
                    theta=rng.choice([256.0, 10000.0, 500000.0]), scale=rng.choice([1.0, 0.5, 1.25]))
    if op == "step":
        return dict(op="step", B=_log(rng, 1, 96), H=_log(rng, 1, 32), d=rng.choice([16, 32, 64, 128]), dtype=dtype,
                    idle=rng.random() < 0.5)
    d = rng.choice([16, 32, 64, 128, 128])
    limit = (24 * 102 * 1008 * 128 if op == "attn" else 24 * 20 * 1008 * 128) // (8 if dtype == "f32" else 1)
    while True:
        B, H, T, U = _log(rng, 1, 16), _log(rng, 1, 32), _log(rng, 1, 100), _log(rng, 1, 4000)
        if B * H * T * U * d <= limit:
            break
    return dict(op=op, B=B, H=H, T=T, U=U, d=d, dtype=dtype, ragged=rng.random() < 0.5, state_in=rng.random() < 0.7)


# -------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) & 0x7FFFFFFFFFFFFFFF)
    return g


def _randn(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _keys(g, shape, dtype):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return (x / x.norm(dim=-1, keepdim=True)).to(dtype)


def _log_decay(g, H):
    # from heads that keep a few tokens to heads that keep ten thousand; the first one forgets nothing
    x = -torch.exp(torch.rand(H, generator=g, device="cuda") * (math.log(0.7) - math.log(1e-4)) + math.log(1e-4))
    x[0] = 0.0
    return x.contiguous()


def _lens(g, B, n):
    x = torch.randint(1, n + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    x[0] = n
    if B > 1:
        x[1] = 0
    return x


def prepare(case, seed):
    g, c = _gen(seed), case
    dt = _DTYPES[c["dtype"]]
    B, H, d = c["B"], c["H"], c["d"]
    st = {"case": c}
    if c["op"] == "rotary":
        T, U = c["T"], c["gh"] * c["gw"]
        n = T * U
        if c["layout"] == "qkv":
            qkv = _randn(g, (B, n, 3, H, d), dt)
            st["x"] = [qkv[:, :, i].permute(0, 2, 1, 3).unflatten(2, (T, U)) for i in range(3)]
        else:
            st["x"] = [_randn(g, (B, H, T, U, d), dt) for _ in range(2)]
        st["y"] = [torch.empty((B, H, T, U, d), dtype=dt, device="cuda") for _ in st["x"]]
        st["pos"] = None
        if c["positions"] == "given":
            st["pos"] = torch.randint(0, 40000, (B, n, 3), generator=g, device="cuda", dtype=torch.int32)
    elif c["op"] == "step":
        st["q"], st["k"], st["v"] = _randn(g, (B, H, d), dt), _keys(g, (B, H, d), dt), _randn(g, (B, H, d), dt)
        st["g"] = _log_decay(g, H)
        st["s_in"] = torch.randn((B, H, d, d), generator=g, device="cuda") * 0.5
        st["s_out"], st["o"] = torch.zeros_like(st["s_in"]), torch.zeros_like(st["q"])
        st["active"] = None
        if c["idle"]:
            st["active"] = (torch.rand(B, generator=g, device="cuda") < 0.8).to(torch.int32)
    else:
        T, U = c["T"], c["U"]
        shape = (B, H, T, U, d)
        st["q"], st["k"], st["v"] = _randn(g, shape, dt), _keys(g, shape, dt), _randn(g, shape, dt)
        st["g"] = _log_decay(g, H)
        st["lens"] = _lens(g, B, T * U) if c["ragged"] else None
        st["s_in"] = torch.randn((B, H, d, d), generator=g, device="cuda") * 0.5 if c["state_in"] else None
        if c["op"] == "attn":
            st["o"] = torch.zeros_like(st["q"])
            st["s_out"] = torch.zeros((B, H, d, d), device="cuda")
        else:
            st["do"] = _randn(g, shape, dt)
            st["ds_out"] = torch.randn((B, H, d, d), generator=g, device="cuda") * 0.5 if c["state_in"] else None
            st["dq"], st["dk"], st["dv"] = (torch.zeros_like(st["q"]) for _ in range(3))
            st["ds_in"] = torch.zeros((B, H, d, d), device="cuda")
    if own:
        st["plan"] = _plan(c, st)
    return st


def _plan(c, st):
    """The shape, the arguments' structures and the workspace that a program keeps."""
    from frame_wise_delta_b200 import vdn
    T, U = (1, 1) if c["op"] == "step" else (c["T"], c["gh"] * c["gw"] if c["op"] == "rotary" else c["U"])
    s = vdn.make_shape(c["B"], c["H"], T, U, c["d"], 0, in_dtype=c["dtype"])
    if c["op"] == "rotary":
        r = vdn.rotary(c["dim_t"], c["dim_h"], c["dim_w"], grid=(c["gh"], c["gw"]), interleaved=c["interleaved"],
                       inverse=c["inverse"], frame0=c["frame0"], theta=c["theta"], scale=(c["scale"],) * 3, pos=st["pos"])
        return {"s": s, "r": r, "rotate": [1, 1, 0][:len(st["x"])]}
    if c["op"] == "step":
        return {"s": s}
    n = (vdn.vdn_decay_attn_workspace_bytes if c["op"] == "attn" else vdn.vdn_decay_attn_backward_workspace_bytes)(s)
    return {"s": s, "ws": vdn.workspace(n), "info": torch.zeros(1, dtype=torch.int32, device="cuda")}


# ----------------------------------------------------------------- one pass
def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rotary":
        return _rotary_plain(state)
    if op == "step":
        return _step_plain(state)
    if op == "attn":
        return _attn_plain(state)
    return _backward_plain(state)


def _run_own(st):
    from frame_wise_delta_b200 import vdn
    p, op = st["plan"], st["case"]["op"]
    if op == "rotary":
        vdn.vdn_rotary(p["s"], p["r"], st["x"], st["y"], p["rotate"])
        return st["y"]
    if op == "step":
        vdn.vdn_decay_step(p["s"], st["q"], st["k"], st["v"], st["g"], st["active"], st["s_in"], st["o"], st["s_out"])
        return {"o": st["o"], "s": st["s_out"]}
    if op == "attn":
        vdn.vdn_decay_attn(p["s"], st["q"], st["k"], st["v"], st["g"], st["lens"], st["s_in"], st["o"], st["s_out"],
                           p["ws"], p["info"])
        return {"o": st["o"], "s": st["s_out"]}
    vdn.vdn_decay_attn_backward(p["s"], st["q"], st["k"], st["v"], st["g"], st["lens"], st["s_in"], st["do"],
                                st["ds_out"], st["dq"], st["dk"], st["dv"], st["ds_in"], p["ws"], p["info"])
    return {"dq": st["dq"], "dk": st["dk"], "dv": st["dv"], "ds": st["ds_in"]}


# -------------------------------------------------------------- plain forms
def _grid_positions(c):
    """[1, T * U, 3]: frame0 + t, row and column of each token."""
    t = torch.arange(c["T"], device="cuda", dtype=torch.float64) + c["frame0"]
    y = torch.arange(c["gh"], device="cuda", dtype=torch.float64)
    x = torch.arange(c["gw"], device="cuda", dtype=torch.float64)
    return torch.stack(torch.meshgrid(t, y, x, indexing="ij"), -1).reshape(1, -1, 3)


def _axis_angles(pos, dim, theta, scale):
    i = torch.arange(dim // 2, device="cuda", dtype=torch.float64)
    return (pos * scale)[..., None] * theta ** (-2.0 * i / max(dim, 1))


def _rotary_plain(st):
    c = st["case"]
    pos = _grid_positions(c) if st["pos"] is None else st["pos"].double()
    dims = (c["dim_t"], c["dim_h"], c["dim_w"])
    # one angle per pair; the pairs' channels as two index lists, the rest of the channels pass through
    ang = torch.cat([_axis_angles(pos[..., a], dims[a], c["theta"], c["scale"]) for a in range(3)], -1)
    first = [torch.arange(n // 2, device="cuda") for n in dims]
    start = [0, dims[0], dims[0] + dims[1]]
    if c["interleaved"]:
        lo = torch.cat([s + 2 * f for s, f in zip(start, first)])
        hi = lo + 1
    else:
        lo = torch.cat([s + f for s, f in zip(start, first)])
        hi = torch.cat([s + n // 2 + f for s, n, f in zip(start, dims, first)])
    cos, sin = ang.cos().float()[:, None], ang.sin().float()[:, None]
    if c["inverse"]:
        sin = -sin
    rotated = [_turn(x, lo, hi, cos, sin) for x in st["x"][:2]]
    return rotated + [x.contiguous() for x in st["x"][2:]]


def _turn(x, lo, hi, cos, sin):
    f = x.flatten(2, 3).float()
    a, b = f[..., lo], f[..., hi]
    y = f.clone()
    y[..., lo] = a * cos - b * sin
    y[..., hi] = a * sin + b * cos
    return y.to(x.dtype).reshape(x.shape)


def _step_plain(st):
    q, k, v = st["q"].float(), st["k"].float(), st["v"].float()
    lam = torch.exp(st["g"])[None, :, None, None]
    s = st["s_in"] * lam + v[..., :, None] * k[..., None, :]
    o = (s @ q[..., None])[..., 0].to(st["q"].dtype)
    if st["active"] is not None:
        on = (st["active"] != 0)[:, None, None]
        s = torch.where(on[..., None], s, st["s_in"])
        o = torch.where(on, o, torch.zeros_like(o))
    return {"o": o, "s": s}


_C = 128  # tokens per chunk of the plain forms


def _tokens(x):
    """[B, H, T, U, d] as float32 [B, H, chunks, _C, d], zeros behind the last token."""
    f = x.flatten(2, 3).float()
    return torch.nn.functional.pad(f, (0, 0, 0, -f.shape[2] % _C)).unflatten(2, (-1, _C))


def _valid(st):
    n = st["q"].shape[2] * st["q"].shape[3]
    lens = st["lens"]
    if lens is None:
        lens = torch.full((st["q"].shape[0],), n, device="cuda", dtype=torch.int32)
    return n, lens.long()


def _power(g, n):
    """exp(g * n) for whole numbers n, 0 where n < 0; g [H], n any shape -> [H, *n.shape] float32."""
    e = g.double().reshape(-1, *([1] * n.dim())) * n.clamp(min=0)
    return torch.where(n >= 0, torch.exp(e), torch.zeros_like(e)).float()


def _chunks(q, k, v, g, back):
    """sum_j exp(g |i - j|) (q_i . k_j) v_j over j <= i (back: j >= i), chunk by chunk."""
    nc = q.shape[2]
    i = torch.arange(_C, device="cuda")
    c = torch.arange(nc, device="cuda")
    gap, ahead = (i[None, :] - i[:, None], c[None, :] - c[:, None]) if back else (i[:, None] - i[None, :], c[:, None] - c[None, :])
    near = (q @ k.transpose(-1, -2)) * _power(g, gap)[None, :, None] @ v
    weight = _power(g, i + 1 if back else _C - 1 - i)[None, :, None, :, None]
    sums = (v * weight).transpose(-1, -2) @ k                                   # a state per chunk
    before = (_power(g, (ahead - 1) * _C)[None] @ sums.flatten(3)).unflatten(3, sums.shape[3:])
    far = (q @ before.transpose(-1, -2)) * _power(g, _C - 1 - i if back else i + 1)[None, :, None, :, None]
    return near + far


def _masked(x, n, lens):
    """Zeros in the rows behind each sequence's last token."""
    t = torch.arange(x.shape[2] * _C, device="cuda").reshape(1, 1, -1, _C, 1)
    return torch.where(t < lens.reshape(-1, 1, 1, 1, 1), x, torch.zeros_like(x))


def _rows(y, like, n, lens):
    y = _masked(y, n, lens).flatten(2, 3)[:, :, :n]
    return y.to(like.dtype).reshape(like.shape)


def _batch_power(g, e):
    """exp(g_h e) for exponents e [B, ...] -> [B, H, ...], 0 where e < 0."""
    x = torch.exp(g.double().reshape(1, -1, *([1] * (e.dim() - 1))) * e.clamp(min=0).unsqueeze(1))
    return torch.where((e >= 0).unsqueeze(1), x, torch.zeros_like(x)).float()


def _attn_plain(st):
    n, lens = _valid(st)
    g = st["g"]
    q, k, v = (_masked(_tokens(st[x]), n, lens) for x in "qkv")
    o = _chunks(q, k, v, g, False)
    t = torch.arange(q.shape[2] * _C, device="cuda").reshape(1, -1, _C)
    last = _batch_power(g, lens.reshape(-1, 1, 1) - 1 - t)[..., None]           # weight of each token in S_out
    s = (v * last).flatten(2, 3).transpose(-1, -2) @ k.flatten(2, 3)
    if st["s_in"] is not None:
        s0 = st["s_in"]
        o = o + (q @ s0[:, :, None].transpose(-1, -2)) * _batch_power(g, t + 1)[..., None]
        s = s + s0 * _batch_power(g, lens)[..., None, None]
    return {"o": _rows(o, st["q"], n, lens), "s": s}


def _backward_plain(st):
    n, lens = _valid(st)
    g = st["g"]
    q, k, v, do = (_masked(_tokens(st[x]), n, lens) for x in ("q", "k", "v", "do"))
    t = torch.arange(q.shape[2] * _C, device="cuda").reshape(1, -1, _C)
    first = _batch_power(g, t + 1)[..., None]
    last = _batch_power(g, lens.reshape(-1, 1, 1) - 1 - t)[..., None]
    dq = _chunks(do, v, k, g, False)
    dk = _chunks(v, do, q, g, True)
    dv = _chunks(k, q, do, g, True)
    ds = (do * first).flatten(2, 3).transpose(-1, -2) @ q.flatten(2, 3)
    if st["s_in"] is not None:
        dq = dq + (do @ st["s_in"][:, :, None]) * first
        z = st["ds_out"]
        dk = dk + (v @ z[:, :, None]) * last
        dv = dv + (k @ z[:, :, None].transpose(-1, -2)) * last
        ds = ds + z * _batch_power(g, lens)[..., None, None]
    return {"dq": _rows(dq, st["q"], n, lens), "dk": _rows(dk, st["q"], n, lens), "dv": _rows(dv, st["q"], n, lens),
            "ds": ds}


# ---------------------------------------------------------------- work, exact
def _esize(c):
    return 2 if c["dtype"] == "bf16" else 4


def work(case):
    c = case
    B, H, d, e = c["B"], c["H"], c["d"], _esize(c)
    if c["op"] == "rotary":
        n = c["T"] * c["gh"] * c["gw"]
        x = (3 if c["layout"] == "qkv" else 2) * 2 * B * H * n * d * e
        return {"bytes": x + (B * n * 12 if c["positions"] == "given" else 0),
                "flops": 2 * B * H * n * 3 * (c["dim_t"] + c["dim_h"] + c["dim_w"])}
    if c["op"] == "step":
        on = 0.8 if c["idle"] else 1.0
        return {"bytes": B * H * (8 * d * d + on * 4 * d * e), "flops": on * B * H * 5 * d * d}
    # a ragged batch: one full sequence, one empty one, the others half full on average
    n = c["T"] * c["U"]
    rows = B * n if not c["ragged"] else (n if B == 1 else n + (B - 2) * (n + 1) / 2)
    st = B * H * d * d * 4
    if c["op"] == "attn":
        return {"bytes": 4 * rows * H * d * e + st * (2 if c["state_in"] else 1), "flops": rows * H * 4 * d * d}
    return {"bytes": 7 * rows * H * d * e + st * (3 if c["state_in"] else 1), "flops": rows * H * 10 * d * d}


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op = case["op"]
    if op == "rotary":
        return _rotary_exact(case, st)
    if op == "step":
        lam = st["g"].double().exp()
        s, o = st["s_in"].double(), torch.zeros_like(st["q"], dtype=torch.float64)
        on = [1] * case["B"] if st["active"] is None else st["active"].tolist()
        for b in range(case["B"]):
            if on[b]:
                s[b] = lam[:, None, None] * s[b] + torch.einsum("hi,hj->hij", st["v"][b].double(), st["k"][b].double())
                o[b] = torch.einsum("hij,hj->hi", s[b], st["q"][b].double())
        return {"o": o, "s": s}
    x = {n: st[n].double().flatten(2, 3) for n in "qkv"}
    B, H, n, d = x["q"].shape
    s0 = st["s_in"].double() if st["s_in"] is not None else torch.zeros((B, H, d, d), dtype=torch.float64, device="cuda")
    lens = [n] * B if st["lens"] is None else st["lens"].tolist()
    if op == "attn":
        o, s = _recurrence(x["q"], x["k"], x["v"], st["g"].double(), s0, lens)
        return {"o": o.reshape(st["q"].shape), "s": s}
    # the gradients of sum(o * do) + sum(s * ds_out) by differentiation of the recurrence
    leaves = [t.requires_grad_() for t in (x["q"], x["k"], x["v"], s0)]
    o, s = _recurrence(*leaves[:3], st["g"].double(), s0, lens)
    loss = (o * st["do"].double().flatten(2, 3)).sum()
    if st["ds_out"] is not None:
        loss = loss + (s * st["ds_out"].double()).sum()
    dq, dk, dv, ds = torch.autograd.grad(loss, leaves)
    shape = st["q"].shape
    return {"dq": dq.reshape(shape), "dk": dk.reshape(shape), "dv": dv.reshape(shape), "ds": ds}


def _recurrence(q, k, v, g, s0, lens, block=96):
    """The recurrence of each sequence, a block of tokens at a time; rows behind a sequence's end are 0."""
    B, H, n, d = q.shape
    rows, states = [], []
    for b in range(B):
        s, out = s0[b], []
        for a in range(0, lens[b], block):
            e = min(a + block, lens[b])
            m = e - a
            t = torch.arange(m, device=q.device, dtype=torch.float64)
            gap = t[:, None] - t[None, :]
            near = torch.exp(g[:, None, None] * gap.clamp(min=0)) * (gap >= 0)
            qb, kb, vb = q[b, :, a:e], k[b, :, a:e], v[b, :, a:e]
            o = torch.einsum("hij,hjv->hiv", torch.einsum("hik,hjk->hij", qb, kb) * near, vb)
            out.append(o + torch.exp(g[:, None] * (t + 1))[..., None] * torch.einsum("hvk,hik->hiv", s, qb))
            s = torch.exp(g * m)[:, None, None] * s + torch.einsum(
                "hjv,hjk->hvk", vb * torch.exp(g[:, None] * (m - 1 - t))[..., None], kb)
        rows.append(torch.cat(out + [torch.zeros((H, n - lens[b], d), dtype=q.dtype, device=q.device)], 1))
        states.append(s)
    return torch.stack(rows), torch.stack(states)


def _rotary_exact(c, st):
    """Complex products in 64 bits, axis by axis."""
    B, n = c["B"], c["T"] * c["gh"] * c["gw"]
    if st["pos"] is not None:
        pos = [st["pos"][..., a].double() for a in range(3)]
    else:
        u = torch.arange(n, device="cuda")
        per = c["gh"] * c["gw"]
        pos = [(u // per + c["frame0"]).double()[None], (u % per // c["gw"]).double()[None], (u % c["gw"]).double()[None]]
    out = []
    for k, x in enumerate(st["x"]):
        y = torch.empty(x.shape, dtype=torch.float64, device="cuda").flatten(2, 3)
        f = x.flatten(2, 3)
        if k == 2:
            out.append(f.double().reshape(x.shape))
            continue
        at = 0
        for a, dim in enumerate((c["dim_t"], c["dim_h"], c["dim_w"])):
            if dim:
                part = f[..., at:at + dim].double()
                z = part.unflatten(-1, (-1, 2)) if c["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
                z = torch.view_as_complex(z.contiguous())
                freq = torch.tensor([c["theta"] ** (-2.0 * i / dim) for i in range(dim // 2)], dtype=torch.float64,
                                    device="cuda")
                ang = (pos[a] * c["scale"])[:, None, :, None] * freq
                z = z * torch.polar(torch.ones_like(ang), -ang if c["inverse"] else ang)
                r = torch.view_as_real(z)
                y[..., at:at + dim] = r.flatten(-2) if c["interleaved"] else r.transpose(-1, -2).flatten(-2)
            at += dim
        y[..., at:] = f[..., at:].double()
        out.append(y.reshape(x.shape))
    return out
