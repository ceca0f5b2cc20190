"""GPU parity of the token-level operators (rotary positions, decay attention,
its gradients, single tokens) with their float64 definitions, their edges
(ragged and empty sequences, poisoned padding, heads that forget nothing or
everything, segments, far positions, strided tensors) and a run of them
together.

Tolerances. Half a step is u = 2^-8 (bf16) or 2^-24 (float32) of a value. A
bf16 output is rounded once (u |o|). On the tensor cores the scores are rounded
to bf16 too (u M_i, M_i = sum_j l^|i-j| |q_i . k_j| |v_j|), and so is the copy of
the state in front of a 64-token chunk that the outputs read (u R_i, R_i the sum
over k of that state's |X_vk| |q_ik|). The weighted values enter with two bf16
parts of their three (2^-15) and everything else is float32, with rounded sums
of at most d + n + 64 terms: below 2^-13 of A_i (M_i with |q|.|k|, and |S| |q|)
for the sizes here. A float32 output is off by 2^-24 (d + 128 + n / 64) A_i at most.
States: in float32 each product is off by 2^-23 at most and a sum of t rounded
additions of random sign by sqrt(t) half steps, t < 600: 2e-6 of the norm."""
import numpy as np
import pytest
import torch

from frame_wise_delta_b200 import vdn
from oracle import token_ops as tok

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _build():
    from frame_wise_delta_b200 import build
    build.build()
    assert torch.cuda.is_available()


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(seed, B, H, T, U, d, dt, names="qkv", g=None):
    r = np.random.default_rng(seed)
    x = {}
    for n in names:
        a = r.standard_normal((B, H, T, U, d))
        if n == "k":
            a /= np.linalg.norm(a, axis=-1, keepdims=True)
        x[n] = torch.from_numpy(a).to("cuda").to(DT[dt])
    if g is None:
        g = -np.exp(r.uniform(np.log(1e-4), np.log(0.7), H))
        g[0] = 0.0
    x["g"] = torch.tensor(np.asarray(g, np.float32), device="cuda")
    x["s"] = torch.from_numpy(r.standard_normal((B, H, d, d)).astype(np.float32) * 0.5).cuda()
    x["z"] = torch.from_numpy(r.standard_normal((B, H, d, d)).astype(np.float32) * 0.5).cuda()
    return x


def _flat(t):
    return _np(t).reshape(t.shape[0], t.shape[1], -1, t.shape[-1])


def _scales(q, k, v, g, lens=None, s_in=None, back=False):
    m, a = tok.decay_scale(q, k, v, g, s_in, back)
    return m, a, tok.state_reads(q, k, v, g, lens, s_in, back)


def _near(got, ref, scales, dt, n, d):
    """|got - ref| within the bound, element by element, on the rows that ref has."""
    rows = np.isfinite(ref)
    m, a, r = scales
    if dt == "bf16":
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * 1.01 * (m + r) + 2.0 ** -13 * a
    else:
        tol = 2.0 ** -24 * (d + 128 + n / 64) * a + 2.0 ** -24 * np.abs(ref)
    off = np.abs(got - ref)[rows] - tol[rows]
    assert np.isfinite(got[rows]).all()
    assert off.size == 0 or off.max() <= 0, float(off.max())


def _state_near(got, ref):
    assert np.linalg.norm(got - ref) <= 2e-6 * np.linalg.norm(ref)


def _poison(x, lens, names):
    """NaN and infinities behind each sequence's end."""
    for b, n in enumerate(lens):
        for k, name in enumerate(names):
            t = x[name].view(x[name].shape[0], x[name].shape[1], -1, x[name].shape[-1])
            t[b, :, n:] = [float("nan"), float("inf"), float("-inf"), 3e38][(b + k) % 4]


MARK = 7.0


def _attn(s, x, lens=None, s_in=True, s_out=None, stream=None):
    o = torch.full((s.B, s.H, s.T, s.U, s.dk), MARK, dtype=vdn.TORCH_DTYPE[s.out_dtype], device="cuda")
    if s_out is None:
        s_out = torch.full_like(x["s"], float("nan"))
    ws = vdn.workspace(vdn.vdn_decay_attn_workspace_bytes(s))
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    vdn.vdn_decay_attn(s, x["q"], x["k"], x["v"], x["g"], lt, x["s"] if s_in else None, o, s_out, ws, info, stream)
    torch.cuda.synchronize()
    assert int(info.item()) == 0
    return o, s_out


CASES = [
    # B, H, T, U, d, in, out, lens, state
    (1, 1, 1, 1, 16, "f32", "f32", None, True),
    (2, 3, 1, 1, 128, "bf16", "bf16", None, True),
    (1, 2, 3, 21, 32, "bf16", "bf16", None, False),
    (2, 2, 1, 64, 64, "bf16", "bf16", None, True),
    (1, 3, 1, 65, 128, "bf16", "bf16", None, True),
    (2, 2, 5, 26, 128, "bf16", "bf16", None, False),
    (1, 2, 1, 257, 16, "bf16", "bf16", None, True),
    (5, 2, 1, 200, 128, "bf16", "bf16", [200, 0, 1, 64, 129], True),
    (5, 2, 1, 200, 64, "bf16", "bf16", [63, 0, 200, 65, 1], True),
    (4, 2, 1, 150, 32, "bf16", "bf16", [150, 149, 0, 128], False),
    (4, 2, 2, 75, 64, "f32", "f32", [150, 0, 7, 64], True),
    (2, 2, 1, 130, 128, "f32", "f32", None, True),
    (2, 2, 1, 100, 32, "bf16", "f32", [100, 33], True),
    (2, 2, 1, 100, 16, "f32", "bf16", None, False),
    (1, 1, 1, 2500, 128, "bf16", "bf16", None, True),   # several segments
    (2, 1, 1, 2500, 64, "bf16", "bf16", [2500, 1300], True),
    (3, 1, 1, 2500, 32, "f32", "f32", [2500, 64, 0], True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
def test_attention(case):
    B, H, T, U, d, di, do, lens, state = case
    x = _inputs(11 + d + U, B, H, T, U, d, di)
    if lens:
        _poison(x, lens, "qkv")
    s = vdn.make_shape(B, H, T, U, d, 0, in_dtype=di, out_dtype=do)
    o, s1 = _attn(s, x, lens, state)
    q, k, v = (_flat(x[n]) for n in "qkv")
    s0 = _np(x["s"]) if state else None
    ref, ref_s = tok.decay_attn(q, k, v, _np(x["g"]), lens, s0)
    keep = np.isfinite(ref)
    q, k, v = (np.where(keep, y, 0.0) for y in (q, k, v))
    _near(_flat(o), ref, _scales(q, k, v, _np(x["g"]), lens, s0), do, T * U, d)
    _state_near(_np(s1), ref_s)
    # rows behind the end are left as they were
    assert (_flat(o)[~keep] == MARK).all()
    # and the call gives the same bits again
    o2, s2 = _attn(s, x, lens, state)
    assert torch.equal(o, o2) and torch.equal(s1, s2)


@pytest.mark.parametrize("d,di", [(128, "bf16"), (64, "bf16"), (32, "f32")])
def test_attention_decays(d, di):
    """Heads that forget nothing, everything, and nearly either."""
    g = [0.0, float("-inf"), -1e-7, -0.3, -0.65, -0.9, -5.0, -80.0]
    x = _inputs(5, 1, len(g), 1, 300, d, di, g=g)
    s = vdn.make_shape(1, len(g), 1, 300, d, 0, in_dtype=di)
    o, s1 = _attn(s, x)
    q, k, v = (_flat(x[n]) for n in "qkv")
    ref, ref_s = tok.decay_attn(q, k, v, np.array(g), None, _np(x["s"]))
    _near(_flat(o), ref, _scales(q, k, v, np.array(g), None, _np(x["s"])), di, 300, d)
    for h in range(len(g)):
        _state_near(_np(s1)[:, h], ref_s[:, h])


@pytest.mark.parametrize("di", ["bf16", "f32"])
def test_state_in_place_and_empty(di):
    x = _inputs(6, 2, 2, 1, 70, 64, di)
    s = vdn.make_shape(2, 2, 1, 70, 64, 0, in_dtype=di)
    o, s1 = _attn(s, x)
    st = x["s"].clone()
    o2, _ = _attn(s, {**x, "s": st}, s_out=st)
    assert torch.equal(o, o2) and torch.equal(st, s1)
    s0 = vdn.make_shape(2, 2, 0, 70, 64, 0, in_dtype=di)
    e = {**x, **{n: x[n][:, :, :0] for n in "qkv"}}
    _, s2 = _attn(s0, e)
    assert torch.equal(s2, x["s"])
    _, s2 = _attn(s0, e, s_in=False)
    assert (s2 == 0).all()


def test_attention_without_final_state_or_info():
    x = _inputs(7, 1, 2, 1, 90, 128, "bf16")
    s = vdn.make_shape(1, 2, 1, 90, 128, 0)
    o = torch.empty_like(x["q"])
    vdn.vdn_decay_attn(s, x["q"], x["k"], x["v"], x["g"], None, x["s"], o, None, None)
    torch.cuda.synchronize()
    assert torch.equal(o, _attn(s, x)[0])


BACK = [
    (1, 2, 1, 1, 16, "f32", None, True),
    (2, 2, 1, 1, 128, "bf16", None, True),
    (1, 3, 3, 31, 128, "bf16", None, True),
    (2, 2, 1, 64, 64, "bf16", None, False),
    (5, 2, 1, 200, 128, "bf16", [200, 0, 1, 64, 129], True),
    (4, 2, 1, 150, 32, "bf16", [150, 149, 0, 128], False),
    (4, 2, 2, 75, 64, "f32", [150, 0, 7, 64], True),
    (2, 2, 1, 130, 128, "f32", None, True),
    (1, 1, 1, 2500, 128, "bf16", None, True),
    (2, 1, 1, 2500, 64, "bf16", [2500, 1300], True),
    (3, 1, 1, 2500, 32, "f32", [2500, 64, 0], True),
]


def _backward(s, x, lens=None, state=True):
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = [torch.full_like(x["q"], MARK) for _ in range(3)]
    ds = torch.full_like(x["s"], float("nan"))
    ws = vdn.workspace(vdn.vdn_decay_attn_backward_workspace_bytes(s))
    info = torch.zeros(1, dtype=torch.int32, device="cuda")
    vdn.vdn_decay_attn_backward(s, x["q"], x["k"], x["v"], x["g"], lt, x["s"] if state else None, x["o"],
                                x["z"] if state else None, *out, ds, ws, info)
    torch.cuda.synchronize()
    assert int(info.item()) == 0
    return out, ds


@pytest.mark.parametrize("case", BACK, ids=str)
def test_backward(case):
    B, H, T, U, d, dt, lens, state = case
    x = _inputs(31 + d + U, B, H, T, U, d, dt, names="qkvo")
    if lens:
        _poison(x, lens, "qkvo")
    s = vdn.make_shape(B, H, T, U, d, 0, in_dtype=dt)
    out, ds = _backward(s, x, lens, state)
    q, k, v, do = (_flat(x[n]) for n in "qkvo")
    s0, z = (_np(x["s"]), _np(x["z"])) if state else (None, None)
    g = _np(x["g"])
    *refs, ref_s = tok.decay_attn_backward(q, k, v, g, do, lens, s0, z)
    keep = np.isfinite(refs[0])
    q, k, v, do = (np.where(keep, y, 0.0) for y in (q, k, v, do))
    tr = lambda t: None if t is None else np.swapaxes(t, -1, -2)  # noqa: E731
    scales = [_scales(do, v, k, g, lens, tr(s0)), _scales(v, do, q, g, lens, tr(z), back=True),
              _scales(k, q, do, g, lens, z, back=True)]
    for got, ref, sc in zip(out, refs, scales):
        _near(_flat(got), ref, sc, dt, T * U, d)
        assert (_flat(got)[~keep] == MARK).all()
    _state_near(_np(ds), ref_s)


def test_backward_decays():
    g = [0.0, float("-inf"), -1e-7, -0.3, -0.65, -0.9, -5.0, -80.0]
    x = _inputs(8, 1, len(g), 1, 300, 128, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(1, len(g), 1, 300, 128, 0)
    out, ds = _backward(s, x)
    q, k, v, do = (_flat(x[n]) for n in "qkvo")
    s0, z = _np(x["s"]), _np(x["z"])
    *refs, ref_s = tok.decay_attn_backward(q, k, v, np.array(g), do, None, s0, z)
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    g = np.array(g)
    scales = [_scales(do, v, k, g, None, tr(s0)), _scales(v, do, q, g, None, tr(z), back=True),
              _scales(k, q, do, g, None, z, back=True)]
    for got, ref, sc in zip(out, refs, scales):
        _near(_flat(got), ref, sc, "bf16", 300, 128)
    for h in range(len(g)):
        assert np.linalg.norm(_np(ds)[:, h] - ref_s[:, h]) <= 2e-6 * np.linalg.norm(ref_s[:, h]) + 1e-30


def test_backward_is_the_difference():
    """The gradients against central differences of the float32 forward pass,
    summed in float64: the loss is linear in each argument, so a difference is
    off by the rounding of the outputs alone (2^-24 each, over the step)."""
    x = _inputs(9, 1, 2, 1, 80, 32, "f32", names="qkvo")
    s = vdn.make_shape(1, 2, 1, 80, 32, 0, in_dtype="f32")
    out, ds = _backward(s, x)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(y):
        o, s1 = _attn(s, y)
        return float((o.double() * x["o"].double()).sum() + (s1.double() * x["z"].double()).sum())

    mag = float((_attn(s, x)[0].double() * x["o"].double()).abs().sum() + (_attn(s, x)[1].double() * x["z"].double()).abs().sum())
    for name, grad in zip("qkvs", [*out, ds]):
        e = torch.randn(x[name].shape, generator=gen, device="cuda")
        h = 0.25
        diff = (loss({**x, name: x[name] + h * e}) - loss({**x, name: x[name] - h * e})) / (2 * h)
        # both losses hold sums of about `mag` whose terms carry 2^-20 each at most
        assert abs(diff - float((grad.double() * e.double()).sum())) <= 2.0 ** -20 * mag / h


STEP = [(1, 1, 16, "f32", "f32", None), (3, 5, 32, "bf16", "bf16", [1, 0, 1]), (2, 3, 64, "bf16", "f32", None),
        (4, 24, 128, "bf16", "bf16", [0, 1, 5, 0]), (2, 2, 128, "f32", "f32", None), (2, 3, 16, "f32", "bf16", [0, -1])]


@pytest.mark.parametrize("case", STEP, ids=str)
@pytest.mark.parametrize("in_place", [False, True])
def test_step(case, in_place):
    B, H, d, di, do, active = case
    g = [[0.0, float("-inf"), -0.01, -2.0][h % 4] for h in range(H)]
    x = _inputs(40 + d, B, H, 1, 1, d, di, g=g)
    s = vdn.make_shape(B, H, 1, 1, d, 0, in_dtype=di, out_dtype=do)
    q, k, v = (x[n].view(B, H, d) for n in "qkv")
    lens = None if active is None else [int(a != 0) for a in active]
    if lens:
        for t in (q, k, v):
            t[[b for b in range(B) if not lens[b]]] = float("nan")
    o = torch.full((B, H, d), MARK, dtype=DT[do], device="cuda")
    st = x["s"].clone()
    s1 = st if in_place else torch.full_like(st, float("nan"))
    vdn.vdn_decay_step(s, q, k, v, x["g"], None if active is None else torch.tensor(active, dtype=torch.int32, device="cuda"),
                       st, o, s1)
    torch.cuda.synchronize()
    fq, fk, fv = (_flat(x[n]) for n in "qkv")
    ref, ref_s = tok.decay_attn(fq, fk, fv, np.array(g), lens, _np(x["s"]))
    keep = np.isfinite(ref)
    fq, fk, fv = (np.where(keep, y, 0.0) for y in (fq, fk, fv))
    _, a = tok.decay_scale(fq, fk, fv, np.array(g), _np(x["s"]))
    got = _np(o)[:, :, None]
    u = 2.0 ** -8 if do == "bf16" else 2.0 ** -24
    tol = u * np.abs(ref) + 2.0 ** -24 * (d + 4) * a
    assert (np.abs(got - ref)[keep] <= tol[keep]).all()
    assert (got[~keep] == MARK).all()
    _state_near(_np(s1), ref_s)
    if lens:
        off = [b for b in range(B) if not lens[b]]
        assert torch.equal(s1[off], x["s"][off])


ROT = [
    # B, H, T, gh, gw, d, dtype, dims, interleaved, inverse, frame0, scale
    (1, 1, 1, 1, 1, 16, "f32", (16, 0, 0), True, False, 0, 1.0),
    (2, 3, 3, 5, 7, 128, "bf16", (44, 42, 42), True, False, 0, 1.0),
    (2, 3, 3, 5, 7, 128, "bf16", (44, 42, 42), False, False, 3, 0.5),
    (1, 2, 2, 4, 9, 128, "bf16", (16, 56, 56), False, True, 0, 1.0),
    (1, 2, 2, 4, 9, 64, "f32", (20, 20, 20), False, False, 999999937, 1.25),
    (2, 1, 4, 3, 3, 64, "f32", (0, 30, 34), True, True, 0, 1.0),
    (1, 5, 2, 3, 5, 32, "bf16", (0, 0, 0), True, False, 0, 1.0),
    (1, 2, 70, 1, 2, 32, "bf16", (8, 4, 4), False, False, 1 << 40, 0.25),
    (3, 2, 1, 1, 700, 16, "f32", (2, 2, 10), False, False, 0, 1.0),
]


@pytest.mark.parametrize("case", ROT, ids=str)
@pytest.mark.parametrize("layout", ["head", "token", "given"])
def test_rotary(case, layout):
    B, H, T, gh, gw, d, dt, dims, inter, inv, frame0, scale = case
    U, n = gh * gw, T * gh * gw
    r = np.random.default_rng(60 + d + n)
    if layout == "token":
        qkv = torch.from_numpy(r.standard_normal((B, n, 3, H, d))).cuda().to(DT[dt])
        xs = [qkv[:, :, i].permute(0, 2, 1, 3).unflatten(2, (T, U)) for i in range(3)]
    else:
        xs = [torch.from_numpy(r.standard_normal((B, H, T, U, d))).cuda().to(DT[dt]) for _ in range(2)]
    rest = sum(dims)
    if rest < d:
        xs[0][..., rest] = float("inf")  # passes through, and spoils nobody
        xs[0][..., d - 1] = float("nan")
    pos, pos_t = tok.grid_positions(T, gh, gw, frame0), None
    if layout == "given":
        pos = r.integers(-5, 2000000, (B, n, 3))
        pos_t = torch.from_numpy(pos.astype(np.int32)).cuda()
    s = vdn.make_shape(B, H, T, U, d, 0, in_dtype=dt)
    rot = vdn.rotary(*dims, grid=(gh, gw), interleaved=inter, inverse=inv, frame0=frame0, theta=1000.0, scale=(scale, 1.0, scale),
                     pos=pos_t)
    ys = [torch.full((B, H, T, U, d), MARK, dtype=DT[dt], device="cuda") for _ in xs]
    turned = [1, 1, 0][:len(xs)]
    vdn.vdn_rotary(s, rot, xs, ys, turned)
    torch.cuda.synchronize()
    u = 2.0 ** -8 if dt == "bf16" else 2.0 ** -24
    for x, y, t in zip(xs, ys, turned):
        if not t:
            assert torch.equal(x, y)
            continue
        assert torch.equal(x[..., rest:].nan_to_num(1.0, 2.0), y[..., rest:].nan_to_num(1.0, 2.0))
        f, got = _flat(x)[..., :rest], _flat(y)[..., :rest]
        ref = tok.rotary(f, pos, dims, 1000.0, (scale, 1.0, scale), inter, inv)
        # the remainder of a turn, its sine and cosine (2 steps each) and the two
        # products in float32: under 16 half steps of the largest value, then the
        # output's rounding; beyond 2^40 turns the product in float64 itself is 2^-12 turns off
        tol = u * np.abs(ref) + (2.0 ** -20 + (0.01 if frame0 > 1 << 30 else 0)) * np.abs(f).max(initial=0)
        assert (np.abs(got - ref) <= tol).all()
    # in place
    if layout != "token":
        z = [x.clone() for x in xs]
        vdn.vdn_rotary(s, rot, z, z, turned)
        assert all(torch.equal(a.nan_to_num(1.0, 2.0), b.nan_to_num(1.0, 2.0)) for a, b in zip(z, ys))


def test_rotary_inverse_undoes():
    x = torch.randn(2, 3, 4, 35, 64, device="cuda")
    s = vdn.make_shape(2, 3, 4, 35, 64, 0, in_dtype="f32")
    y, z = torch.empty_like(x), torch.empty_like(x)
    for inter in (True, False):
        vdn.vdn_rotary(s, vdn.rotary(20, 22, 22, grid=(5, 7), interleaved=inter, frame0=123456), [x], [y])
        vdn.vdn_rotary(s, vdn.rotary(20, 22, 22, grid=(5, 7), interleaved=inter, frame0=123456, inverse=True), [y], [z])
        # two rotations, each off by 16 half steps of the largest value at most
        assert float((x - z).abs().max()) <= 32 * 2.0 ** -24 * float(x.abs().max())


def _serve(prompt, steps, B, H, d, dt):
    """A prompt's tokens, then single tokens, from a token-major projection."""
    n = prompt + steps
    r = np.random.default_rng(77)
    qkv = torch.from_numpy(r.standard_normal((B, n, 3, H, d)) * 0.3).cuda().to(DT[dt])
    g = torch.tensor([0.0, -0.02, -0.5][:H], device="cuda")
    dims = (d // 2, d // 4, d // 4)

    def rotated(a, b):
        s = vdn.make_shape(B, H, b - a, 1, d, 0, in_dtype=dt)
        xs = [qkv[:, a:b, i].permute(0, 2, 1, 3).unflatten(2, (b - a, 1)) for i in range(3)]
        ys = [torch.empty((B, H, b - a, 1, d), dtype=DT[dt], device="cuda") for _ in xs]
        vdn.vdn_rotary(s, vdn.rotary(*dims, grid=(1, 1), frame0=a), xs, ys, [1, 1, 0])
        return s, ys

    def attend(a, b, state):
        s, (q, k, v) = rotated(a, b)
        o, st = torch.empty_like(q), torch.empty((B, H, d, d), device="cuda")
        ws = vdn.workspace(vdn.vdn_decay_attn_workspace_bytes(s))
        vdn.vdn_decay_attn(s, q, k, v, g, None, state, o, st, ws)
        return o, st, (q, k, v)

    whole, end, (q, k, v) = attend(0, n, None)
    o, state, _ = attend(0, prompt, None)
    outs = [o]
    for i in range(prompt, n):
        s, ys = rotated(i, i + 1)
        y = [t.view(B, H, d) for t in ys]
        o1 = torch.empty_like(y[0])
        vdn.vdn_decay_step(s, *y, g, None, state, o1, state)
        outs.append(o1.view(B, H, 1, 1, d))
    torch.cuda.synchronize()
    got = torch.cat(outs, 2)
    ref, ref_s = tok.decay_attn(_flat(q), _flat(k), _flat(v), _np(g))
    for t in (whole, got):
        _near(_flat(t), ref, _scales(_flat(q), _flat(k), _flat(v), _np(g)), dt, n, d)
    _state_near(_np(state), ref_s)
    _state_near(_np(end), ref_s)


@pytest.mark.parametrize("d,dt", [(128, "bf16"), (64, "bf16"), (32, "f32")])
def test_prompt_then_tokens(d, dt):
    _serve(150, 6, 2, 3, d, dt)


@pytest.mark.parametrize("n", [100, 2500])
def test_other_stream_and_graph(n):
    """On a side stream, and captured: replays follow the inputs, two graphs share a workspace in turn."""
    x = _inputs(12, 1, 2, 1, n, 128, "bf16", names="qkvo")
    y = _inputs(13, 1, 2, 1, n, 128, "bf16", names="qkvo", g=x["g"].cpu().numpy())
    s = vdn.make_shape(1, 2, 1, n, 128, 0)
    want, want_y = (_attn(s, x), _backward(s, x)), (_attn(s, y), _backward(s, y))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        o, s1 = _attn(s, x)
    assert torch.equal(o, want[0][0]) and torch.equal(s1, want[0][1])
    z = {k: t.clone() for k, t in x.items()}
    ws = vdn.workspace(max(vdn.vdn_decay_attn_workspace_bytes(s), vdn.vdn_decay_attn_backward_workspace_bytes(s)))
    o, s1, ds = torch.empty_like(z["q"]), torch.empty_like(z["s"]), torch.empty_like(z["s"])
    grads = [torch.empty_like(z["q"]) for _ in range(3)]
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        vdn.vdn_decay_attn(s, z["q"], z["k"], z["v"], z["g"], None, z["s"], o, s1, ws)
    with torch.cuda.graph(g2):
        vdn.vdn_decay_attn_backward(s, z["q"], z["k"], z["v"], z["g"], None, z["s"], z["o"], z["z"], *grads, ds, ws)
    for src, (fw, bw) in ((x, want), (y, want_y), (x, want)):
        for k in z:
            z[k].copy_(src[k])
        g1.replay()
        g2.replay()
        g1.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, fw[0]) and torch.equal(s1, fw[1])
        assert all(torch.equal(a, b) for a, b in zip(grads, bw[0])) and torch.equal(ds, bw[1])


def test_segments_summed_in_parts():
    """Enough pairs for a few segments each, whose sums are cut further; both walks, ragged ends in every part."""
    B, H, n, d = 2, 10, 1500, 64
    lens = [1500, 1130]
    x = _inputs(15, B, H, 1, n, d, "bf16", names="qkvo")
    s = vdn.make_shape(B, H, 1, n, d, 0)
    _poison(x, lens, "qkvo")
    out, ds = _backward(s, x, lens)
    o, s1 = _attn(s, x, lens)
    q, k, v, do = (_flat(x[c]) for c in "qkvo")
    g, s0, z = _np(x["g"]), _np(x["s"]), _np(x["z"])
    ref, ref_s = tok.decay_attn(q, k, v, g, lens, s0)
    *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do, lens, s0, z)
    keep = np.isfinite(ref)
    q, k, v, do = (np.where(keep, y, 0.0) for y in (q, k, v, do))
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    _near(_flat(o), ref, _scales(q, k, v, g, lens, s0), "bf16", n, d)
    for got, want, sc in zip(out, refs, [_scales(do, v, k, g, lens, tr(s0)), _scales(v, do, q, g, lens, tr(z), back=True),
                                         _scales(k, q, do, g, lens, z, back=True)]):
        _near(_flat(got), want, sc, "bf16", n, d)
    _state_near(_np(s1), ref_s)
    _state_near(_np(ds), ref_ds)


@pytest.mark.parametrize("di,n", [("bf16", 3100), ("f32", 1100)])
def test_many_heads_in_segments(di, n):
    """24 heads of 128 channels, long enough for segments (their join then takes four values a thread),
    ragged; some of the heads against the definition."""
    B, H, d, pick = 2, 24, 128, [0, 11, 23]
    lens = [n, n - 777]
    x = _inputs(21, B, H, 1, n, d, di, names="qkvo")
    s = vdn.make_shape(B, H, 1, n, d, 0, in_dtype=di)
    assert vdn.vdn_decay_attn_workspace_bytes(s) > 0
    o, s1 = _attn(s, x, lens)
    out, ds = _backward(s, x, lens)
    for b in range(B):
        q, k, v, do = (_flat(x[c][b:b + 1, pick, :, :lens[b]]) for c in "qkvo")
        s0, z, g = _np(x["s"][b:b + 1, pick]), _np(x["z"][b:b + 1, pick]), _np(x["g"][pick])
        ref, ref_s = tok.decay_attn(q, k, v, g, None, s0)
        *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do, None, s0, z)
        tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
        scales = [_scales(q, k, v, g, None, s0), _scales(do, v, k, g, None, tr(s0)),
                  _scales(v, do, q, g, None, tr(z), back=True), _scales(k, q, do, g, None, z, back=True)]
        for got, want, sc in zip([o, *out], [ref, *refs], scales):
            _near(_flat(got[b:b + 1, pick, :, :lens[b]]), want, sc, di, n, d)
        _state_near(_np(s1[b:b + 1, pick]), ref_s)
        _state_near(_np(ds[b:b + 1, pick]), ref_ds)


@pytest.mark.parametrize("d", [64, 128])
def test_steep_decays(d):
    """Heads that forget within a chunk, on either side of each of the kernel's forms, forward and backward."""
    g = [-0.974, -0.976, -1.5, -2.5, -4.0, -4.61, -4.63, -12.0]
    x = _inputs(19, 1, len(g), 1, 150, d, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(1, len(g), 1, 150, d, 0)
    o, s1 = _attn(s, x)
    out, ds = _backward(s, x)
    q, k, v, do = (_flat(x[c]) for c in "qkvo")
    s0, z, g = _np(x["s"]), _np(x["z"]), np.array(g, np.float32).astype(np.float64)
    ref, ref_s = tok.decay_attn(q, k, v, g, None, s0)
    *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do, None, s0, z)
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    scales = [_scales(q, k, v, g, None, s0), _scales(do, v, k, g, None, tr(s0)),
              _scales(v, do, q, g, None, tr(z), back=True), _scales(k, q, do, g, None, z, back=True)]
    for got, want, sc in zip([o, *out], [ref, *refs], scales):
        _near(_flat(got), want, sc, "bf16", 150, d)
    for h in range(len(g)):
        _state_near(_np(s1)[:, h], ref_s[:, h])
        _state_near(_np(ds)[:, h], ref_ds[:, h])


@pytest.mark.parametrize("power", [-50, 40])
@pytest.mark.parametrize("n", [100, 2500])
def test_powers_of_two_pass_through(n, power):
    """Values and state times a power of two: the same bits times that power (gradients are often
    tiny), for heads whose weights span the widest range as well."""
    g = [0.0, -0.01, -0.7, -0.97, -1.2, -6.0]
    x = _inputs(20, 1, len(g), 1, n, 128, "bf16", g=g)
    s = vdn.make_shape(1, len(g), 1, n, 128, 0)
    o, s1 = _attn(s, x)
    f = 2.0 ** power
    o2, s2 = _attn(s, {**x, "v": x["v"] * f, "s": x["s"] * f})
    assert torch.equal(o * f, o2) and torch.equal(s1 * f, s2)


@pytest.mark.parametrize("di", ["bf16", "f32"])
def test_lengths_are_clamped(di):
    x = _inputs(16, 3, 2, 1, 100, 32, di)
    s = vdn.make_shape(3, 2, 1, 100, 32, 0, in_dtype=di)
    a = _attn(s, x, [100, 0, 37])
    b = _attn(s, x, [2 ** 31 - 1, -(2 ** 31), 37])
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_rotary_reads_a_broadcast_axis():
    x = torch.randn(1, 1, 4, 6, 32, device="cuda").expand(3, 5, 4, 6, 32)
    s = vdn.make_shape(3, 5, 4, 6, 32, 0, in_dtype="f32")
    r = vdn.rotary(16, 8, 8, grid=(2, 3))
    y, z = torch.empty(3, 5, 4, 6, 32, device="cuda"), torch.empty(3, 5, 4, 6, 32, device="cuda")
    vdn.vdn_rotary(s, r, [x], [y])
    vdn.vdn_rotary(s, r, [x.contiguous()], [z])
    assert torch.equal(y, z)
    with pytest.raises(vdn.VdnError):
        vdn.vdn_rotary(s, r, [z], [x])


@pytest.mark.slow
def test_offsets_beyond_32_bits():
    """140 000 pairs of 128 tokens, 2.3e9 values a tensor: the last pair as exact as if it were alone."""
    B, H, n, d = 1000, 140, 128, 128
    one = _inputs(17, 1, 1, 1, n, d, "bf16")
    big = {}
    for c in "qkv":
        big[c] = torch.zeros((B, H, 1, n, d), dtype=torch.bfloat16, device="cuda")
        big[c][-1, -1] = one[c][0, 0]
    g = torch.full((H,), float(one["g"][0]), device="cuda")
    s, s1 = vdn.make_shape(B, H, 1, n, d, 0), vdn.make_shape(1, 1, 1, n, d, 0)
    o = torch.full_like(big["q"], MARK)
    vdn.vdn_decay_attn(s, big["q"], big["k"], big["v"], g, None, None, o, None, None)
    want = torch.empty_like(one["q"])
    vdn.vdn_decay_attn(s1, one["q"], one["k"], one["v"], one["g"], None, None, want, None, None)
    assert torch.equal(o[-1, -1], want[0, 0])
    assert (o[0, 0] == 0).all() and (o[B // 2, 3] == 0).all()
    vdn.vdn_rotary(s, vdn.rotary(64, 32, 32, grid=(8, 16)), [big["v"]], [o])
    vdn.vdn_rotary(s1, vdn.rotary(64, 32, 32, grid=(8, 16)), [one["v"]], [want])
    assert torch.equal(o[-1, -1], want[0, 0])
    del big, o
    torch.cuda.empty_cache()


def test_two_streams_at_once():
    """Calls with workspaces of their own on two streams do not disturb each other."""
    xs = [_inputs(18 + i, 1, 2, 1, 2500, 128, "bf16") for i in range(2)]
    s = vdn.make_shape(1, 2, 1, 2500, 128, 0)
    want = [_attn(s, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [vdn.workspace(vdn.vdn_decay_attn_workspace_bytes(s)) for _ in xs]
    outs = [(torch.empty_like(x["q"]), torch.empty_like(x["s"])) for x in xs]
    torch.cuda.synchronize()
    for _ in range(20):
        for x, st, w, (o, s1) in zip(xs, streams, ws, outs):
            vdn.vdn_decay_attn(s, x["q"], x["k"], x["v"], x["g"], None, x["s"], o, s1, w, stream=st)
    torch.cuda.synchronize()
    for (o, s1), (a, b) in zip(outs, want):
        assert torch.equal(o, a) and torch.equal(s1, b)


def test_binding_refuses_other_shapes():
    x = _inputs(14, 1, 2, 1, 20, 64, "bf16")
    s = vdn.make_shape(1, 2, 1, 20, 64, 0)
    o, st = torch.empty_like(x["q"]), torch.empty_like(x["s"])
    ok = [s, x["q"], x["k"], x["v"], x["g"], None, x["s"], o, st, None]
    for at, bad in ((1, x["q"].float()), (2, x["k"][:, :1]), (4, x["g"].double()), (5, torch.zeros(1, device="cuda")),
                    (6, x["s"].transpose(2, 3)), (7, o.cpu()), (8, st[:1, :1])):
        args = list(ok)
        args[at] = bad
        with pytest.raises(vdn.VdnError):
            vdn.vdn_decay_attn(*args)


def _decayed(q, k, v, g, lens=None, s_in=None, back=False):
    return *tok.decayed_scale(q, k, v, g, lens, s_in, back), tok.state_reads(q, k, v, g, lens, s_in, back)


def _near_decayed(got, ref, scales, dt, n, d, floor):
    """_near with the state's share of the bound decayed as in the output, and `floor` for what lies below
    float32's range: a factor that is under 2^-126 counts as 0."""
    m, a, r = scales
    rows = np.isfinite(ref)
    if dt == "bf16":
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -8 * 1.01 * (m + r) + 2.0 ** -13 * a
    else:
        tol = 2.0 ** -24 * (d + 128 + n / 64) * a + 2.0 ** -24 * np.abs(ref)
    off = (np.abs(got - ref) - tol - floor)[rows]
    assert np.isfinite(got[rows]).all()
    assert off.size == 0 or off.max() <= 0, float(off.max())


@pytest.mark.parametrize("power", [0, 90])
@pytest.mark.parametrize("d,dt", [(64, "bf16"), (128, "bf16"), (64, "f32")])
def test_steep_heads_let_nothing_through(d, dt, power):
    """Heads that forget within a chunk: what is left of the start state, however large, and of a sequence's
    first tokens decays on as the formula says, down to float32's smallest numbers."""
    g = [-0.98, -1.2, -1.37, -1.4, -2.5, -5.0, -12.0, float("-inf")]
    n, f = 200, 2.0 ** power
    x = _inputs(23, 1, len(g), 1, n, d, dt, names="qkvo", g=g)
    x["v"][:, :, :, 3:] = 0                       # the first tokens alone write (back: the last ones)
    x["o"][:, :, :, :n - 3] = 0
    x["s"] *= f
    x["z"] *= f
    s = vdn.make_shape(1, len(g), 1, n, d, 0, in_dtype=dt)
    o, _ = _attn(s, x)
    out, _ = _backward(s, x)
    q, k, v, do = (_flat(x[c]) for c in "qkvo")
    s0, z, g = _np(x["s"]), _np(x["z"]), np.array(g, np.float32).astype(np.float64)
    ref, _ = tok.decay_attn(q, k, v, g, None, s0)
    *refs, _ = tok.decay_attn_backward(q, k, v, g, do, None, s0, z)
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    args = [(q, k, v, s0, False), (do, v, k, tr(s0), False), (v, do, q, tr(z), True), (k, q, do, z, True)]
    for got, want, (a, b, c, st, back) in zip([o, *out], [ref, *refs], args):
        # a sum's d + 64 terms lose less than 2^-126 times their other factors each
        floor = 2.0 ** -118 * tok.decay_scale(a, b, c, g, st, back)[1]
        _near_decayed(_flat(got), want, _decayed(a, b, c, g, None, st, back), dt, n, d, floor)
    # the head that keeps nothing knows the token itself alone, whose other factor is 0 here
    dq, dk, dv = (_flat(t)[0, -1] for t in out)
    assert (_flat(o)[0, -1, 3:] == 0).all() and (dq == 0).all() and (dk == 0).all() and (dv[:n - 3] == 0).all()


def test_steep_heads_take_large_values():
    """Values of 2^100 in heads that forget within a chunk: the same bits times 2^100."""
    g = [-1.0, -1.38, -1.4, -6.0, float("-inf")]
    x = _inputs(24, 1, len(g), 1, 150, 128, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(1, len(g), 1, 150, 128, 0)
    f = 2.0 ** 100
    y = {**x, **{c: x[c] * f for c in "vsoz"}}
    (o, s1), (o2, s2) = _attn(s, x), _attn(s, y)
    assert torch.equal(o * f, o2) and torch.equal(s1 * f, s2)
    # dV and dS_in are linear in dO and dS_out, dQ and dK are products with V and S_in as well
    (g1, d1), (g2, d2) = _backward(s, x), _backward(s, {**y, "v": x["v"], "s": x["s"]})
    assert all(torch.equal(a * f, b) for a, b in zip([*g1, d1], [*g2, d2]))


@pytest.mark.parametrize("n", [100, 2500])
@pytest.mark.parametrize("d", [64, 128])
def test_large_powers_of_two_pass_through(n, d):
    """Values and state beyond 2^70 in heads that carry a factor inside: the same bits times that power (sums
    here stay below 2^7 times it, under the 2^82 of the steepest of these heads)."""
    g = [-0.01, -0.3, -0.5, -0.7, -0.97]
    x = _inputs(25, 1, len(g), 1, n, d, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(1, len(g), 1, n, d, 0)
    f = 2.0 ** 74
    (o, s1), (o2, s2) = _attn(s, x), _attn(s, {**x, "v": x["v"] * f, "s": x["s"] * f})
    assert torch.equal(o * f, o2) and torch.equal(s1 * f, s2)
    (g1, d1), (g2, d2) = _backward(s, x), _backward(s, {**x, "o": x["o"] * f, "z": x["z"] * f})
    assert all(torch.equal(a * f, b) for a, b in zip([*g1, d1], [*g2, d2]))


@pytest.mark.parametrize("n", [100, 2500])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_empty_sequences_hand_their_state_on(n, dt):
    """Any float32 state, in every kind of head, forward and back, beside a sequence with tokens."""
    g = [0.0, -0.01, -0.5, -0.7, -0.97, -1.2, -6.0, float("-inf")]
    x = _inputs(26, 2, len(g), 1, n, 64, dt, names="qkvo", g=g)
    lens = [0, 70]
    for c in "sz":
        x[c][0] = torch.tensor([3.4e38, -1e30, 1e-30, 1e-42, 0.0, -2.5], device="cuda").repeat(len(g) * 64 * 64 // 6 + 1)[
            :len(g) * 64 * 64].view(len(g), 64, 64)
    s = vdn.make_shape(2, len(g), 1, n, 64, 0, in_dtype=dt)
    o, s1 = _attn(s, x, lens)
    out, ds = _backward(s, x, lens)
    assert torch.equal(s1[0], x["s"][0]) and torch.equal(ds[0], x["z"][0])
    assert all((t[0] == MARK).all() for t in (o, *out))


FAR = [
    # frame0, theta, scale
    (1 << 31, 10000.0, 1.0), ((1 << 40) + 12345, 256.0, 0.5), (1234567890123, 500000.0, 1.25), ((1 << 52) - 2, 10000.0, 1.0),
    (-(1 << 52), 10000.0, 0.1), (-(1 << 45) + 1, 1000.0, 100.0), (1 << 50, 1.0, 1.0), (1 << 52, 1e300, 1.0), (1 << 44, 0.5, 3.0),
]


@pytest.mark.parametrize("frame0,theta,scale", FAR)
@pytest.mark.parametrize("inter", [True, False])
def test_rotary_far_frames(frame0, theta, scale, inter):
    """Every frame that a call takes, against angles from 60 digits, with the bound of the near ones: the
    remainder of a turn, its sine and cosine and the two products in float32."""
    T, d, dim = 3, 64, 60
    r = np.random.default_rng(70)
    x = torch.from_numpy(r.standard_normal((1, 2, T, 1, d))).float().cuda()
    y = torch.empty_like(x)
    s = vdn.make_shape(1, 2, T, 1, d, 0, in_dtype="f32")
    vdn.vdn_rotary(s, vdn.rotary(dim, 2, 2, grid=(1, 1), interleaved=inter, frame0=frame0, theta=theta, scale=(scale, 1.0, 1.0)),
                   [x], [y])
    _far_near(x, y, tok.far_angles([frame0 + t for t in range(T)], dim, theta, scale), dim, inter)


def _far_near(x, y, ang, dim, inter):
    f, got = _flat(x)[..., :dim], _flat(y)[..., :dim]
    a, b = (f[..., 0::2], f[..., 1::2]) if inter else (f[..., :dim // 2], f[..., dim // 2:])
    c, s = np.cos(ang), np.sin(ang)
    u, v = a * c - b * s, a * s + b * c
    ref = np.stack([u, v], -1).reshape(f.shape) if inter else np.concatenate([u, v], -1)
    assert (np.abs(got - ref) <= 2.0 ** -24 * np.abs(ref) + 2.0 ** -20 * np.abs(f).max()).all()


@pytest.mark.parametrize("theta,scale", [(10000.0, 1.0), (256.0, 1000.0)])
def test_rotary_far_positions(theta, scale):
    """Given positions over the whole of int32."""
    d, pos = 32, [2 ** 31 - 1, -(2 ** 31), 123456789, -1, 2 ** 30 + 1]
    n = len(pos)
    r = np.random.default_rng(71)
    x = torch.from_numpy(r.standard_normal((1, 2, n, 1, d))).float().cuda()
    y = torch.empty_like(x)
    pt = torch.tensor([[[0, 0, p] for p in pos]], dtype=torch.int32, device="cuda")
    s = vdn.make_shape(1, 2, n, 1, d, 0, in_dtype="f32")
    vdn.vdn_rotary(s, vdn.rotary(0, 0, d, theta=theta, scale=(1.0, 1.0, scale), pos=pt), [x], [y])
    _far_near(x, y, tok.far_angles(pos, d, theta, scale), d, True)


@pytest.mark.parametrize("lens", [None, [300, 129]], ids=["whole", "ragged"])
@pytest.mark.parametrize("d,di,do", [(128, "bf16", "bf16"), (64, "bf16", "bf16"), (16, "bf16", "bf16"), (32, "f32", "f32"),
                                     (128, "f32", "f32"), (64, "bf16", "f32"), (32, "f32", "bf16")])
def test_decays_within_the_decayed_bound(d, di, do, lens):
    """Every kind of head against the bound whose state share decays with the tokens, small writes beside a
    start state of ordinary size, so that the state's share is what an output near it consists of."""
    g = [0.0, -1e-7, -1e-3, -0.05, -0.3, -0.65, -0.9, -1.1, -1.5, -5.0, -80.0, float("-inf")]
    B, n = 1 if lens is None else 2, 300
    x = _inputs(27 + d, B, len(g), 1, n, d, di, names="qkvo", g=g)
    x["v"] *= 2.0 ** -10
    x["o"] *= 2.0 ** -10
    s = vdn.make_shape(B, len(g), 1, n, d, 0, in_dtype=di, out_dtype=do)
    o, s1 = _attn(s, x, lens)
    q, k, v, do_ = (_flat(x[c]) for c in "qkvo")
    s0, z, g = _np(x["s"]), _np(x["z"]), np.array(g, np.float32).astype(np.float64)
    ref, ref_s = tok.decay_attn(q, k, v, g, lens, s0)
    keep = np.isfinite(ref)
    q, k, v, do_ = (np.where(keep, y, 0.0) for y in (q, k, v, do_))
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    cases = [(o, ref, (q, k, v, s0, False))]
    if di == do:
        out, ds = _backward(s, x, lens)
        *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do_, lens, s0, z)
        cases += list(zip(out, refs, [(do_, v, k, tr(s0), False), (v, do_, q, tr(z), True), (k, q, do_, z, True)]))
        for h in range(len(g)):
            assert np.linalg.norm(_np(ds)[:, h] - ref_ds[:, h]) <= 2e-6 * np.linalg.norm(ref_ds[:, h]) + 1e-36
    for h in range(len(g)):
        _state_near(_np(s1)[:, h], ref_s[:, h])
    for got, want, (a, b, c, st, back) in cases:
        floor = 2.0 ** -118 * tok.decay_scale(a, b, c, g, st, back)[1]
        _near_decayed(_flat(got), want, _decayed(a, b, c, g, lens, st, back), do, n, d, floor)


SEGMENTS = [
    # d, in, out, n, lens
    (16, "bf16", "bf16", 2500, [2500, 1317, 0]), (32, "bf16", "bf16", 2500, [2500, 64, 1]), (16, "f32", "f32", 1500, None),
    (16, "bf16", "f32", 1500, [1500, 700, 65]), (64, "bf16", "f32", 1500, None), (128, "bf16", "f32", 1000, [1000, 999, 0]),
    (32, "f32", "bf16", 1500, [3, 1500, 1000]), (128, "f32", "bf16", 1000, None),
]


@pytest.mark.parametrize("case", SEGMENTS, ids=str)
def test_segments_of_every_width_and_type(case):
    """Sequences long enough to be cut, whole and ragged; the backward pass where the types allow it."""
    d, di, do, n, lens = case
    B, H = 3, 2
    x = _inputs(28 + d, B, H, 1, n, d, di, names="qkvo", g=[-1e-3, -0.2])
    s = vdn.make_shape(B, H, 1, n, d, 0, in_dtype=di, out_dtype=do)
    assert vdn.vdn_decay_attn_workspace_bytes(s) > 0
    if lens:
        _poison(x, lens, "qkvo")
    o, s1 = _attn(s, x, lens)
    q, k, v, do_ = (_flat(x[c]) for c in "qkvo")
    g, s0, z = _np(x["g"]), _np(x["s"]), _np(x["z"])
    ref, ref_s = tok.decay_attn(q, k, v, g, lens, s0)
    keep = np.isfinite(ref)
    cases = [(o, ref, lambda: (q, k, v, s0, False))]
    _state_near(_np(s1), ref_s)
    if di == do:
        assert vdn.vdn_decay_attn_backward_workspace_bytes(s) > 0
        out, ds = _backward(s, x, lens)
        *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do_, lens, s0, z)
        tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
        cases += list(zip(out, refs, [lambda: (do_, v, k, tr(s0), False), lambda: (v, do_, q, tr(z), True),
                                      lambda: (k, q, do_, z, True)]))
        _state_near(_np(ds), ref_ds)
    q, k, v, do_ = (np.where(keep, y, 0.0) for y in (q, k, v, do_))
    for got, want, args in cases:
        a, b, c, st, back = args()
        _near_decayed(_flat(got), want, _decayed(a, b, c, g, lens, st, back), do, n, d, 0.0)
        assert (_flat(got)[~keep] == MARK).all()


@pytest.mark.parametrize("d", [32, 128])
def test_steep_heads_in_segments(d):
    """Cut sequences of heads that forget within a chunk, ragged, in the form with two powers and in the other."""
    g = [-0.99, -1.38, -1.42, -3.0]
    n, lens = 2500, [2500, 1331]
    x = _inputs(29, 2, len(g), 1, n, d, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(2, len(g), 1, n, d, 0)
    assert vdn.vdn_decay_attn_workspace_bytes(s) > 0
    _poison(x, lens, "qkvo")
    o, s1 = _attn(s, x, lens)
    out, ds = _backward(s, x, lens)
    q, k, v, do = (_flat(x[c]) for c in "qkvo")
    g, s0, z = _np(x["g"]), _np(x["s"]), _np(x["z"])
    ref, ref_s = tok.decay_attn(q, k, v, g, lens, s0)
    *refs, ref_ds = tok.decay_attn_backward(q, k, v, g, do, lens, s0, z)
    keep = np.isfinite(ref)
    q, k, v, do = (np.where(keep, y, 0.0) for y in (q, k, v, do))
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    for got, want, (a, b, c, st, back) in zip([o, *out], [ref, *refs], [
            (q, k, v, s0, False), (do, v, k, tr(s0), False), (v, do, q, tr(z), True), (k, q, do, z, True)]):
        floor = 2.0 ** -118 * tok.decay_scale(a, b, c, g, st, back)[1]
        _near_decayed(_flat(got), want, _decayed(a, b, c, g, lens, st, back), "bf16", n, d, floor)
        assert (_flat(got)[~keep] == MARK).all()
    _state_near(_np(s1), ref_s)
    _state_near(_np(ds), ref_ds)


@pytest.mark.parametrize("n,at", [(200, 100), (2500, 1500)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("name", ["q", "k", "v", "o"])
def test_how_far_a_nan_reaches(name, dt, n, at):
    """One value that is no number: the other heads, and of its own the chunks on the far side of either
    walk, come out as without it."""
    x = _inputs(30, 2, 2, 1, n, 64, dt, names="qkvo", g=[-0.01, -1.2])
    s = vdn.make_shape(2, 2, 1, n, 64, 0, in_dtype=dt)
    clean, (want, _) = _attn(s, x)[0], _backward(s, x)
    y = {**x, name: x[name].clone()}
    for h in range(2):
        y[name][1, h, 0, at, 5] = float("nan")
    o, (got, _) = _attn(s, y)[0], _backward(s, y)
    lo, hi = at // 64 * 64, at // 64 * 64 + 64
    for a, b, back in ((o, clean, False), (got[0], want[0], False), (got[1], want[1], True), (got[2], want[2], True)):
        assert torch.equal(a[0], b[0])
        far = slice(hi, n) if back else slice(0, lo)
        assert torch.equal(a[1][..., far, :], b[1][..., far, :])


@pytest.mark.parametrize("d,n,lens", [(16, 1, None), (128, 1, None), (16, 256, [256, 0]), (64, 70, None), (32, 300, [300, 129]),
                                      (128, 300, [300, 200]), (128, 1500, None), (64, 1500, [1500, 1337])], ids=str)
def test_bf16_outputs_are_off_by_their_own_rounding(d, n, lens):
    """Scores and the state's copy enter in two bf16 parts (2^-16 each), the weighted values in two that are
    cut off, and the product of the second parts is left out: 2^-14 of M_i and R_i together. The float32 sums
    of d + 64 terms and a few chunks' states: 2^-15 of A_i. The output's rounding, half a step, is what
    remains: the error's norm is that of the rounded definition's to 2 %, (2^-14 / 2^-9.2)^2 < 0.2 % of its
    square and twice the chance of a rounding that falls the other way."""
    g = [0.0, -1e-4, -0.01, -0.1, -0.5, -0.95, -1.2, -3.0]
    B = 1 if lens is None else 2
    x = _inputs(33 + d + n, B, len(g), 1, n, d, "bf16", names="qkvo", g=g)
    s = vdn.make_shape(B, len(g), 1, n, d, 0)
    o, _ = _attn(s, x, lens)
    out, _ = _backward(s, x, lens)
    q, k, v, do = (_flat(x[c]) for c in "qkvo")
    s0, z, g = _np(x["s"]), _np(x["z"]), np.array(g, np.float32).astype(np.float64)
    ref, _ = tok.decay_attn(q, k, v, g, lens, s0)
    *refs, _ = tok.decay_attn_backward(q, k, v, g, do, lens, s0, z)
    keep = np.isfinite(ref)
    q, k, v, do = (np.where(keep, y, 0.0) for y in (q, k, v, do))
    tr = lambda t: np.swapaxes(t, -1, -2)  # noqa: E731
    for got, want, (a, b, c, st, back) in zip([o, *out], [ref, *refs], [
            (q, k, v, s0, False), (do, v, k, tr(s0), False), (v, do, q, tr(z), True), (k, q, do, z, True)]):
        m, sums, reads = _decayed(a, b, c, g, lens, st, back)
        off = np.abs(_flat(got) - want)[keep]
        tol = (2.0 ** -8 * np.abs(want) + 2.0 ** -14 * (m + reads) + 2.0 ** -15 * sums)[keep]
        assert (off <= tol).all()
        rounded = _np(torch.from_numpy(np.nan_to_num(want)).to(torch.bfloat16))
        assert np.linalg.norm(off) <= 1.02 * np.linalg.norm((rounded - want)[keep])
