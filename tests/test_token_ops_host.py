"""The token-level operators without a GPU: their float64 definitions pinned
against explicit sums, finite differences and rotations, and the entry points'
refusals, which come before the device is touched."""
import ctypes

import numpy as np
import pytest

from frame_wise_delta_b200 import build, vdn
from oracle import token_ops as tok


@pytest.fixture(scope="module")
def L():
    build.build()
    return vdn.lib()


# ------------------------------------------------------------- definitions
def _draw(seed, B=2, H=3, n=9, d=4):
    r = np.random.default_rng(seed)
    q, k, v, do = (r.standard_normal((B, H, n, d)) for _ in range(4))
    g = -np.exp(r.uniform(-4, 1, H))
    g[0] = 0.0
    s, z = (r.standard_normal((B, H, d, d)) for _ in range(2))
    return q, k, v, do, g, s, z


def test_attention_is_the_decayed_sum():
    q, k, v, _, g, s, _ = _draw(1)
    o, s1 = tok.decay_attn(q, k, v, g, None, s)
    n = q.shape[2]
    for h in range(3):
        for i in range(n):
            want = np.exp(g[h] * (i + 1)) * np.einsum("bvk,bk->bv", s[:, h], q[:, h, i])
            for j in range(i + 1):
                want = want + np.exp(g[h] * (i - j)) * (q[:, h, i] * k[:, h, j]).sum(-1)[:, None] * v[:, h, j]
            np.testing.assert_allclose(o[:, h, i], want, rtol=1e-12, atol=1e-12)
    # cutting a sequence in two changes nothing
    o1, mid = tok.decay_attn(q[:, :, :4], k[:, :, :4], v[:, :, :4], g, None, s)
    o2, end = tok.decay_attn(q[:, :, 4:], k[:, :, 4:], v[:, :, 4:], g, None, mid)
    np.testing.assert_allclose(np.concatenate([o1, o2], 2), o, rtol=1e-12)
    np.testing.assert_allclose(end, s1, rtol=1e-12)


def test_state_reads_are_the_state_in_front():
    """With one token per chunk R_i is |l X_{i-1}| |q_i|; with one chunk it is the start state's share."""
    q, k, v, _, g, s, _ = _draw(5)
    r = tok.state_reads(q, k, v, g, None, s, chunk=1)
    for i in range(q.shape[2]):
        _, x = tok.decay_attn(q[:, :, :i], k[:, :, :i], v[:, :, :i], g, None, s)
        want = np.einsum("bhvk,bhk->bhv", np.abs(x) * np.exp(g)[None, :, None, None], np.abs(q[:, :, i]))
        np.testing.assert_allclose(r[:, :, i], want, rtol=1e-12)
    r = tok.state_reads(q, k, v, g, [9, 4], s, back=True)
    want = np.einsum("bhvk,bhk->bhv", np.abs(s), np.abs(q[:, :, 3]))
    np.testing.assert_allclose(r[1, :, 3], want[1], rtol=1e-12)
    assert (r[1, :, 4:] == 0).all()


def test_the_state_decays_in_the_scale():
    """Values of one sign: the scale is the output itself, walking forward and back, forgetting heads too."""
    q, k, v, do, g, s, z = (np.abs(x) for x in _draw(6))
    g = np.array([0.0, -3.0, -np.inf])
    lens = [9, 4]
    rows = np.arange(9)[None, None, :, None] < np.array(lens)[:, None, None, None]
    o, _ = tok.decay_attn(q, k, v, g, lens, s)
    _, a = tok.decayed_scale(q, k, v, g, lens, s)
    np.testing.assert_allclose(np.where(rows, a, 0), np.where(rows, o, 0), rtol=1e-12)
    _, _, dv, _ = tok.decay_attn_backward(q, k, v, g, do, lens, s, z)
    # dV walks back over (K, Q, dO): what lies behind a sequence's end is not part of it
    cut = lambda x: np.where(rows, x, 0)  # noqa: E731
    _, a = tok.decayed_scale(cut(k), cut(q), cut(do), g, lens, z, back=True)
    np.testing.assert_allclose(cut(a), cut(dv), rtol=1e-12)


def test_the_decayed_scale_sees_a_leak_of_the_state():
    """A head that forgets in a few tokens, with small writes: a share of 2^-13 of the start state in every
    output stays within the undecayed scale's slack and breaks the decayed one's, forward and back."""
    r = np.random.default_rng(7)
    q, k, v = (r.standard_normal((1, 1, 60, 16)) for _ in range(3))
    v *= 2.0 ** -13
    g, s = np.array([-5.0]), r.standard_normal((1, 1, 16, 16))
    for back in (False, True):
        leak = 2.0 ** -13 * np.abs(np.einsum("bhvk,bhik->bhiv", s, q))
        reads = tok.state_reads(q, k, v, g, None, s, back)
        (m, a), (m1, a1) = tok.decay_scale(q, k, v, g, s, back), tok.decayed_scale(q, k, v, g, None, s, back)
        np.testing.assert_array_equal(m, m1)
        far = slice(0, 50) if back else slice(10, 60)
        assert (leak <= 2.0 ** -13 * a)[:, :, far].all()
        tol = 2.0 ** -8 * (m1 + reads) + 2.0 ** -13 * a1
        assert (leak > 3 * tol)[:, :, far].mean() > 0.9


@pytest.mark.parametrize("lens", [None, [9, 4], [0, 1]])
def test_gradients_are_the_differences(lens):
    q, k, v, do, g, s, z = _draw(2)

    def loss(q, k, v, s):
        o, s1 = tok.decay_attn(q, k, v, g, lens, s)
        return np.nansum(o * do) + (s1 * z).sum()

    grads = tok.decay_attn_backward(q, k, v, g, do, lens, s, z)
    r = np.random.default_rng(3)
    args = [q, k, v, s]
    for which, grad in enumerate(grads):
        for _ in range(6):
            e = r.standard_normal(args[which].shape)
            up, dn = [x.copy() for x in args], [x.copy() for x in args]
            up[which] += 1e-6 * e
            dn[which] -= 1e-6 * e
            diff = (loss(*up) - loss(*dn)) / 2e-6
            # a rounding of the loss (2^-53 |loss|) over the step of 2e-6, and no
            # third-order term: the loss is cubic at most, linear in each argument
            assert abs(diff - np.nansum(grad * e)) < 1e-8 * max(1.0, abs(loss(*args)))


def test_rotary_turns_pairs():
    r = np.random.default_rng(4)
    x = r.standard_normal((1, 2, 6, 16))
    pos = tok.grid_positions(1, 2, 3, 5)
    for inter in (True, False):
        y = tok.rotary(x, pos, (4, 6, 2), 100.0, interleaved=inter)
        np.testing.assert_allclose(y[..., 12:], x[..., 12:])
        # lengths stay, the inverse undoes it
        np.testing.assert_allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        np.testing.assert_allclose(tok.rotary(y, pos, (4, 6, 2), 100.0, interleaved=inter, inverse=True), x, atol=1e-14)
        # products depend on the difference of positions alone
        z = tok.rotary(x, pos + 11, (4, 6, 2), 100.0, interleaved=inter)
        np.testing.assert_allclose(np.einsum("bhid,bhjd->bhij", y, y), np.einsum("bhid,bhjd->bhij", z, z), atol=1e-12)
    # one pair by hand: section of 4 channels, second pair, frame 5: 5 * 100^(-1/2) = 0.5
    y = tok.rotary(x, pos, (4, 0, 0), 100.0)
    c, s = np.cos(0.5), np.sin(0.5)
    np.testing.assert_allclose(y[0, 0, 0, 2], x[0, 0, 0, 2] * c - x[0, 0, 0, 3] * s)
    np.testing.assert_allclose(y[0, 0, 0, 3], x[0, 0, 0, 2] * s + x[0, 0, 0, 3] * c)


def test_far_angles():
    """Near positions as in float64; far ones by the sum of two nearer angles; whole turns by hand."""
    pos = np.array([0, 1, -7, 12345])
    a = tok.far_angles(pos, 12, 500.0, 0.75)
    want = pos[:, None] * 0.75 * 500.0 ** (-2.0 * np.arange(6) / 12)
    np.testing.assert_allclose(np.exp(1j * a), np.exp(1j * want), atol=1e-11)
    assert np.abs(a).max() <= np.pi
    far = tok.far_angles([2 ** 51 + 12345, 2 ** 51], 12, 500.0, 0.75)
    np.testing.assert_allclose(np.exp(1j * (far[0] - far[1])), np.exp(1j * a[3]), atol=1e-11)
    # the C library reduces by pi in full as well
    assert abs(np.sin(tok.far_angles([2 ** 52], 2, 1.0, 1.0)[0, 0]) - np.sin(2.0 ** 52)) < 1e-15


# ----------------------------------------------------------------- refusals
def _p(s):
    return ctypes.cast(ctypes.pointer(s), ctypes.c_void_p)


def _shape(**kw):
    base = dict(B=2, H=3, T=1, U=40, d=16, n_text=0, in_dtype="bf16")
    base.update(kw)
    return vdn.make_shape(**base)


def _attn(L, s, **kw):
    a = dict(Q=16, K=32, V=48, g=16, lens=None, S_in=None, O=64, S_out=None, ws=None, bytes=0, info=None)
    a.update(kw)
    return L.vdn_decay_attn(_p(s), *[a[x] for x in ("Q", "K", "V", "g", "lens", "S_in", "O", "S_out", "ws", "bytes", "info")],
                            None)


@pytest.mark.parametrize("kw,word", [
    (dict(Q=None), "Q is NULL"), (dict(K=8), "K is not 16-byte"), (dict(V=None), "V is NULL"), (dict(O=None), "O is NULL"),
    (dict(g=None), "log_decay is NULL"), (dict(g=4), "log_decay is not"), (dict(lens=2), "lens is not 4-byte"),
    (dict(S_in=8), "S_in is not"), (dict(S_out=24), "S_out is not"), (dict(info=2), "info is not"), (dict(O=16), "O is an input"),
    (dict(O=48), "O is an input"),
])
def test_attention_refusals(L, kw, word):
    assert _attn(L, _shape(), **kw) == vdn.VDN_ERR_INVALID
    assert word in vdn.vdn_last_error()


def test_attention_shapes_and_workspace(L):
    assert _attn(L, _shape(d=48)) == vdn.VDN_ERR_UNSUPPORTED
    assert _attn(L, _shape(T=65536, U=65536)) == vdn.VDN_ERR_UNSUPPORTED
    assert L.vdn_decay_attn(None, *[16] * 8, None, 0, None, None) == vdn.VDN_ERR_INVALID
    s = _shape(H=1, B=1, U=60000)
    need = vdn.vdn_decay_attn_workspace_bytes(s)
    assert need > 0 and need % 256 == 0
    assert _attn(L, s) == vdn.VDN_ERR_INVALID and "workspace is NULL" in vdn.vdn_last_error()
    assert _attn(L, s, ws=256, bytes=need - 1) == vdn.VDN_ERR_INVALID and "required" in vdn.vdn_last_error()
    assert _attn(L, s, ws=128, bytes=need) == vdn.VDN_ERR_INVALID and "256-byte" in vdn.vdn_last_error()
    # short sequences take none, and an empty problem touches nothing
    assert vdn.vdn_decay_attn_workspace_bytes(_shape()) == 0
    assert _attn(L, _shape(B=0), Q=None, K=None, V=None, O=None, g=None) == vdn.VDN_OK
    assert vdn.vdn_decay_attn_workspace_bytes(_shape(d=48)) == 0


def _back(L, s, **kw):
    a = dict(Q=16, K=32, V=48, g=16, lens=None, S_in=None, dO=64, dS_out=None, dQ=80, dK=96, dV=112, dS_in=None, ws=None,
             bytes=0, info=None)
    a.update(kw)
    return L.vdn_decay_attn_backward(_p(s), *a.values(), None)


@pytest.mark.parametrize("kw,word", [
    (dict(dO=None), "dO is NULL"), (dict(dK=None), "dK is NULL"), (dict(dQ=64), "dQ is an input"), (dict(dV=32), "dV is an input"),
    (dict(dK=80), "dQ and dK"), (dict(dS_in=128, S_in=128), "dS_in is an input"), (dict(dS_in=128, dS_out=128), "dS_in is an input"),
    (dict(dS_in=8), "dS_in is not"), (dict(dS_out=4), "dS_out is not"),
])
def test_backward_refusals(L, kw, word):
    assert _back(L, _shape(), **kw) == vdn.VDN_ERR_INVALID
    assert word in vdn.vdn_last_error()


def test_backward_needs_one_type(L):
    assert _back(L, _shape(out_dtype="f32")) == vdn.VDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,word", [
    (dict(Q=None), "Q is NULL"), (dict(S_in=None), "S_in is NULL"), (dict(S_out=None), "S_out is NULL"), (dict(O=16), "O is an input"),
    (dict(active=2), "active is not"),
])
def test_step_refusals(L, kw, word):
    a = dict(Q=16, K=32, V=48, g=16, active=None, S_in=64, O=80, S_out=64)
    a.update(kw)
    assert L.vdn_decay_step(_p(_shape(U=1)), *a.values(), None) == vdn.VDN_ERR_INVALID
    assert word in vdn.vdn_last_error()


def test_step_takes_one_token(L):
    assert L.vdn_decay_step(_p(_shape(U=2)), *[16] * 3, 16, None, 64, 80, 64, None) == vdn.VDN_ERR_INVALID
    assert "one token" in vdn.vdn_last_error()


def _rot(L, s, r=None, io=None, n=1, **kw):
    a = dict(dim_t=4, dim_h=4, dim_w=4, grid=(5, 8))
    a.update(kw)
    r = vdn.rotary(**a) if r is None else r
    if io is None:
        io = (vdn.vdn_rotary_io * 3)()
        for i in range(3):
            io[i].x, io[i].y, io[i].rotate = 1024 * (2 * i + 1), 1024 * (2 * i + 2), 1
            for f in (io[i].x_stride, io[i].y_stride):
                f[0], f[1], f[2] = s.H * s.T * s.U * s.dk, s.T * s.U * s.dk, s.dk
    return L.vdn_rotary(_p(s), ctypes.byref(r), ctypes.byref(io), n, None), io


@pytest.mark.parametrize("kw,word", [
    (dict(dim_t=3), "even"), (dict(dim_h=-2), "even"), (dict(dim_t=10), "exceed d"), (dict(grid=(5, 7)), "grid"),
    (dict(grid=(0, 0)), "grid"), (dict(theta=0.0), "theta"), (dict(theta=float("inf")), "theta"), (dict(scale=(1.0, float("nan"), 1.0)), "scale"),
    (dict(frame0=1 << 53), "frame0"), (dict(scale=(1e9, 1.0, 1.0)), "turns"), (dict(n=0), "n_io"), (dict(n=4), "n_io"),
])
def test_rotary_refusals(L, kw, word):
    st, _ = _rot(L, _shape(), **kw)
    assert st == vdn.VDN_ERR_INVALID
    assert word in vdn.vdn_last_error()


@pytest.mark.parametrize("field,value,word", [
    ("x", None, "io.x is NULL"), ("y", 8, "io.y is not"), ("x_stride", (-8, 640, 16), "strides"), ("x_stride", (1920, 644, 16), "strides"),
    ("y_stride", (1920, 640, 8), "overlap"), ("y_stride", (640, 640, 16), "overlap"), ("y_stride", (0, 640, 16), "overlap"),
    ("y_stride", (1 << 61, 640, 16), "stride too large"), ("rotate", 2, "rotate"), ("y", 3 * 1024, "another tensor"), ("y", 1024, "in place"),
])
def test_rotary_io_refusals(L, field, value, word):
    s = _shape()
    _, io = _rot(L, s, n=0)
    if field in ("x_stride", "y_stride"):
        getattr(io[0], field)[:] = value
    else:
        setattr(io[0], field, value)
    if word == "in place":
        io[0].x_stride[:] = (3840, 640, 16)
    st, _ = _rot(L, s, io=io, n=2)
    assert st == vdn.VDN_ERR_INVALID
    assert word in vdn.vdn_last_error()


def test_binding_checks_types_and_shapes(L):
    import torch
    with pytest.raises(vdn.VdnError):
        vdn.rotary(4, 4, 4, pos=torch.zeros(1, 3))
    with pytest.raises(vdn.VdnError):
        vdn._arg(torch.zeros(3), torch.float32, (2,), -1, "log_decay")
    with pytest.raises(vdn.VdnError):
        vdn._arg(torch.zeros(3), torch.float32, (3,), 0, "log_decay")  # a host tensor
    shape = (2, 3, 2, 20, 16)
    x = torch.zeros(2, 40, 3, 3, 16, dtype=torch.bfloat16)[:, :, 1].permute(0, 2, 1, 3).unflatten(2, (2, 20))
    assert vdn._rows(x, shape, torch.bfloat16, -1, "X")[1:] == (40 * 9 * 16, 16, 9 * 16)
    for bad in (x.transpose(2, 3).contiguous().transpose(2, 3), x.float(), x.transpose(0, 1)):
        with pytest.raises(vdn.VdnError):
            vdn._rows(bad, shape, torch.bfloat16, -1, "X")
    # the call packs three vdn_rotary_io as words
    assert ctypes.sizeof(vdn.vdn_rotary_io) == 9 * 8 and vdn.vdn_rotary_io.rotate.offset == 64


# ------------------------------------------------------- sizes of zero, binding
@pytest.mark.parametrize("kw", [dict(U=0), dict(T=3, U=0), dict(T=0), dict(B=0), dict(H=0), dict(T=0, U=0)])
@pytest.mark.parametrize("grid", [(5, 8), (0, 0), (0, 8)])
def test_rotary_of_no_tokens(L, kw, grid):
    """No tokens: nothing to turn, whatever the grid (one of zero tokens has no rows or no columns); with
    tokens the grid has to hold them."""
    import torch
    s = _shape(**kw)
    assert _rot(L, s, grid=grid)[0] == vdn.VDN_OK
    assert _rot(L, _shape(), grid=(0, 8))[0] == vdn.VDN_ERR_INVALID
    # the binding takes the tensors of such a call as they come
    shape = (s.B, s.H, s.T, s.U, s.dk)
    x = torch.empty(shape, dtype=torch.bfloat16)
    assert vdn._rows(x, shape, torch.bfloat16, -1, "X")[0] == 0


def test_info_is_a_word():
    """The kernels write 32 bits there: smaller and other words are refused, no word at all is none."""
    import torch
    assert vdn._word(None, -1) is None and vdn._word(4096, -1) == 4096
    t = torch.zeros(2, dtype=torch.int32)
    assert vdn._word(t, -1) == t.data_ptr() and vdn._word(t[1:], -1) == t.data_ptr() + 4
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(1), torch.zeros(1, dtype=torch.int64),
                torch.zeros(0, dtype=torch.int32), torch.zeros(1, dtype=torch.int16)):
        with pytest.raises(vdn.VdnError, match="info"):
            vdn._word(bad, -1)
    with pytest.raises(vdn.VdnError, match="info"):
        vdn._word(t, 0)  # a host tensor
