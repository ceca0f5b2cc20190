"""Plain float64 definitions of the token-level operators (rotary positions,
decay attention, its gradients), one token at a time. Arrays are [B, H, n, d];
states [B, H, d_v, d_k]; `lens` holds the tokens of each sequence or is None."""
from __future__ import annotations

from decimal import Decimal, localcontext

import numpy as np


def _lens(lens, B, n):
    return [n] * B if lens is None else [min(max(int(x), 0), n) for x in lens]


def decay_attn(q, k, v, log_decay, lens=None, s_in=None):
    """S_i = exp(g) S_{i-1} + v_i k_i^T, o_i = S_i q_i. Rows behind a
    sequence's end are NaN (they are nobody's business). Returns (o, S)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, n, d = q.shape
    lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    o = np.full(v.shape, np.nan)
    s = np.zeros((B, H, d, d)) if s_in is None else np.array(s_in, np.float64)
    for b, length in enumerate(_lens(lens, B, n)):
        for i in range(length):
            s[b] = lam * s[b] + v[b, :, i, :, None] * k[b, :, i, None, :]
            o[b, :, i] = np.einsum("hvk,hk->hv", s[b], q[b, :, i])
    return o, s


def decay_attn_backward(q, k, v, log_decay, do, lens=None, s_in=None, ds_out=None):
    """Gradients of sum(o do) + sum(S ds_out): (dq, dk, dv, ds_in)."""
    q, k, v, do = (np.asarray(x, np.float64) for x in (q, k, v, do))
    B, H, n, d = q.shape
    lam = np.exp(np.asarray(log_decay, np.float64))[:, None, None]
    dq, dk, dv = (np.full(v.shape, np.nan) for _ in range(3))
    s = np.zeros((B, H, d, d)) if s_in is None else np.array(s_in, np.float64)
    z = np.zeros((B, H, d, d)) if ds_out is None else np.array(ds_out, np.float64)
    for b, length in enumerate(_lens(lens, B, n)):
        for i in range(length):
            s[b] = lam * s[b] + v[b, :, i, :, None] * k[b, :, i, None, :]
            dq[b, :, i] = np.einsum("hvk,hv->hk", s[b], do[b, :, i])
        for i in range(length - 1, -1, -1):
            z[b] = z[b] + do[b, :, i, :, None] * q[b, :, i, None, :]
            dk[b, :, i] = np.einsum("hvk,hv->hk", z[b], v[b, :, i])
            dv[b, :, i] = np.einsum("hvk,hk->hv", z[b], k[b, :, i])
            z[b] = lam * z[b]
    return dq, dk, dv, z


def decay_scale(q, k, v, log_decay, s_in=None, back=False, z=None):
    """Two sizes that bound rounding errors of one operator's outputs o_i:
    M_i = sum_j l^|i-j| |q_i . k_j| |v_j| over the tokens of the sum, and A_i,
    the same with |q_i| . |k_j| and the carried state's |S| |q_i| as well."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    n = q.shape[2]
    g = np.asarray(log_decay, np.float64)[None, :, None, None]
    i = np.arange(n)
    gap = (i[None, :] - i[:, None]) if back else (i[:, None] - i[None, :])
    with np.errstate(invalid="ignore"):
        w = np.where(gap > 0, np.exp(g * np.maximum(gap, 1)), gap == 0)
    m = (np.abs(q @ np.swapaxes(k, -1, -2)) * w) @ np.abs(v)
    a = ((np.abs(q) @ np.swapaxes(np.abs(k), -1, -2)) * w) @ np.abs(v)
    if s_in is not None:
        a = a + np.abs(q) @ np.swapaxes(np.abs(np.asarray(s_in, np.float64)), -1, -2)
    return m, a


def decayed_scale(q, k, v, log_decay, lens=None, s_in=None, back=False):
    """decay_scale with the carried state's share decayed as it is in the output:
    A_i takes l^(i+1) |S| |q_i|, on the walk back l^(len-1-i) |S| |q_i|."""
    m, a = decay_scale(q, k, v, log_decay, None, back)
    if s_in is not None:
        q = np.asarray(q, np.float64)
        B, n = q.shape[0], q.shape[2]
        i = np.arange(n)[None, :]
        e = np.array(_lens(lens, B, n))[:, None] - 1 - i if back else np.broadcast_to(i + 1, (B, n))
        g = np.asarray(log_decay, np.float64)[None, :, None]
        with np.errstate(invalid="ignore"):
            w = np.where(e[:, None] > 0, np.exp(g * np.maximum(e[:, None], 1)), e[:, None] == 0)
        a = a + w[..., None] * (np.abs(q) @ np.swapaxes(np.abs(np.asarray(s_in, np.float64)), -1, -2))
    return m, a


def state_reads(q, k, v, log_decay, lens=None, s_in=None, back=False, chunk=64):
    """R_i = sum_k |X_vk| |q_ik|, X the state in front of token i's chunk (on the
    walk back: behind it) with its decay up to token i: what a relative error of
    that state's values can make of o_i."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    B, H, n, d = q.shape
    g = np.asarray(log_decay, np.float64)

    def power(e):
        return np.where(e == 0, 1.0, np.exp(g * max(e, 1)))[:, None, None]

    r = np.zeros(v.shape)
    for b, length in enumerate(_lens(lens, B, n)):
        x = np.zeros((H, d, d)) if s_in is None else np.array(s_in[b], np.float64)
        starts = list(range(0, length, chunk))
        for a in starts[::-1] if back else starts:
            e = min(a + chunk, length)
            for i in range(a, e):
                f = power(e - 1 - i if back else i - a + 1)
                r[b, :, i] = np.einsum("hvk,hk->hv", np.abs(x) * f, np.abs(q[b, :, i]))
            x = power(e - a) * x
            for j in range(a, e):
                x = x + power(j - a + 1 if back else e - 1 - j) * v[b, :, j, :, None] * k[b, :, j, None, :]
    return r


def far_angles(pos, dim, theta, scale):
    """pos * scale * theta^(-2 i / dim) less whole turns, [n, dim / 2], from 60 digits: whole numbers of any size."""
    with localcontext() as c:
        c.prec = 60
        turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803483")
        out = np.empty((len(pos), dim // 2))
        for i in range(dim // 2):
            step = Decimal(scale) * Decimal(theta) ** (Decimal(-2 * i) / dim)
            for j, x in enumerate(pos):
                a = Decimal(int(x)) * step
                out[j, i] = a - (a / turn).to_integral_value() * turn
    return out


def rotary(x, pos, dims, theta, scale=(1.0, 1.0, 1.0), interleaved=True, inverse=False):
    """x [B, H, n, d] turned at pos [B or 1, n, 3], each pair as a complex number."""
    y = np.array(x, np.float64)
    at = 0
    for axis, dim in enumerate(dims):
        half = dim // 2
        if half:
            i = np.arange(half)
            a, b = (at + 2 * i, at + 2 * i + 1) if interleaved else (at + i, at + half + i)
            ang = (np.asarray(pos, np.float64)[..., axis] * scale[axis])[:, None, :, None] * theta ** (-2.0 * i / dim)
            z = (y[..., a] + 1j * y[..., b]) * np.exp((-1j if inverse else 1j) * ang)
            y[..., a], y[..., b] = z.real, z.imag
        at += dim
    return y


def grid_positions(T, gh, gw, frame0=0):
    """[1, T * gh * gw, 3]: (frame, row, column) of every token."""
    t, r, c = np.meshgrid(np.arange(T) + frame0, np.arange(gh), np.arange(gw), indexing="ij")
    return np.stack([t, r, c], -1).reshape(1, -1, 3).astype(np.float64)
