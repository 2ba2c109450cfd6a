"""fp64 references of the gated linear recurrence, the 8-bit checkpoints and the
norm and rotation of B and C -- TEST INFRASTRUCTURE, token by token or block
by block from the definitions; it shares no code with the CUDA library.

Gated linear recurrence, with s(v) = 1 / (1 + e^-v):
    a_t = exp(A s(r_t)),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t,  y_t = h_t
"""
from __future__ import annotations

import numpy as np

__all__ = ["glr", "glr_grad", "pack8", "unpack8", "norm_rotate", "norm_rotate_grad"]


def _s(v):
    return 1.0 / (1.0 + np.exp(-v))


def _spans(shape, cu):
    """(batch row, first token, end) of each sequence."""
    if cu is None:
        return [(b, 0, shape[1]) for b in range(shape[0])]
    return [(0, int(cu[j]), int(cu[j + 1])) for j in range(len(cu) - 1)]


def _parts(x, r, i, A):
    gate, inp = _s(r), _s(i)
    a = np.exp(A * gate)
    return gate, inp, a, np.sqrt(-np.expm1(2 * A * gate))


def glr(x, r, i, A, h0=None, cu=None):
    """(y [B,T,C], final [S,C], before [B,T,C]: the state before each token)."""
    x, r, i, A = (np.asarray(v, dtype=np.float64) for v in (x, r, i, A))
    _, inp, a, m = _parts(x, r, i, A)
    spans = _spans(x.shape, cu)
    y, before = np.zeros_like(x), np.zeros_like(x)
    final = np.zeros((len(spans), x.shape[2]))
    for s, (b, lo, hi) in enumerate(spans):
        h = np.zeros(x.shape[2]) if h0 is None else np.asarray(h0[s], dtype=np.float64)
        for t in range(lo, hi):
            before[b, t] = h
            h = a[b, t] * h + m[b, t] * inp[b, t] * x[b, t]
            y[b, t] = h
        final[s] = h
    return y, final, before


def glr_grad(x, r, i, A, dy, h0=None, dfinal=None, cu=None, kept=None, chunk=64):
    """Reverse mode of ``glr``: dict with dx, dr, di, dA, dh0.  With ``kept`` (the
    states before each token of the forward pass that was run), the state is
    taken from it at the first token of every ``chunk`` of a sequence and
    computed from x, r, i as given here in between."""
    x, r, i, A, dy = (np.asarray(v, dtype=np.float64) for v in (x, r, i, A, dy))
    gate, inp, a, m = _parts(x, r, i, A)
    spans = _spans(x.shape, cu)
    before = glr(x, r, i, A, h0, cu)[2] if kept is None else np.array(kept, dtype=np.float64)
    if kept is not None:
        for b, lo, hi in spans:
            for t in range(lo + 1, hi):
                if (t - lo) % chunk:
                    before[b, t] = a[b, t - 1] * before[b, t - 1] + m[b, t - 1] * inp[b, t - 1] * x[b, t - 1]
    dx, dr, di = np.zeros_like(x), np.zeros_like(x), np.zeros_like(x)
    dA, dh0 = np.zeros_like(A), np.zeros((len(spans), x.shape[2]))
    for s, (b, lo, hi) in enumerate(spans):
        k = np.zeros_like(A) if dfinal is None else np.asarray(dfinal[s], dtype=np.float64)
        for t in range(hi - 1, lo - 1, -1):
            at, mt, g, p = a[b, t], m[b, t], gate[b, t], inp[b, t]
            G = dy[b, t] + k
            # the root's derivative is 0 where the root is
            root = np.divide(at * at * p * x[b, t], mt, out=np.zeros_like(mt), where=mt > 0)
            dl = G * (at * before[b, t] - root)
            dx[b, t] = G * mt * p
            di[b, t] = G * mt * x[b, t] * p * (1 - p)
            dr[b, t] = dl * A * g * (1 - g)
            dA += dl * g
            k = at * G
        dh0[s] = k
    return dict(dx=dx, dr=dr, di=di, dA=dA, dh0=dh0)


def pack8(x, block=64):
    """(codes int64, exps int64) of an activation whose last axis is cut into
    blocks: the least exponent byte e from 1 to 248 with max < 127.5 * 2^(e - 127)
    (at 248 codes saturate at 127);
    255 (and codes 0) for a block that is not finite."""
    x = np.asarray(x, dtype=np.float64)
    n = -(-x.shape[-1] // block)
    codes = np.zeros(x.shape, dtype=np.int64)
    exps = np.zeros((*x.shape[:-1], n), dtype=np.int64)
    for at in np.ndindex(*exps.shape):
        part = x[at[:-1]][at[-1] * block: (at[-1] + 1) * block]
        if not np.all(np.isfinite(part)):
            exps[at] = 255
            continue
        e, top = 1, np.max(np.abs(part))
        while e < 248 and not top < 127.5 * 2.0 ** (e - 127):
            e += 1
        exps[at] = e
        codes[at[:-1]][at[-1] * block: (at[-1] + 1) * block] = np.clip(np.rint(part / 2.0 ** (e - 127)), -127, 127)
    return codes, exps


def unpack8(codes, exps, block=64):
    step = np.repeat(np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127)), block, axis=-1)
    return codes * step[..., : codes.shape[-1]]


def _pairs(rotary, interleaved):
    j = np.arange(rotary // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)


def _turn(z, angle, p, q):
    o = np.array(z, dtype=np.float64)
    c, s = np.cos(angle)[:, :, None, :], np.sin(angle)[:, :, None, :]
    o[..., p] = z[..., p] * c - z[..., q] * s
    o[..., q] = z[..., p] * s + z[..., q] * c
    return o


def norm_rotate(x, w, positions, inv_freq, eps, interleaved):
    """x [B,T,G,N] normed over N, times w (None: 1), rotated by position * inv_freq."""
    x = np.asarray(x, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return _turn(n if w is None else n * w, angle, *_pairs(2 * len(inv_freq), interleaved))


def norm_rotate_grad(do, x, w, positions, inv_freq, eps, interleaved):
    """(dx, dw) for the cotangent do of ``norm_rotate``."""
    x, do = np.asarray(x, dtype=np.float64), np.asarray(do, dtype=np.float64)
    w = np.ones(x.shape[-1]) if w is None else np.asarray(w, dtype=np.float64)
    angle = np.asarray(positions, dtype=np.float64)[..., None] * np.asarray(inv_freq, dtype=np.float64)
    dz = _turn(do, -angle, *_pairs(2 * len(inv_freq), interleaved))
    size = np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    d = dz * w
    dx = d / size - x * np.mean(d * x, axis=-1, keepdims=True) / size ** 3
    return dx, np.sum(dz * x / size, axis=(0, 1, 2))
