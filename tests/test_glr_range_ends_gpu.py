"""The gated linear recurrence at the ends of its decays' range, channel by channel:
rates so small that 1 - a^2 is below the smallest normal number, decays far
below one, and products of decays that all but vanish.

Tolerance, before the first run: 1e-5 of a channel's largest magnitude.  A decay
e^l carries |l| times the relative error of l (the gate's: three hardware
functions, 3e-7) and an exponential's argument rounded to 2^-24 of itself; the
decays here multiply to e^-20 at most, so 20 * 4e-7 = 8e-6 bounds them.
"""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def host(t):
    return t.double().cpu().numpy()


def on(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DEV).to(dtype)


def close(got, want, what, rel=1e-5):
    """Channel by channel (the last axis)."""
    got, want = host(got).reshape(-1, want.shape[-1]), want.reshape(-1, want.shape[-1])
    top = np.abs(want).max(axis=0)
    off = np.abs(got - want).max(axis=0)
    bad = np.flatnonzero(~(off <= rel * top))
    assert bad.size == 0, f"{what}: channels {bad}: {off[bad] / np.where(top[bad] == 0, 1, top[bad])}"


@pytest.mark.parametrize("total", [86.0, 88.0, 100.0, 1e4])
def test_nothing_is_left_of_a_large_state(oracle, total):
    """A state of 1e6 that a tile's decays take to nothing leaves no trace in what small
    inputs build up: a step of 1e6 is larger than that."""
    T, C = 130, 8
    rng = np.random.default_rng(3)
    A = np.full(C, -2 * total / 64, dtype=np.float32)
    x = (1e-3 * rng.standard_normal((1, T, C))).astype(np.float32)
    zero = np.zeros((1, T, C), dtype=np.float32)
    dy = (1e-3 * rng.standard_normal((1, T, C))).astype(np.float32)
    h0, df = 1e6 * np.sign(rng.standard_normal((2, 1, C))).astype(np.float32)
    y, fin, saved = binding.glr_forward(on(x), on(zero), on(zero), on(A), init_state=on(h0), return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(on(dy), saved, dfinal_state=on(df), return_dinit_state=True)
    v = [np.asarray(t, dtype=np.float64) for t in (x, zero, zero, A)]
    yr, fr, before = oracle.glr(*v, h0)
    gr = oracle.glr_grad(*v, dy.astype(np.float64), h0, df)
    # of what the inputs and cotangents of a tile build up: about 1e-3
    assert np.abs(host(saved.chunk_states)[1:] - before[0, 64::64]).max() <= 1e-5 * 1e-3
    assert np.abs(host(fin) - fr).max() <= 1e-5 * 1e-3
    assert np.abs(host(g["dinit_state"]) - gr["dh0"]).max() <= 1e-5 * 1e-3
    assert np.abs(host(y)[0, 64:] - yr[0, 64:]).max() <= 1e-5 * 1e-3


def tiny(T):
    """Rates whose 1 - a^2 is subnormal or 0, closed and half-open gates; a usual one."""
    A = np.array([-1e-20, -1e-20, -1e-39, -1e-39, -1e-45, 0.0, -1e-37, -0.1], dtype=np.float32)
    r = np.array([-45.0, 0.0, 0.0, 30.0, 0.0, 0.0, -2.0, 0.0], dtype=np.float32)
    rng = np.random.default_rng(T)
    x, dy, h0 = (rng.standard_normal((1, n, 8)).astype(np.float32) for n in (T, T, 1))
    return A, np.broadcast_to(r, (1, T, 8)), np.full((1, T, 8), 0.25, dtype=np.float32), x, dy, h0[0]


@pytest.mark.parametrize("T", [1, 5, 130])
@pytest.mark.parametrize("save", ["inputs", "packed8"])
def test_rates_below_the_normal_numbers(oracle, T, save):
    A, r, i, x, dy, h0 = tiny(T)
    y, saved = binding.glr_forward(on(x), on(r), on(i), on(A), init_state=on(h0), save=save)
    g = binding.glr_backward(on(dy), saved, return_dinit_state=True)
    assert all(torch.isfinite(g[k]).all() for k in ("dx", "dr", "di", "dA", "dinit_state"))
    if save == "packed8":
        x, r, i = (oracle.unpack8(*oracle.pack8(v)) for v in (x, r, i))
    # the reference's root is below 1e-18 there: what it scales vanishes beside x and dy
    flat = [0, 2, 3, 4, 5]
    for k in ("dx", "di", "dr"):
        assert g[k][..., flat].abs().max() <= 1e-15 * T * np.abs(dy).max() * np.abs(x).max()
    v = [np.asarray(t, dtype=np.float64) for t in (x, r, i, A, dy, h0)]
    kept = oracle.glr(*v[:4], v[5])[2]
    # a rate that is 0: the root's derivative is taken as 0, dl = G a h
    G = np.cumsum(v[4][0, ::-1], axis=0)[::-1]
    gate = 1 / (1 + np.exp(-np.maximum(v[1][0], -43.0)))
    zero = [2, 3, 4, 5]  # A of 1e-39 and below
    want = (G * v[5] * gate).sum(axis=0)[zero]
    terms = np.abs(G * v[5] * gate).sum(axis=0)[zero]
    if save == "inputs":
        assert (np.abs(host(g["dA"])[zero] - want) <= 1e-5 * terms).all()
    close(y[..., flat], np.broadcast_to(v[5], (1, T, 8))[..., flat], "y")
    if save == "inputs":
        gr = oracle.glr_grad(*v[:5], v[5], kept=kept)
        close(g["dx"][..., 6:], gr["dx"][..., 6:], "dx")
        # dl = G (a h - a^2 s(i) x / m): 1e-5 of the two terms, which all but cancel in the
        # last channel at T = 1 (0.95763 and 0.95824)
        gate, inp = 1 / (1 + np.exp(-v[1])), 1 / (1 + np.exp(-v[2]))
        a = np.exp(v[3] * gate)
        with np.errstate(divide="ignore", invalid="ignore"):
            m = np.sqrt(-np.expm1(2 * v[3] * gate))
            G = gr["dx"] / (m * inp)
            terms = np.abs(G * v[3] * gate * (1 - gate)) * (np.abs(a * kept) + np.abs(a * a * inp * v[0] / m))
        off = np.abs(host(g["dr"]) - gr["dr"])
        assert (off[0, :, 6:].max(axis=0) <= 1e-5 * terms[0, :, 6:].max(axis=0)).all()
