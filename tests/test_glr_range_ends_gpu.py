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
