"""The gated linear recurrence over gates that do not change: a state that a closed
gate holds over tens of thousands of tokens, and one that a steady input builds
up.  Roundings of one sign, which random gates would average out, add up there.

With constant r, i, x and dy everything is a geometric sum, so the fp64 values are
closed forms: with l = A s(r), a = e^l,
    h_t = a^(t+1) h0 + u (a^(t+1) - 1) / (a - 1),
    G_t = dy (a^(T-t) - 1) / (a - 1) + a^(T-1-t) dfinal.

Tolerance, before the first run: 1e-5 of the largest magnitude, the header's, but
channel by channel, as the scales differ.  The gates' errors are below 2e-6 of l
(e^-r from an argument of up to 43 log2(e) = 62, half a step of which is 2^-19, and
three hardware functions), and a relative error e of l moves a^t by at most
e |l t| a^t <= 0.37 e and a geometric sum by at most e; inside a tile a state is
rounded at most 24 times (8 tokens, 8 warps, 8 more in their sums), 24 * 2^-24 = 1.5e-6.
dA's terms have one sign or cancel: 1e-5 of the sum of their magnitudes.  Where all of
a channel's values are below the smallest normal number (products e^-93), two steps
of 2^-149 a value: two products are rounded there.
"""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")

# A and r: decays of 1 - 1e-6 to 1 - 0.023 a token
RATES = [(-1e-6, 30.0), (-0.02, -10.0), (-0.2, -12.0), (-0.002, -4.0), (-1e-3, 30.0), (-1e-4, 30.0), (-1e-5, 30.0),
         (-0.04, 0.0), (-0.3, -2.5)]
# x, h0, dy, dfinal: a steady input from zero; a state that is only held; both
INPUTS = [(1.0, 0.0, 1.0, 0.0), (0.0, 1.0, 0.0, 1.0), (0.7, -3.0, -0.3, 2.0)]


def s(v):
    return 1.0 / (1.0 + np.exp(-v))


def problem(T, rates=RATES):
    """One channel for every pair of rates and inputs, i = 0.5 throughout: the numbers
    as the call sees them, in fp64 and on the device."""
    rows = np.array([(*a, *b) for b in INPUTS for a in rates], dtype=np.float32)
    A, r, x, h0, dy, df = (np.ascontiguousarray(c) for c in rows.T)
    i = np.full_like(A, 0.5)
    on = lambda v: torch.from_numpy(v).to(DEV)  # noqa: E731
    wide = lambda v: on(v).expand(1, T, len(A)).contiguous()  # noqa: E731
    dev = dict(x=wide(x), r=wide(r), i=wide(i), dy=wide(dy), A=on(A), h0=on(h0)[None], df=on(df)[None])
    return {k: v.astype(np.float64) for k, v in dict(A=A, r=r, i=i, x=x, h0=h0, dy=dy, df=df).items()}, dev


def exact(n, T, at):
    """The state after the tokens `at`, and the gradients there."""
    sr, si = s(n["r"]), s(n["i"])
    l, a = n["A"] * sr, np.exp(n["A"] * sr)
    m = np.sqrt(-np.expm1(2 * l))
    t = np.asarray(at, dtype=np.float64)[:, None]
    after = lambda k: np.exp(l * k) * n["h0"] + m * si * n["x"] * np.expm1(l * k) / np.expm1(l)  # noqa: E731
    G = n["dy"] * np.expm1(l * (T - t)) / np.expm1(l) + np.exp(l * (T - 1 - t)) * n["df"]
    dl = G * (a * after(t) - a * a * si * n["x"] / m)
    return dict(y=after(t + 1), before=after(t), dx=G * m * si, di=G * m * n["x"] * si * s(-n["i"]),
                dr=dl * l * s(-n["r"]), dinit=a * G, terms=dl * sr)


def close(got, want, what, top=None, values=1):
    """Channel by channel, along the first axis; each a sum of `values`."""
    got = got.double().cpu().numpy()
    top = np.abs(want).max(axis=0) if top is None else top
    worst = np.maximum(np.abs(got - want).max(axis=0) - values * 2.0 ** -148, 0) / np.where(top == 0, 1.0, top)
    assert (worst <= 1e-5).all(), f"{what}: {dict(zip(np.flatnonzero(worst > 1e-5), worst[worst > 1e-5]))}"


@pytest.mark.parametrize("T", [4096, 65536])
def test_constant_gates(T):
    n, p = problem(T)
    y, fin, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(p["dy"], saved, dfinal_state=p["df"], return_dinit_state=True)
    e = exact(n, T, range(T))
    close(y[0], e["y"], "y")
    close(fin, e["y"][-1:], "final", np.abs(e["y"]).max(axis=0))
    close(saved.chunk_states, e["before"][::64], "chunk_states", np.abs(e["y"]).max(axis=0))
    for k in ("dx", "dr", "di"):
        close(g[k][0], e[k], k)
    close(g["dinit_state"], e["dinit"][:1], "dinit")
    close(g["dA"][None], e["terms"].sum(axis=0)[None], "dA", np.abs(e["terms"]).sum(axis=0), values=T)
    assert binding.device_status() == 0


# a token's change far below a step of the state (2^-25 of it and less), for thousands of
# tiles, and states that come to rest where what a tile adds is what it takes
HELD = [(-2e-8, 30.0), (-1e-3, -33.0), (-1.7e-9, 30.0), (-6e-7, 1.0), (-1e-3, -20.0), (-1e-5, 30.0), (-1e-4, 30.0),
        (-5e-6, 2.0)]


@pytest.mark.parametrize("T", [65536, 1 << 20])
def test_states_that_hardly_change(T):
    """The changes of a tile add up, whatever a step of the state that they change."""
    n, p = problem(T, HELD)
    y, fin, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(p["dy"], saved, dfinal_state=p["df"], return_dinit_state=True)
    at = np.arange(0, T, 64)
    e = exact(n, T, at)
    close(y[0, ::64], e["y"], "y")
    close(saved.chunk_states, e["before"], "chunk_states")
    # (of the largest state: one that has decayed below 2^-126 rests on a multiple of 2^-149)
    close(fin, exact(n, T, [T - 1])["y"], "final", np.abs(e["y"]).max(axis=0))
    for k in ("dx", "dr", "di"):
        close(g[k][0, ::64], e[k], k)
    close(g["dinit_state"], e["dinit"][:1], "dinit", np.abs(e["dinit"]).max(axis=0))
    assert binding.device_status() == 0
