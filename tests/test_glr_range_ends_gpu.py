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
    return torch.from_numpy(np.array(a, dtype=np.float32, order="C")).to(DEV).to(dtype)


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


# tokens and the logarithm of all of their decays together
LENGTHS = [(1, 20.0), (1, 15.0), (1, 10.0), (1, 0.7), (2, 20.0), (3, 20.0), (9, 20.0), (17, 20.0), (70, 20.0),
           (70, 3.0), (200, 20.0), (1000, 20.0), (1000, 2.0)]


def vanishing(T, total):
    """Every token's decay e^(-total / T), by gates at different places; no input, so that
    nothing but what is left of the state (and of its cotangent) comes out."""
    r = np.array([0.0, 1.0, -1.0, 3.0, -4.0, 30.0, 0.5, -7.0], dtype=np.float32)
    A = (-total / T * (1 + np.exp(-r.astype(np.float64)))).astype(np.float32)
    rng = np.random.default_rng(T)
    h0, df = rng.standard_normal((2, 1, 8)).astype(np.float32)
    wide = lambda v: np.broadcast_to(v, (1, T, 8)).astype(np.float32)  # noqa: E731
    return A, wide(r), wide(0.5), wide(0.0), wide(0.0), h0, df


@pytest.mark.parametrize("T,total", LENGTHS)
def test_what_is_left_of_a_state(oracle, T, total):
    A, r, i, x, dy, h0, df = vanishing(T, total)
    v = [np.asarray(t, dtype=np.float64) for t in (x, r, i, A)]
    y, fin, saved = binding.glr_forward(on(x), on(r), on(i), on(A), init_state=on(h0), return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(on(dy), saved, dfinal_state=on(df), return_dinit_state=True)
    yr, fr, _ = oracle.glr(*v, h0)
    close(y, yr, "y")
    close(fin, fr, "final")
    gr = oracle.glr_grad(*v, dy.astype(np.float64), h0, df)
    close(g["dinit_state"], gr["dh0"], "dinit")
    # the reference's 1 - s(r) keeps 2^-53 of one only, 1e-3 of itself at r = 30; s(-r) is the same
    gate = 1 / (1 + np.exp(-v[1]))
    # the states that the backward pass forms again have a as 1 + (a - 1), off by 2^-25 of one:
    # that of the state before, or 2^-25 / a of what is left of it,
    # at every token, and 2^-25 once more for the product's own rounding
    rel = 1e-5 + (T - 1) * 2.0 ** -24 * np.exp(total / T)
    close(g["dr"], gr["dr"] / (1 - gate) * (gate * np.exp(-v[1])), "dr", rel)
    close(g["dA"][None], gr["dA"][None], "dA", rel)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("total", [0.3, 0.7, 5.0, 10.0, 15.0, 20.0])
def test_step_keeps_what_is_left_of_a_state(oracle, total, dtype):
    t = dict(bf16=torch.bfloat16, f32=torch.float32)[dtype]
    A, r, i, x, _, h0, _ = vanishing(1, total)
    r = host(on(r, t))
    state = on(h0)
    y = binding.glr_step(state, on(x[:, 0], t), on(r[:, 0], t), on(i[:, 0], t), on(A))
    _, fr, _ = oracle.glr(x, r, i, A, h0)
    close(state, fr, "state")
    close(y, fr, "y", rel=1e-5 + (2.0 ** -8 if dtype == "bf16" else 0.0))


def test_steep_and_flat_channels_side_by_side(oracle):
    """Decays from 1 - 1e-6 to e^-12 among the 64 channels of a tile, inputs and
    cotangents everywhere, in whole tiles and ragged ones."""
    B, T, C = 1, 333, 100
    rng = np.random.default_rng(5)
    A = -np.exp(np.linspace(np.log(1e-6), np.log(20.0), C)).astype(np.float32)
    rng.shuffle(A)
    x, r, i, dy = (rng.standard_normal((B, T, C)).astype(np.float32) for _ in range(4))
    h0, df = rng.standard_normal((2, B, C)).astype(np.float32)
    y, fin, saved = binding.glr_forward(on(x), on(r), on(i), on(A), init_state=on(h0), return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(on(dy), saved, dfinal_state=on(df), return_dinit_state=True)
    v = [np.asarray(t, dtype=np.float64) for t in (x, r, i, A)]
    yr, fr, _ = oracle.glr(*v, h0)
    gr = oracle.glr_grad(*v, dy.astype(np.float64), h0, df)
    close(y, yr, "y")
    assert np.abs(host(fin) - fr).max() <= 1e-5 * np.abs(yr).max()
    for k in ("dx", "dr", "di"):
        close(g[k], gr[k], k)
    assert np.abs(host(g["dinit_state"]) - gr["dh0"]).max() <= 1e-5 * np.abs(gr["dh0"]).max()


@pytest.mark.parametrize("neighbour", [-0.1, -30.0])
@pytest.mark.parametrize("rate", [1e-6, 0.3, 5.0])
def test_a_positive_rate_is_a_nan(rate, neighbour):
    """Whatever the rates beside it, forwards, backwards and in a step."""
    T, C = 70, 16
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    x, r, i, dy = torch.randn(4, 1, T, C, generator=gen, device=DEV)
    A = torch.full((C,), neighbour, device=DEV)
    A[3] = rate
    others = [c for c in range(C) if c != 3]
    y, fin, saved = binding.glr_forward(x, r, i, A, return_final_state=True, save="inputs")
    g = binding.glr_backward(dy, saved)
    state = torch.zeros(1, C, device=DEV)
    binding.glr_step(state, *(t[:, 0].contiguous() for t in (x, r, i)), A)
    for t in (y, fin, state, g["dx"], g["dr"], g["di"], g["dA"]):
        assert torch.isnan(t[..., 3]).all() and torch.isfinite(t[..., others]).all()


def test_sum_of_a_rate_over_a_long_sequence():
    """dA over 2^24 tokens whose terms are all of one sign and all but the same."""
    T, C = 1 << 24, 8
    one = torch.ones(1, T, C, device=DEV)
    A = on(np.linspace(-0.5, -0.05, C))
    y, saved = binding.glr_forward(one, 0 * one, one, A, save="inputs")
    dA = host(binding.glr_backward(one, saved)["dA"])
    # steady from a few hundred tokens on: h = u / (1 - a), G = dy / (1 - a); the first and
    # the last of them are a share of 1e-4 of the sum at most and are added one by one
    a, si = np.exp(host(A) / 2), 1 / (1 + np.exp(-1.0))
    u = np.sqrt(1 - a * a) * si
    edge = 2000
    t = np.arange(edge, dtype=np.float64)[:, None]
    h, G = u / (1 - a), 1 / (1 - a)
    rest = a * a * si / np.sqrt(1 - a * a)
    dl = G * (a * h - rest)
    first = G * (a * (h * (1 - a ** t)) - rest)
    last = G * (1 - a ** (t + 1)) * (a * h - rest)
    want = 0.5 * ((T - 2 * edge) * dl + first.sum(axis=0) + last.sum(axis=0))
    assert (np.abs(dA - want) <= 1e-5 * np.abs(want)).all(), dA / want - 1
