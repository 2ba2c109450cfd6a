"""The position rotation at far positions, by value: angles reduced on the host in
exact arithmetic, from the inverse frequencies as the call sees them.

Tolerance, before the first run: what the other tests of the rotation ask near the
origin.  4e-6 of the largest value, and half a step (2^-8) more in bf16: the
angle's fraction of a turn is rounded once, 2^-25 of a turn.
"""
from fractions import Fraction

import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
# pi to 60 digits
PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494")
POSITIONS = [3, -(1 << 20) - 1, (1 << 33) + 7, -(1 << 33), (1 << 40) + 12345, -(1 << 47) + 3, (1 << 50) + 11,
             (1 << 53) - 1, -(1 << 53), 1 << 53]


def reduced(positions, freqs):
    """positions * freqs, less whole turns, in fp64."""
    out = np.empty((len(positions), len(freqs)))
    for a, p in enumerate(positions):
        for b, f in enumerate(freqs):
            angle = Fraction(int(p)) * Fraction(float(f))
            out[a, b] = float(angle - 2 * PI * round(angle / (2 * PI)))
    return out


def turned(x, angle, interleaved):
    n, half = x.shape[-1], angle.shape[-1]
    p, q = (np.arange(half) * 2, np.arange(half) * 2 + 1) if interleaved else (np.arange(half), np.arange(half) + half)
    c, s = np.cos(angle)[None, :, None], np.sin(angle)[None, :, None]
    o = x.copy()
    o[..., p], o[..., q] = x[..., p] * c - x[..., q] * s, x[..., p] * s + x[..., q] * c
    return o


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n,rotary", [(64, 32), (30, 10)])
def test_far_positions_by_value(n, rotary, interleaved, dtype):
    T, half = len(POSITIONS), rotary // 2
    gen = torch.Generator(device=DEV)
    gen.manual_seed(n)
    rnd = lambda: torch.randn(1, T, 2, n, generator=gen, device=DEV).to(dtype)  # noqa: E731
    B, C, dB, dC = rnd(), rnd(), rnd(), rnd()
    pos = torch.tensor(POSITIONS, device=DEV)[None]
    freq = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float32) / half)
    Bo, Co = binding.norm_rotate(B, C, pos, freq, interleaved=interleaved)
    g = binding.norm_rotate_backward(dB, dC, B, C, pos, freq, interleaved=interleaved)
    angle = reduced(POSITIONS, freq.double().cpu().numpy())
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 0.0
    for out, x, dx, do in ((Bo, B, g["dB"], dB), (Co, C, g["dC"], dC)):
        x, do = x.double().cpu().numpy(), do.double().cpu().numpy()
        size = np.sqrt((x * x).mean(axis=-1, keepdims=True) + 1e-5)
        want = turned(x / size, angle, interleaved)
        d = turned(do, -angle, interleaved)
        grad = d / size - x * (d * x).mean(axis=-1, keepdims=True) / size ** 3
        for got, w in ((out, want), (dx, grad)):
            got = got.double().cpu().numpy()
            for t in range(T):
                bad = np.abs(got[0, t] - w[0, t]) > rel * np.abs(w[0, t]) + 4e-6 * np.abs(w).max()
                assert not bad.any(), (POSITIONS[t], np.abs(got[0, t] - w[0, t]).max())
