"""Pins of the fp64 references of the gated linear recurrence, the 8-bit
checkpoints and the norm and rotation (CPU only): gradients against central
differences of the forward references, the forward ones against a second
writing of the definition."""
import numpy as np
import pytest

STEP = 1e-6


def differences(f, v):
    g = np.zeros_like(v)
    for at in np.ndindex(*v.shape):
        keep = v[at]
        v[at] = keep + STEP
        up = f()
        v[at] = keep - STEP
        g[at] = (up - f()) / (2 * STEP)
        v[at] = keep
    return g


def close(a, b):
    # central differences: STEP^2 of the third derivative plus 1e-16 / STEP of the
    # sum (values of about 10): 1e-8 here
    np.testing.assert_allclose(a, b, rtol=1e-6, atol=2e-8)


@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4, 9]])
def test_glr_gradients_against_differences(oracle, cu):
    rng = np.random.default_rng(1)
    shape = (1, 9, 3) if cu else (2, 5, 3)
    S = len(cu) - 1 if cu else 2
    v = {k: rng.standard_normal(shape) for k in "xri"}
    v["A"] = -np.abs(rng.standard_normal(3)) - 0.05
    v["h0"] = rng.standard_normal((S, 3))
    dy, df = rng.standard_normal(shape), rng.standard_normal((S, 3))

    def loss():
        y, fin, _ = oracle.glr(v["x"], v["r"], v["i"], v["A"], v["h0"], cu)
        return float(np.sum(y * dy) + np.sum(fin * df))

    g = oracle.glr_grad(v["x"], v["r"], v["i"], v["A"], dy, v["h0"], df, cu)
    for k, d in (("x", "dx"), ("r", "dr"), ("i", "di"), ("A", "dA"), ("h0", "dh0")):
        close(g[d], differences(loss, v[k]))


def test_glr_against_the_sum_over_sources(oracle):
    """h_t as the sum over tokens of the decays since, times what each brought in."""
    rng = np.random.default_rng(2)
    x, r, i = (rng.standard_normal((1, 6, 2)) for _ in range(3))
    A, h0 = np.array([-0.3, -2.0]), rng.standard_normal((1, 2))
    y, fin, before = oracle.glr(x, r, i, A, h0)
    a = np.exp(A / (1 + np.exp(-r[0])))
    u = np.sqrt(1 - a * a) / (1 + np.exp(-i[0])) * x[0]
    for t in range(6):
        want = np.prod(a[: t + 1], axis=0) * h0[0]
        for s in range(t + 1):
            want = want + np.prod(a[s + 1: t + 1], axis=0) * u[s]
        np.testing.assert_allclose(y[0, t], want, rtol=1e-12)
    np.testing.assert_array_equal(fin[0], y[0, -1])
    np.testing.assert_array_equal(before[0, 1:], y[0, :-1])


def test_glr_kept_states_of_the_same_inputs_change_nothing(oracle):
    rng = np.random.default_rng(3)
    x, r, i, dy = (rng.standard_normal((1, 9, 2)) for _ in range(4))
    A = np.array([-0.3, -2.0])
    kept = oracle.glr(x, r, i, A)[2]
    a, b = oracle.glr_grad(x, r, i, A, dy), oracle.glr_grad(x, r, i, A, dy, kept=kept, chunk=4)
    for k in a:
        np.testing.assert_allclose(a[k], b[k], rtol=1e-12, atol=1e-14)


def test_pack8(oracle):
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 70)) * np.exp(3 * rng.standard_normal((3, 1)))
    x[0, :64] = 0
    x[1, 65] = np.inf
    x[2, 0], x[2, 1:64] = 127.5, 1.0  # exactly 127.5 takes the next step
    x[2, 64:] = [127.49, -63.5, 0.5, 1.5, 2.5, -0.5]
    codes, exps = oracle.pack8(x)
    back = oracle.unpack8(codes, exps)
    assert exps[0, 0] == 1 and not codes[0, :64].any()
    assert exps[1, 1] == 255 and np.isnan(back[1, 64:]).all()
    assert exps[2, 0] == 128 and codes[2, 0] == 64 and codes[2, 1] == 0
    assert exps[2, 1] == 127 and list(codes[2, 64:]) == [127, -64, 0, 2, 2, 0]
    assert np.abs(codes).max() <= 127
    ok = np.isfinite(x) & np.isfinite(back)
    tops = np.repeat(np.stack([np.abs(x[:, :64]).max(1), np.abs(x[:, 64:]).max(1)], 1), 64, axis=1)[:, :70]
    assert (np.abs(x - back)[ok] <= np.maximum(tops[ok] / 127.5, 2.0 ** -127)).all()


@pytest.mark.parametrize("rotary,interleaved", [(0, False), (4, False), (6, True), (2, True)])
def test_norm_rotate(oracle, rotary, interleaved):
    rng = np.random.default_rng(5)
    x, do = rng.standard_normal((2, 3, 2, 6)), rng.standard_normal((2, 3, 2, 6))
    w, pos = rng.standard_normal(6), rng.integers(-50, 50, (2, 3))
    freq = 1.0 / 10.0 ** np.arange(rotary // 2)
    args = (pos, freq, 1e-3, interleaved)
    o = oracle.norm_rotate(x, w, *args)
    # as complex numbers
    n = x / np.sqrt((x ** 2).sum(-1, keepdims=True) / 6 + 1e-3) * w
    for j in range(rotary // 2):
        p, q = (2 * j, 2 * j + 1) if interleaved else (j, j + rotary // 2)
        z = (n[..., p] + 1j * n[..., q]) * np.exp(1j * pos * freq[j])[..., None]
        np.testing.assert_allclose(o[..., p], z.real, atol=1e-13)
        np.testing.assert_allclose(o[..., q], z.imag, atol=1e-13)
    np.testing.assert_allclose(o[..., rotary:], n[..., rotary:], atol=1e-13)

    def loss():
        return float(np.sum(oracle.norm_rotate(x, w, *args) * do))

    dx, dw = oracle.norm_rotate_grad(do, x, w, *args)
    close(dx, differences(loss, x))
    close(dw, differences(loss, w))
    # a planted mistake is seen: the angle's sign left as it was
    wrong = oracle.norm_rotate_grad(do, x, w, -pos, *args[1:])[0]
    assert rotary == 0 or np.abs(wrong - dx).max() > 1e-3
