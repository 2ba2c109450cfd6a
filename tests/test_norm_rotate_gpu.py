"""GPU parity of the norm and rotation of B and C against the fp64 reference.

Tolerances, before the first run.  An fp32 value is a product of x, rstd (2 ulp),
a weight and a sine or cosine (fp32 storage: a few ulp; the angle's fraction is
rounded once, 2^-25 of a turn, 2e-7 rad), two products added: below 1e-6 of the
row's largest value; 4e-6 is asked.  bf16 storage takes the hardware's sine and
cosine (2^-20): 4e-6 too, plus half a step, eps / 2 = 2^-8 of each value.  The
weights' gradients sum tokens * G terms: 2e-5 of the largest.  dv is the
difference rstd d - rstd x (rstd^2 mean(d x)); by Cauchy-Schwarz the second term
is at most rstd max|d| sqrt(N) in a value, and with one value a row (N = 1) the two
cancel but for a share eps / (v^2 + eps) of either.  Their roundings are
relative to themselves, 2^-24 times the handful of operations that formed
them, whatever is left of the difference: 4e-6 is of the largest rstd |d| there.
"""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def host(t):
    return t.double().cpu().numpy()


def close(got, want, dtype=torch.float32, rel=4e-6, what="", top=0.0):
    got = host(got)
    half = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0
    bad = np.abs(got - want) > rel * max(top, np.max(np.abs(want))) + half * np.abs(want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3e}"


def problem(b, t, g, n, rotary, dtype, seed=0, layout="own", far=False):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV)  # noqa: E731
    ty = TYPES[dtype]
    if layout == "own":
        B, C = (3 * rnd(b, t, g, n)).to(ty), (0.1 * rnd(b, t, g, n)).to(ty)
    else:  # slices of a projection's rows, behind `layout` other values
        rows = rnd(b, t, layout + 2 * g * n).to(ty)
        B = rows[..., layout: layout + g * n].unflatten(-1, (g, n))
        C = rows[..., layout + g * n:].unflatten(-1, (g, n))
    pos = torch.randint(-5, 1 << 20 if far else 4096, (b, t), generator=gen, device=DEV)
    freq = 10000.0 ** (-torch.arange(rotary // 2, device=DEV, dtype=torch.float32) / max(1, rotary // 2))
    return dict(B=B, C=C, pos=pos, freq=freq, wB=1 + 0.3 * rnd(n), wC=1 + 0.3 * rnd(n),
                dB=rnd(b, t, g, n).to(ty), dC=rnd(b, t, g, n).to(ty))


# (batch, seqlen, groups, dstate, rotary, layout): vectors and single values, one
# token and many, rotary none, part and all, odd sizes, slices on and off a vector's alignment
CASES = [(1, 1, 1, 128, 128, "own"), (2, 33, 3, 64, 32, 8), (1, 100, 2, 96, 64, "own"), (3, 5, 1, 256, 256, 16),
         (1, 7, 5, 8, 8, "own"), (2, 9, 2, 40, 0, 4), (1, 50, 2, 24, 12, "own"), (1, 5, 1, 1, 0, "own"),
         (2, 11, 3, 7, 6, "own"), (1, 20, 2, 128, 128, 1), (1, 3, 2, 250, 250, 3), (64, 1, 8, 128, 64, "own"),
         (1, 3000, 1, 16, 16, "own"), (2, 3, 2, 200, 2, "own"), (1, 9, 2, 64, 36, "own"), (2, 7, 3, 256, 4, 8),
         (1, 30, 2, 128, 64, 2), (1, 6, 5, 40, 20, 6)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward_and_backward(oracle, case, dtype, inter):
    b, t, g, n, rotary, layout = case
    p = problem(b, t, g, n, rotary, dtype, seed=sum(map(int, case[:5])), layout=layout, far=n % 3 == 2)
    kw = dict(weight_B=p["wB"], weight_C=p["wC"], eps=1e-4, interleaved=inter)
    Bo, Co = binding.norm_rotate(p["B"], p["C"], p["pos"], p["freq"], **kw)
    gr = binding.norm_rotate_backward(p["dB"], p["dC"], p["B"], p["C"], p["pos"], p["freq"], **kw)
    v = {k: host(x) for k, x in p.items()}
    ty = TYPES[dtype]
    args = (v["pos"], v["freq"], 1e-4, inter)
    close(Bo, oracle.norm_rotate(v["B"], v["wB"], *args), ty, what="B")
    close(Co, oracle.norm_rotate(v["C"], v["wC"], *args), ty, what="C")
    for k in "BC":
        dx, dw = oracle.norm_rotate_grad(v["d" + k], v[k], v["w" + k], *args)
        rstd = 1 / np.sqrt(np.mean(v[k] ** 2, axis=-1, keepdims=True) + 1e-4)
        d = oracle.norm_rotate_grad(v["d" + k], np.zeros_like(v[k]), v["w" + k], args[0], args[1], 1.0, inter)[0]
        close(gr["d" + k], dx, ty, what="d" + k, top=np.max(rstd * np.abs(d)))
        close(gr["dweight_" + k], dw, rel=2e-5, what="dw" + k)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [64, 20])
def test_without_weights(oracle, dtype, n):
    p = problem(2, 9, 2, n, 8, dtype, seed=3)
    Bo, Co = binding.norm_rotate(p["B"], p["C"], p["pos"], p["freq"], weight_C=p["wC"])
    gr = binding.norm_rotate_backward(p["dB"], p["dC"], p["B"], p["C"], p["pos"], p["freq"], weight_C=p["wC"])
    v = {k: host(x) for k, x in p.items()}
    args = (v["pos"], v["freq"], 1e-5, False)
    close(Bo, oracle.norm_rotate(v["B"], None, *args), TYPES[dtype])
    close(gr["dB"], oracle.norm_rotate_grad(v["dB"], v["B"], None, *args)[0], TYPES[dtype])
    assert gr["dweight_B"] is None and gr["dweight_C"] is not None


@pytest.mark.parametrize("n,rotary", [(64, 32), (30, 10)])
def test_far_positions_zero_rows_and_nan(oracle, n, rotary):
    """Positions to 2^40 keep their angle; a row of zeros stays zero; a NaN stays
    in its row."""
    p = problem(1, 6, 2, n, rotary, "f32", seed=4)
    p["pos"][0] = torch.tensor([0, -1, 1 << 20, (1 << 40) + 12345, -(1 << 33), 7], device=DEV)
    p["B"][0, 1, 0] = 0
    Bo, Co = binding.norm_rotate(p["B"], p["C"], p["pos"], p["freq"])
    v = {k: host(x) for k, x in p.items()}
    # the angle itself is a 64-bit number: 2^40 rad is off by 2^-13 * 2^-... = 1e-4 in the
    # reference, so that row is compared by its norms, which the rotation keeps
    ref = oracle.norm_rotate(v["B"], None, v["pos"], v["freq"], 1e-5, False)
    for t in (0, 1, 2, 5):
        np.testing.assert_allclose(host(Bo)[0, t], ref[0, t], atol=4e-6 * np.abs(ref).max())
    h = rotary // 2
    for o, r in ((host(Bo)[0, 3], ref[0, 3]),):
        np.testing.assert_allclose(o[:, :h] ** 2 + o[:, h:rotary] ** 2, r[:, :h] ** 2 + r[:, h:rotary] ** 2,
                                   rtol=1e-4, atol=1e-6)
    assert not Bo[0, 1, 0].any()
    p["B"][0, 2, 1, 3] = float("nan")
    B2, C2 = binding.norm_rotate(p["B"], p["C"], p["pos"], p["freq"])
    assert torch.isnan(B2[0, 2, 1]).all() and torch.equal(C2, Co)
    B2[0, 2, 1] = Bo[0, 2, 1]
    assert torch.equal(B2, Bo)


def test_before_the_scan(oracle):
    """With the scan that takes them: rotating by position leaves the masked products
    C_t . B_s a function of t - s, so shifted positions give the same y."""
    b, t, H, P, g, n = 1, 192, 4, 64, 2, 64
    p = problem(b, t, g, n, n, "f32", seed=6)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(9)
    x = torch.randn(b, t, H, P, generator=gen, device=DEV)
    dt = 0.01 + 0.1 * torch.rand(b, t, H, generator=gen, device=DEV)
    A = -torch.rand(H, generator=gen, device=DEV)
    ys = []
    for shift in (0, 100):
        pos = (torch.arange(t, device=DEV) + shift)[None].contiguous()
        B, C = binding.norm_rotate(p["B"], p["C"], pos, p["freq"], weight_B=p["wB"], weight_C=p["wC"])
        ys.append(host(binding.forward(x, dt, A, B, C, chunk_len=64)))
    v = {k: host(w) for k, w in p.items()}
    pos = np.arange(t)[None]
    want, _ = oracle.ssd_recurrent(host(x), host(dt), host(A),
                                   oracle.norm_rotate(v["B"], v["wB"], pos, v["freq"], 1e-5, False),
                                   oracle.norm_rotate(v["C"], v["wC"], pos, v["freq"], 1e-5, False))
    for y in ys:  # the scan's bound for fp32
        assert np.abs(y - want).max() <= 1e-4 * np.abs(want).max()


def test_same_bits_captured(oracle):
    p = problem(2, 700, 2, 64, 64, "bf16", seed=7)
    kw = dict(weight_B=p["wB"], weight_C=p["wC"])
    ins = (p["B"], p["C"], p["pos"], p["freq"])
    want = binding.norm_rotate_backward(p["dB"], p["dC"], *ins, **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = binding.norm_rotate_backward(p["dB"], p["dC"], *ins, **kw)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


def test_offsets_past_32_bits():
    """More than 2^31 values a tensor, slices of one projection among them."""
    b, t, g, n = 2, 140000, 32, 256
    gen = torch.Generator(device=DEV)
    gen.manual_seed(8)
    rows = torch.randn(b, t, 2 * g * n, generator=gen, device=DEV, dtype=torch.bfloat16)
    B, C = (v.unflatten(-1, (g, n)) for v in rows.split(g * n, -1))
    pos = torch.arange(t, device=DEV).expand(b, t).contiguous()
    freq = 10000.0 ** (-torch.arange(64, device=DEV, dtype=torch.float32) / 64)
    Bo, Co = binding.norm_rotate(B, C, pos, freq)
    at = slice(t - 100, t)
    few = [v[1:, at] for v in (B, C)]
    assert rows.numel() > 1 << 32
    B1, C1 = binding.norm_rotate(*few, pos[1:, at].contiguous(), freq)
    assert torch.equal(Bo[1:, at], B1) and torch.equal(Co[1:, at], C1)
    gr = binding.norm_rotate_backward(Bo, Co, B, C, pos, freq)
    g1 = binding.norm_rotate_backward(B1, C1, *few, pos[1:, at].contiguous(), freq)
    assert torch.equal(gr["dB"][1:, at], g1["dB"]) and torch.equal(gr["dC"][1:, at], g1["dC"])
