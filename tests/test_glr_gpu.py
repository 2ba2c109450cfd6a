"""GPU parity of the gated linear recurrence (forward, backward, step) against the
fp64 reference, on inputs that both sides see with the same rounding.

Tolerances, before the first run.  fp32 results: each value carries the gates'
errors (the hardware's 2^x, 1/x and 1/sqrt are within 2^-22, three or four of
them a value: below 1e-6) and the sum's roundings; the decays are kept as
a - 1, so that their relative error does not grow with the memory of the
channel.  1e-5 of the largest magnitude holds both with a factor of ten.
Values stored in bf16 add half a step of it, eps / 2 = 2^-8 of each value.
dA sums B T terms of either sign whose roundings are independent: 2e-5 of the
largest magnitude.
"""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(a, dtype=torch.float32):
    return torch.tensor(np.asarray(a), device=DEV).to(dtype)


def host(t):
    return t.double().cpu().numpy()


def close(got, want, dtype=torch.float32, rel=1e-5, what=""):
    got, want = host(got), np.asarray(want)
    assert got.shape == want.shape, what
    half = torch.finfo(dtype).eps / 2 if dtype == torch.bfloat16 else 0.0
    top = np.max(np.abs(want)) if want.size else 0.0
    bad = np.abs(got - want) > rel * top + half * np.abs(want)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.abs(got - want).max():.3e} of {top:.3e}"


def problem(shape, dtype, seed=0, S=None):
    """Inputs on the device; decays of 0.5 to 0.9999 a token, as learnt ones are."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    t = TYPES[dtype]
    S = shape[0] if S is None else S
    rnd = lambda *s, to=t: torch.randn(*s, generator=g, device=DEV).to(to)  # noqa: E731
    p = dict(x=rnd(*shape), r=2 * rnd(*shape), i=2 * rnd(*shape), dy=rnd(*shape))
    p["A"] = -torch.exp(-9 * torch.rand(shape[-1], generator=g, device=DEV))
    p["h0"], p["dfin"] = rnd(S, shape[-1], to=torch.float32), rnd(S, shape[-1], to=torch.float32)
    return p


SHAPES = [(1, 1, 1), (2, 3, 2), (1, 63, 64), (3, 64, 65), (2, 65, 130), (1, 129, 7), (2, 300, 96), (1, 2500, 33),
          (5, 128, 200)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("extras", [True, False])
def test_forward_and_backward(oracle, shape, dtype, extras):
    p = problem(shape, dtype)
    h0, df = (p["h0"], p["dfin"]) if extras else (None, None)
    y, fin, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=h0, return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(p["dy"], saved, dfinal_state=df, return_dinit_state=True)
    n = {k: host(v) for k, v in p.items()}
    yr, fr, _ = oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"] if extras else None)
    gr = oracle.glr_grad(n["x"], n["r"], n["i"], n["A"], n["dy"], n["h0"] if extras else None,
                         n["dfin"] if extras else None)
    t = TYPES[dtype]
    close(y, yr, t, what="y")
    close(fin, fr, what="final")
    for k in ("dx", "dr", "di"):
        close(g[k], gr[k], t, what=k)
    close(g["dA"], gr["dA"], rel=2e-5, what="dA")
    close(g["dinit_state"], gr["dh0"], what="dinit")
    assert binding.device_status() == 0


CUS = [[0, 5], [0, 0, 1, 2, 2, 66, 130, 130], [0, 64, 128, 129, 400], [0, 0, 0, 7],
       list(range(0, 201)) + [300, 300, 555]]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cu", CUS, ids=[str(len(c) - 1) + "seqs" for c in CUS])
@pytest.mark.parametrize("C", [34, 129])
def test_packed_sequences(oracle, cu, dtype, C):
    """Empty and one-token sequences, more than one launch holds, ends inside a
    chunk; the states of an empty sequence pass through."""
    p = problem((1, cu[-1], C), dtype, seed=3, S=len(cu) - 1)
    y, fin, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], cu_seqlens=cu,
                                        return_final_state=True, save="inputs")
    g = binding.glr_backward(p["dy"], saved, dfinal_state=p["dfin"], return_dinit_state=True)
    n = {k: host(v) for k, v in p.items()}
    yr, fr, _ = oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"], cu)
    gr = oracle.glr_grad(n["x"], n["r"], n["i"], n["A"], n["dy"], n["h0"], n["dfin"], cu)
    t = TYPES[dtype]
    close(y, yr, t, what="y")
    close(fin, fr, what="final")
    for k in ("dx", "dr", "di"):
        close(g[k], gr[k], t, what=k)
    close(g["dA"], gr["dA"], rel=2e-5, what="dA")
    close(g["dinit_state"], gr["dh0"], what="dinit")
    for j in range(len(cu) - 1):
        if cu[j] == cu[j + 1]:
            assert torch.equal(fin[j], p["h0"][j]) and torch.equal(g["dinit_state"][j], p["dfin"][j])
    # without states given: zeros
    y0, fin0 = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], cu_seqlens=cu, return_final_state=True)
    close(y0, oracle.glr(n["x"], n["r"], n["i"], n["A"], None, cu)[0], t)
    assert all(not fin0[j].any() for j in range(len(cu) - 1) if cu[j] == cu[j + 1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shape,cu", [((2, 70, 64), None), ((1, 200, 130), None), ((1, 130, 67), [0, 1, 1, 66, 130]),
                                      ((3, 1, 5), None), ((2, 65, 36), None), ((1, 128, 200), [0, 64, 128]),
                                      ((1, 3, 1), None)])
def test_saved_in_8_bits(oracle, shape, cu, dtype):
    """The checkpoints that the forward pass writes are pack8's; the backward pass
    is the gradient at the values they stand for, from the kept states."""
    p = problem(shape, dtype, seed=5, S=len(cu) - 1 if cu else None)
    args = (p["x"], p["r"], p["i"], p["A"])
    y, saved = binding.glr_forward(*args, init_state=p["h0"], cu_seqlens=cu, save="packed8")
    assert torch.equal(y, binding.glr_forward(*args, init_state=p["h0"], cu_seqlens=cu))
    n = {k: host(v) for k, v in p.items()}
    q = {}
    for k, s in (("x", saved.x), ("r", saved.r), ("i", saved.i)):
        codes, exps = oracle.pack8(n[k])
        assert np.array_equal(s.codes.cpu().numpy(), codes) and np.array_equal(s.exps.cpu().numpy(), exps)
        q[k] = oracle.unpack8(codes, exps)
    g = binding.glr_backward(p["dy"], saved, dfinal_state=p["dfin"], return_dinit_state=True)
    kept = oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"], cu)[2]
    gr = oracle.glr_grad(q["x"], q["r"], q["i"], n["A"], n["dy"], n["h0"], n["dfin"], cu, kept=kept,
                         chunk=binding.GLR_CHUNK)
    for k in ("dx", "dr", "di"):
        close(g[k], gr[k], TYPES[dtype], what=k)
    close(g["dA"], gr["dA"], rel=2e-5, what="dA")
    close(g["dinit_state"], gr["dh0"], what="dinit")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 33), (64, 512), (2, 1027)])
def test_step(oracle, B, C, dtype):
    p = problem((B, 1, C), dtype, seed=7)
    state = p["h0"].clone()
    y = binding.glr_step(state, p["x"][:, 0], p["r"][:, 0], p["i"][:, 0], p["A"])
    n = {k: host(v) for k, v in p.items()}
    yr, fr, _ = oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"])
    close(y, yr[:, 0], TYPES[dtype])
    close(state, fr)


def test_prefill_then_steps_is_one_sequence(oracle):
    p = problem((2, 75, 48), "bf16", seed=8)
    y, state = binding.glr_forward(*(p[k][:, :70].contiguous() for k in "xri"), p["A"], init_state=p["h0"],
                                   return_final_state=True)
    ys = [y] + [binding.glr_step(state, *(p[k][:, t].contiguous() for k in "xri"), p["A"])[:, None]
                for t in range(70, 75)]
    n = {k: host(v) for k, v in p.items()}
    yr, fr, _ = oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"])
    close(torch.cat(ys, 1), yr, torch.bfloat16)
    close(state, fr)


@pytest.mark.parametrize("seed", range(5))
def test_saturated_gates(oracle, seed):
    """Gates open and closed as far as they go, decays that vanish, A = 0: finite,
    and the reference's values; a NaN stays in its channel from its token on."""
    B, T, C = 1, 130, 8
    p = problem((B, T, C), "f32", seed=9)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    vals = torch.tensor([-200.0, -60.0, -30.0, 0.0, 30.0, 60.0, 200.0, 1.0], device=DEV)
    p["r"] = vals[torch.randint(0, 8, (B, T, C), device=DEV, generator=gen)]
    p["i"] = vals[torch.randint(0, 8, (B, T, C), device=DEV, generator=gen)]
    p["A"] = torch.tensor([0.0, -1e-6, -1e-3, -0.5, -1.0, -8.0, -80.0, -1e4], device=DEV)
    y, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], save="inputs")
    g = binding.glr_backward(p["dy"], saved)
    n = {k: host(v) for k, v in p.items()}
    close(y, oracle.glr(n["x"], n["r"], n["i"], n["A"], n["h0"])[0])
    gr = oracle.glr_grad(n["x"], n["r"], n["i"], n["A"], n["dy"], n["h0"])
    for k in ("dx", "di"):
        close(g[k], gr[k], what=k)
    # dr, dA: a gate closed to 2e-19 (the kernels' least) instead of e^-200 leaves
    # the root's derivative where the reference has almost 0 * infinity
    open_ = n["r"] > -43
    assert torch.isfinite(g["dr"]).all() and torch.isfinite(g["dA"]).all()
    # compared channel by channel: their scales differ by orders of magnitude
    for c in range(1, C):
        m = open_[..., c]
        np.testing.assert_allclose(host(g["dr"])[..., c][m], gr["dr"][..., c][m],
                                   atol=1e-5 * np.abs(gr["dr"][..., c]).max())
    p["x"][0, 70, 3] = float("nan")
    y2 = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"])
    assert torch.isnan(y2[0, 70:, 3]).all() and torch.equal(y2[0, :70], y[0, :70])
    keep = [c for c in range(C) if c != 3]
    assert torch.equal(y2[..., keep], y[..., keep])


def test_same_bits_every_time_and_on_two_streams():
    p = problem((1, 6000, 256), "bf16", seed=11)
    first = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], return_final_state=True, save="inputs")
    g0 = binding.glr_backward(p["dy"], first[2])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for k in range(6):
        y, f, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], return_final_state=True, save="inputs",
                                          stream=streams[k % 2])
        got.append((y, f, binding.glr_backward(p["dy"], saved, stream=streams[k % 2].cuda_stream)))
    torch.cuda.synchronize()
    for y, f, g in got:
        assert torch.equal(y, first[0]) and torch.equal(f, first[1])
        assert all(torch.equal(g[k], g0[k]) for k in ("dx", "dr", "di", "dA"))
    assert binding.device_status() == 0


def test_streams_by_object_and_handle():
    """The default stream from another one, a torch stream and its handle; the offsets
    given to the forward pass may change before the backward one."""
    p = problem((1, 300, 64), "f32", seed=12, S=2)
    cu = np.array([0, 100, 300])
    args = (p["x"], p["r"], p["i"], p["A"])
    want, saved = binding.glr_forward(*args, cu_seqlens=cu, save="inputs")
    g = binding.glr_backward(p["dy"], saved)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = [binding.glr_forward(*args, cu_seqlens=cu, stream=t) for t in (0, None, s, s.cuda_stream)]
    y, kept = binding.glr_forward(*args, cu_seqlens=cu, save="inputs")
    cu[1] = 200
    again = binding.glr_backward(p["dy"], kept)
    torch.cuda.synchronize()
    assert all(torch.equal(t, want) for t in got + [y])
    assert all(torch.equal(again[k], g[k]) for k in ("dx", "dr", "di", "dA"))


def test_captured_and_replayed():
    """Two graphs of the whole training step, replayed in turn on other inputs."""
    p = problem((2, 500, 96), "bf16", seed=13)
    q = problem((2, 500, 96), "bf16", seed=14)

    def step(p):
        y, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], save="packed8")
        return y, binding.glr_backward(p["dy"], saved)

    want = []
    for v in (p, q):
        y, g = step(v)
        want.append([y.clone()] + [g[k].clone() for k in ("dx", "dr", "di", "dA")])
    torch.cuda.synchronize()
    bufs = [{k: v.clone() for k, v in p.items()} for _ in range(2)]
    graphs, outs = [], []
    for b in bufs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, g = step(b)
        graphs.append(graph)
        outs.append([y] + [g[k] for k in ("dx", "dr", "di", "dA")])
    for first, second in ((p, q), (q, p), (p, p)):
        for b, v in zip(bufs, (first, second)):
            for k in b:
                b[k].copy_(v[k])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for o, v in zip(outs, (first, second)):
            for a, w in zip(o, want[0] if v is p else want[1]):
                assert torch.equal(a, w)


def test_out_and_untouched_neighbours(oracle):
    """Writes stay inside the outputs: guard rows before and behind."""
    C, T = 33, 67
    p = problem((1, T, C), "bf16", seed=15)
    big = torch.full((T + 64, C), 7.0, dtype=torch.bfloat16, device=DEV)
    out = big[32: 32 + T].unsqueeze(0)
    if out.data_ptr() % 16:
        pytest.skip("rows of this size do not fall on 16 bytes")
    y = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], out=out)
    assert y.data_ptr() == out.data_ptr()
    assert (big[:32] == 7).all() and (big[32 + T:] == 7).all()
    assert torch.equal(y, binding.glr_forward(p["x"], p["r"], p["i"], p["A"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [128, 37])
def test_checkpoints_of_values_at_the_edge(dtype, C):
    """Infinities, NaN, zeros and the largest numbers among the inputs: the forward
    pass writes the checkpoints that pack8 writes."""
    p = problem((1, 40, C), dtype, seed=17)
    top = torch.finfo(TYPES[dtype]).max
    for k, v in (("x", top), ("r", float("inf")), ("i", float("nan"))):
        p[k][0, 3, 1], p[k][0, 9, C - 1], p[k][0, 20] = v, -v, 0
    _, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], save="packed8")
    for k, s in (("x", saved.x), ("r", saved.r), ("i", saved.i)):
        q = binding.pack8(p[k])
        assert torch.equal(s.codes, q.codes) and torch.equal(s.exps, q.exps)


def test_any_bits_of_a_nan():
    """A NaN of all ones, the bits that mark what is not written yet between tiles,
    in the inputs and in the states given: it comes out as a NaN, and nothing waits for it."""
    p = problem((1, 400, 70), "f32", seed=18)
    ones = torch.tensor([-1], dtype=torch.int32, device=DEV).view(torch.float32)
    p["x"][0, 100, 3], p["r"][0, 150, 4], p["i"][0, 64, 5] = ones, ones, ones
    p["h0"][0, 6], p["dfin"][0, 7], p["dy"][0, 200, 8] = ones, ones, ones
    y, fin, saved = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], return_final_state=True,
                                        save="inputs")
    g = binding.glr_backward(p["dy"], saved, dfinal_state=p["dfin"], return_dinit_state=True)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    first = {3: 100, 4: 150, 5: 64, 6: 0}
    for c in range(70):
        t = first.get(c, 400)
        assert torch.isnan(y[0, t:, c]).all() and torch.isfinite(y[0, :t, c]).all(), c
    assert torch.isnan(fin[0, list(first)]).all()
    # backwards from the cotangents' NaN to the start (and through a gate that is one)
    assert torch.isnan(g["dx"][0, :, 7]).all() and torch.isnan(g["dx"][0, :201, 8]).all()
    assert torch.isfinite(g["dx"][0, 201:, 8]).all() and torch.isnan(g["dinit_state"][0, [4, 7, 8]]).all()
    quiet = [c for c in range(70) if c not in (3, 4, 5, 6, 7, 8)]
    assert all(torch.isfinite(g[k][..., quiet]).all() for k in ("dx", "dr", "di", "dA"))


def test_a_long_chain_and_a_single_one():
    """Many tiles of one chain in flight at once; the bits are those of any other cut
    of the batch into calls."""
    p = problem((3, 20000, 64), "bf16", seed=19)
    y, fin = binding.glr_forward(p["x"], p["r"], p["i"], p["A"], init_state=p["h0"], return_final_state=True)
    for b in range(3):
        yb, fb = binding.glr_forward(*(p[k][b: b + 1] for k in "xri"), p["A"], init_state=p["h0"][b: b + 1],
                                     return_final_state=True)
        assert torch.equal(yb[0], y[b]) and torch.equal(fb[0], fin[b])
    cu = [0, 20000, 40000, 60000]
    yv, fv = binding.glr_forward(*(p[k].view(1, 60000, 64) for k in "xri"), p["A"], init_state=p["h0"],
                                 cu_seqlens=cu, return_final_state=True)
    assert torch.equal(yv.view_as(y), y) and torch.equal(fv, fin)
    assert binding.device_status() == 0


def test_offsets_past_32_bits():
    """More than 2^31 values a tensor: the last row's bits are those of a call of its own."""
    B, T, C = 3, 70000, 10240
    g = torch.Generator(device=DEV)
    g.manual_seed(21)
    x = torch.randn(B, T, C, generator=g, device=DEV, dtype=torch.bfloat16)
    A = -torch.exp(-5 * torch.rand(C, generator=g, device=DEV))
    r, i = x.roll(1, 0), x.roll(1, 2)
    y, saved = binding.glr_forward(x, r, i, A, save="packed8")
    last = slice(B - 1, B)
    one, kept = binding.glr_forward(x[last], r[last], i[last], A, save="packed8")
    assert torch.equal(y[last], one)
    assert torch.equal(saved.r.codes[last], kept.r.codes) and torch.equal(saved.r.exps[last], kept.r.exps)
    grads = binding.glr_backward(y, saved)
    alone = binding.glr_backward(one, kept)
    for k in ("dx", "dr", "di"):
        assert torch.equal(grads[k][last], alone[k])
    q = binding.pack8(r)
    assert torch.equal(q.codes, saved.r.codes) and torch.equal(q.exps, saved.r.exps)
    assert torch.equal(binding.unpack8(q)[last], binding.unpack8(kept.r))
