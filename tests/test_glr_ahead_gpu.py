"""The forward pass of few chains forms a tile's gates ahead of the state before it,
that of many does not: the bits of a row are the same in both, with everything
that the pass leaves, whole tiles or ragged ones, packed or not, and long rows
agree with the fp64 reference."""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def problem(B, T, C, seed=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, r, i = (rnd(B, T, C).bfloat16() for _ in range(3))
    return x, r, i, -torch.exp(-9 * torch.rand(C, generator=g, device=DEV)), rnd(B, C)


@pytest.mark.parametrize("T,C,save", [(2560, 128, "packed8"), (2501, 72, "inputs"), (641, 200, "packed8"),
                                      (64, 128, "inputs"), (1, 64, "packed8")])
def test_a_row_alone_and_among_many(T, C, save):
    # 256 rows: more chains than half the groups of any launch (3 on each of 148 SMs)
    x, r, i, A, h0 = problem(256, T, C)
    y, fin, saved = binding.glr_forward(x, r, i, A, init_state=h0, return_final_state=True, save=save)
    states = saved.chunk_states.unflatten(0, (256, -1))
    for b in (0, 101, 255):
        at = slice(b, b + 1)
        y1, fin1, s1 = binding.glr_forward(x[at], r[at], i[at], A, init_state=h0[at], return_final_state=True, save=save)
        assert torch.equal(y1, y[at]) and torch.equal(fin1, fin[at]) and torch.equal(s1.chunk_states, states[b])
        if save == "packed8":
            for one, many in ((s1.x, saved.x), (s1.r, saved.r), (s1.i, saved.i)):
                assert torch.equal(one.codes, many.codes[at]) and torch.equal(one.exps, many.exps[at])
    assert binding.device_status() == 0


def test_packed_sequences_alone_and_among_many():
    lens = [3, 0, 700, 64, 1, 129, 2000] + [5] * 70
    cu = np.concatenate([[0], np.cumsum(lens)])
    x, r, i, A, h0 = problem(1, int(cu[-1]), 256, seed=1)
    h0 = h0.expand(len(lens), -1).contiguous()
    y, fin = binding.glr_forward(x, r, i, A, init_state=h0, cu_seqlens=cu, return_final_state=True)
    few = cu[:8]  # 7 sequences
    part = [t[:, : few[-1]].contiguous() for t in (x, r, i)]
    y1, fin1 = binding.glr_forward(*part, A, init_state=h0[:7].contiguous(), cu_seqlens=few, return_final_state=True)
    assert torch.equal(y1, y[:, : few[-1]]) and torch.equal(fin1, fin[:7])
    assert binding.device_status() == 0


def test_many_tiles_a_group(oracle):
    # 2 chains of 600 tiles: groups come round to the same chain again
    x, r, i, A, h0 = problem(1, 600 * 64 - 5, 128, seed=2)
    y, fin, saved = binding.glr_forward(x, r, i, A, init_state=h0, return_final_state=True, save="inputs")
    v = [t.double().cpu().numpy() for t in (x, r, i, A, h0)]
    yr, fr, before = oracle.glr(*v)
    # bf16 values are off by half a step, 2^-8 of themselves; fp32 ones by the gates'
    # errors, below 1e-6 a value: 1e-5 of the largest holds them
    assert np.all(np.abs(y.double().cpu().numpy() - yr) <= 2.0 ** -8 * np.abs(yr) + 1e-5 * np.abs(yr).max())
    for got, want in ((fin, fr), (saved.chunk_states, before[0, ::64])):
        assert np.abs(got.double().cpu().numpy() - want).max() <= 1e-5 * np.abs(yr).max()
    again = binding.glr_forward(x, r, i, A, init_state=h0)
    assert torch.equal(again, y) and binding.device_status() == 0
