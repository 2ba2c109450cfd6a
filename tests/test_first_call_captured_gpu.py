"""The first call that a process makes of an operator may be under capture: its
one-time set-up (error word, workspace pool, shared-memory limits) does not end
the capture, and the replay gives the bits of a call outside."""
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

BODY = """
import torch
from structured_state_space_mamba_b200 import binding
gen = torch.Generator(device="cuda").manual_seed(3)
rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")
x, r, i, dy = (rnd(2, 130, 72).bfloat16() for _ in range(4))
A, w, h = -torch.rand(72, device="cuda"), rnd(24), rnd(2, 72)
rows, pos, fr = rnd(2, 130, 72).bfloat16(), torch.arange(130, device="cuda").repeat(2, 1), torch.rand(12, device="cuda")
Bm, Cm = rows.unflatten(-1, (3, 24)), dy.unflatten(-1, (3, 24))


def train():
    y, saved = binding.glr_forward(x, r, i, A, save="packed8")
    g = binding.glr_backward(dy, saved)
    return [y] + [g[k] for k in ("dx", "dr", "di", "dA")]


def step():
    s = h.clone()
    return [binding.glr_step(s, *(t[:, 0].contiguous() for t in (x, r, i)), A), s]


def pack():
    p = binding.pack8(x)
    return [p.codes, p.exps, binding.unpack8(p, torch.bfloat16)]


def rotate():
    out = binding.norm_rotate(Bm, Cm, pos, fr, weight_B=w)
    g = binding.norm_rotate_backward(Bm, Cm, Bm, Cm, pos, fr, weight_B=w)
    return list(out) + [g["dB"], g["dC"], g["dweight_B"]]


call = {"train": train, "step": step, "pack": pack, "rotate": rotate}[WHICH]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = call()
graph.replay()
torch.cuda.synchronize()
want = call()
assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
assert binding.device_status() == 0
"""


@pytest.mark.parametrize("which", ["train", "step", "pack", "rotate"])
def test_first_call_under_capture(which):
    r = subprocess.run([sys.executable, "-c", f"WHICH = {which!r}\n{BODY}"], capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-2000:]
