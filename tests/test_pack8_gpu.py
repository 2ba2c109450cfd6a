"""GPU tests of the 8-bit checkpoints: every code and exponent is the reference's
(the format leaves no choice), and values read back exactly in both types."""
import numpy as np
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def values(shape, dtype, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    # magnitudes over the whole range of the type, halves and quarters among them (ties)
    x = torch.where(torch.rand(shape, generator=g, device=DEV) < 0.3, torch.round(x * 8) / 4, x)
    return (x * torch.exp2(torch.randint(-20, 20, (*shape[:-1], 1), generator=g, device=DEV).float())).to(dtype)


SHAPES = [(1, 1), (3, 7), (5, 64), (4, 65), (1000, 8), (17, 72), (2, 3, 200), (33, 1027), (257, 512), (64,)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_codes_exponents_and_values(oracle, shape, dtype):
    x = values(shape, dtype, 1)
    p = binding.pack8(x)
    codes, exps = oracle.pack8(x.double().cpu().numpy())
    assert np.array_equal(p.codes.cpu().numpy(), codes)
    assert np.array_equal(p.exps.cpu().numpy(), exps)
    want = torch.from_numpy(oracle.unpack8(codes, exps))
    for t in (torch.float32, torch.bfloat16):
        got = binding.unpack8(p, t)
        assert got.dtype == t and torch.equal(got.double().cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cols", [64, 40, 33])
def test_zeros_tiny_huge_and_not_finite(oracle, dtype, cols):
    tiny, top = torch.finfo(dtype).tiny, torch.finfo(dtype).max
    x = torch.zeros(8, cols, dtype=dtype, device=DEV)
    x[1], x[1, 0] = tiny, tiny / 4 if dtype == torch.float32 else tiny
    x[2] = -top
    x[3, 5] = float("inf")
    x[4, 5] = float("nan")
    x[5, 5] = -float("inf")
    x[6, 0], x[6, 1] = 127.5, 127.0
    x[7, 0] = 2.0 ** -133 if dtype == torch.float32 else 2.0 ** -130
    p = binding.pack8(x)
    codes, exps = oracle.pack8(x.double().cpu().numpy())
    assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.exps.cpu().numpy(), exps)
    back = binding.unpack8(p, torch.float32).double().cpu().numpy()
    np.testing.assert_array_equal(back, oracle.unpack8(codes, exps))
    assert np.isnan(back[3:6]).all() and np.isfinite(back[[0, 1, 2, 6, 7]]).all()


def test_a_large_activation_on_another_stream():
    x = values((4096, 5120), torch.bfloat16, 2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    p = binding.pack8(x, stream=s)
    got = binding.unpack8(p, stream=s)
    s.synchronize()
    top = x.float().unflatten(-1, (-1, 64)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, 64).flatten(-2) \
        if x.dim() == 3 else x.float().unflatten(-1, (-1, 64)).abs().amax(-1).repeat_interleave(64, -1)
    assert ((got.float() - x.float()).abs() <= top / 127.5).all()
    # packing what was read back gives it again
    again = binding.unpack8(binding.pack8(got))
    assert torch.equal(again, got)


@pytest.mark.parametrize("shape", [dict(batch=2, seqlen=200, nheads=4, headdim=64, dstate=64, ngroups=2, chunk_len=64, dtype="bf16"),
                                   dict(batch=1, seqlen=96, nheads=3, headdim=5, dstate=7, ngroups=1, chunk_len=32, dtype="f32")],
                         ids=["bf16", "f32"])
def test_ssd_backward_from_checkpoints(shape):
    """ssd_backward_packed8 is ssd_backward at the values read back, bit for bit."""
    from structured_state_space_mamba_b200.inputs import make_inputs
    inp = make_inputs(**shape, seed=5, init_state=True)
    t = torch.bfloat16 if shape["dtype"] == "bf16" else torch.float32
    dev = lambda a, ty=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(DEV).to(ty)  # noqa: E731
    x, B, C = dev(inp.x, t), dev(inp.B, t), dev(inp.C, t)
    dt, A, D, h0 = dev(inp.dt), dev(inp.A), dev(inp.D), dev(inp.h0)
    dy = torch.randn_like(x)
    px, pB, pC = binding.pack8(x), binding.pack8(B), binding.pack8(C)
    kw = dict(D=D, chunk_len=inp.chunk_len, init_state=h0, dfinal_state=torch.randn_like(h0))
    got = binding.backward_packed8(px, dt, A, pB, pC, dy, **kw)
    want = binding.backward(binding.unpack8(px, t), dt, A, binding.unpack8(pB, t), binding.unpack8(pC, t), dy, **kw)
    for k in want:
        assert torch.equal(got[k], want[k]), k
    for bad in (dict(x=x), dict(B=pC.codes), dict(dy=dy[:, :5]), dict(dt=dt.double())):
        a = dict(x=px, dt=dt, A=A, B=pB, C=pC, dy=dy)
        a.update(bad)
        with pytest.raises(ValueError):
            binding.backward_packed8(**a, **kw)
