"""The decode step of as many rows as it takes: 2^31 - 1 of them, whose last ones are
one step of the grid from the end of 32-bit indices."""
import pytest
import torch

from structured_state_space_mamba_b200 import binding

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.mark.parametrize("B", [65535, 65536, 200001, (1 << 31) - 1])
def test_every_row_takes_one_step(B):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    # 2^16 - 1 different rows, over and over: a row's bits are those of a call of its own
    n = 65535
    few = [torch.randn(n, 1, generator=gen, device=DEV).bfloat16() for _ in range(3)]
    start = torch.randn(n, 1, generator=gen, device=DEV)
    A = torch.full((1,), -0.3, device=DEV)

    def wide(v):
        out = v.new_empty(B, 1)
        whole = B // n * n
        out[:whole].view(-1, n).copy_(v.view(1, n).expand(whole // n, n))
        out[whole:] = v[: B - whole]
        return out

    state, (x, r, i) = wide(start), (wide(v) for v in few)
    y = binding.glr_step(state, x, r, i, A)
    del x, r, i
    want_state = start.clone()
    want = binding.glr_step(want_state, *few, A)
    whole = B // n * n
    for got, w in ((y, want), (state, want_state)):
        assert all(torch.equal(part, w.view(1, n).expand_as(part)) for part in got[:whole].view(-1, n).split(1024))
        assert torch.equal(got[whole:], w[: B - whole])
