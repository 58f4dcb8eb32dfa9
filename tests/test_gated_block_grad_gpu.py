"""The example's autograd function without an initial state."""
import pytest
import torch

from test_gated_block_gpu import example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("b,t,d", [(2, 1, 8), (2, 6, 10), (1, 300, 64)])
def test_gradient_without_an_initial_state(cuda_dev, b, t, d):
    """As from a state of zeros, to the bit."""
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(3)
    x = torch.randn((b, t, d), generator=gen, device=cuda_dev).requires_grad_()
    gate = (-torch.rand((b, t, d), generator=gen, device=cuda_dev)).requires_grad_()
    zeros = torch.zeros((b, d), device=cuda_dev, requires_grad=True)
    w = torch.randn((b, t, d), generator=gen, device=cuda_dev)
    v = torch.randn((b, d), generator=gen, device=cuda_dev)
    results = []
    for h0 in (None, zeros):
        h, state = example.GatedScan.apply(x, gate, h0)
        grads = torch.autograd.grad((h * w).sum() + (state * v).sum(), (x, gate))
        results.append((h, state, *grads))
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(*results))
