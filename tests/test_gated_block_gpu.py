"""The operators together, as examples/gated_block.py runs them.

Bound: with the same rounding points, two ways of computing the block differ in the
order of fp32 sums, which moves a value that is rounded (to 16 bits: u, g, h, out;
to 8 bits: y) to its neighbour now and then.  Half a unit (2^-9 relative) on every
value of the four 16-bit tensors of a block is far more: 4 * 2^-9 per block, in
the 2-norm.
"""
import importlib.util
import os

import pytest
import torch

import memory_bound_gemv_02_gb300 as g

pytestmark = pytest.mark.gpu

_path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_block.py")
_spec = importlib.util.spec_from_file_location("gated_block", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

BOUND = 4 * 2.0 ** -9


def _apart(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def _plain_block(block, x, stream, state):
    """The block in fp64 with the operators' rounding points."""
    bf16 = torch.bfloat16
    s = x.double() + stream.double()
    y = s * block.norm.double() / (s.square().mean(-1, keepdim=True) + 1e-6).sqrt()
    scale = (y.abs().amax(-1, keepdim=True) / 448).float().double()
    y = (y / scale).float().to(torch.float8_e4m3fn).double() * scale
    u = y @ (block.w_u.double() * block.s_u.double()[:, None]).T + block.b_u.double()
    gate = y @ (block.w_g.double() * block.s_g.double()[:, None]).T + block.b_g.double()
    u, gate = u.to(bf16).double(), torch.nn.functional.logsigmoid(gate).to(bf16).double()
    h, v = [], state.double()
    for t in range(x.shape[1]):
        v = gate[:, t].exp() * v + u[:, t]
        h.append(v)
    h = torch.stack(h, 1).to(bf16).double()
    return (h @ block.w_o.double().T).to(bf16), s.to(bf16), v


@pytest.mark.parametrize("b,t,d,width", [(1, 1, 64, 96), (2, 100, 256, 300), (3, 33, 100, 77), (1, 700, 512, 1024)])
def test_block_against_plain(cuda_dev, b, t, d, width):
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(b + t)
    x, stream = (torch.randn((b, t, d), generator=gen, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
    state = torch.randn((b, width), generator=gen, device=cuda_dev)
    block = example.GatedBlock(d, width, cuda_dev, seed=t)
    out, kept, last = _plain_block(block, x, stream, state)
    got = block(x, stream, state)
    assert torch.equal(stream, kept)
    assert _apart(got, out) <= BOUND
    assert _apart(state, last) <= BOUND


@pytest.mark.parametrize("b,d,width", [(1, 256, 512), (4, 200, 301)])
def test_prompt_and_single_tokens_agree(cuda_dev, b, d, width):
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(d)
    blocks = [example.GatedBlock(d, width, cuda_dev, seed) for seed in range(2)]
    x = torch.randn((b, 60, d), generator=gen, device=cuda_dev).to(torch.bfloat16)
    whole_states = [k.new_state(b) for k in blocks]
    whole = example.run_blocks(blocks, x, whole_states)
    states = [k.new_state(b) for k in blocks]
    parts = [example.run_blocks(blocks, x[:, :40].contiguous(), states)]
    parts += [example.run_blocks(blocks, x[:, i:i + 1].contiguous(), states) for i in range(40, 60)]
    assert _apart(torch.cat(parts, 1), whole) <= 2 * BOUND
    for one, many in zip(states, whole_states):
        assert _apart(one, many) <= 2 * BOUND


def test_decoding_in_a_graph(cuda_dev):
    """A decode step captured once and replayed moves the state on as the calls do."""
    b, d, width = 2, 128, 256
    block = example.GatedBlock(d, width, cuda_dev)
    x = torch.randn((b, 1, d), device=cuda_dev).to(torch.bfloat16)
    state, token = block.new_state(b), x.clone()
    want_state = state.clone()
    example.run_blocks([block], token, [state.clone()])  # first use outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = example.run_blocks([block], token, [state])
    state.zero_()
    for i in range(3):
        token.copy_(x * (i + 1))
        graph.replay()
        want = example.run_blocks([block], x * (i + 1), [want_state])
        assert torch.equal(out, want) and torch.equal(state, want_state)


def test_gradient_of_the_autograd_function(cuda_dev):
    """Against central differences in fp32: step 1e-2 gives a truncation of some 1e-4
    (third derivatives are of order 1) and rounding of 1e-6 / 1e-2; the sum of 120
    terms is of order 1, so 1e-2 of it is allowed."""
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(5)
    x = torch.randn((2, 6, 10), generator=gen, device=cuda_dev).requires_grad_()
    gate = (-torch.rand((2, 6, 10), generator=gen, device=cuda_dev)).requires_grad_()
    h0 = torch.randn((2, 10), generator=gen, device=cuda_dev).requires_grad_()
    dh = torch.randn((2, 6, 10), generator=gen, device=cuda_dev)
    ds = torch.randn((2, 10), generator=gen, device=cuda_dev)

    def loss(x, gate, h0):
        h, state = example.GatedScan.apply(x, gate, h0)
        return (h.double() * dh).sum() + (state.double() * ds).sum()

    grads = torch.autograd.grad(loss(x, gate, h0), (x, gate, h0))
    for i, grad in enumerate(grads):
        args = [x.detach(), gate.detach(), h0.detach()]
        along = torch.randn(grad.shape, generator=gen, device=cuda_dev)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + 1e-2 * along, args[i] - 1e-2 * along
        slope = (loss(*up) - loss(*down)) / 2e-2
        size = (grad.double() * along).abs().sum()
        assert abs(slope - (grad.double() * along).sum()) <= 1e-2 * size, i
    assert g.gemv_wait_timeouts() == 0
