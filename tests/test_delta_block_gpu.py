"""The layer norm and the gated delta rule with the operators around them, as
examples/delta_block.py runs them.

Bound: with the same rounding points, two ways of computing the block differ in the
order of fp32 sums (in the rule's chunks, by 2^-16 of its products), which moves a
value that is rounded to 16 bits to its neighbour now and then.  Half a unit (2^-9
relative) on every value of the six 16-bit tensors of a block (y, the projections,
unit q and k, o, its norm, out) is far more: 6 * 2^-9 per block, in the 2-norm.
"""
import importlib.util
import os
import subprocess
import sys

import pytest
import torch

import memory_bound_gemv_02_gb300 as g

pytestmark = pytest.mark.gpu

_root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
_path = os.path.join(_root, "examples", "delta_block.py")
_spec = importlib.util.spec_from_file_location("delta_block", _path)
example = importlib.util.module_from_spec(_spec)
_spec.loader.exec_module(example)

BOUND = 6 * 2.0 ** -9


def _apart(a, b):
    return ((a.double() - b.double()).norm() / b.double().norm()).item()


def _norm(x, eps):
    c = x - x.mean(-1, keepdim=True)
    return c / (c.square().mean(-1, keepdim=True) + eps).sqrt()


def _plain_block(block, x, stream, state):
    """The block in fp64 with the operators' rounding points."""
    r = lambda v: v.to(torch.bfloat16).double()  # noqa: E731
    b, t, _ = x.shape
    s = x.double() + stream.double()
    y = r(_norm(s, 1e-5) * block.norm.double() + block.shift.double())
    qkv = r(y @ block.w_qkv.double().T)
    wide = block.keys * block.dk
    units = qkv[..., :2 * wide].reshape(b, t, 2, block.keys, block.dk)
    units = r(units / (units.square().mean(-1, keepdim=True) + 1e-6).sqrt() * block.dk ** -0.5)
    group = block.heads // block.keys
    q, k = (units[:, :, i].repeat_interleave(group, 2) for i in range(2))
    v = qkv[..., 2 * wide:].reshape(b, t, block.heads, block.dv)
    a = torch.sigmoid((y @ block.w_g.double().T + block.b_g.double()))
    beta = torch.sigmoid(y @ block.w_b.double().T)
    S, o = state.double(), []
    for i in range(t):
        S = S * a[:, i, :, None, None]
        d = beta[:, i, :, None] * (v[:, i] - torch.einsum("bhkv,bhk->bhv", S, k[:, i]))
        S = S + k[:, i, :, :, None] * d[..., None, :]
        o.append(torch.einsum("bhkv,bhk->bhv", S, q[:, i]) * block.dk ** -0.5)
    o = r(_norm(r(torch.stack(o, 1)), 1e-5))
    return (o.reshape(b, t, -1) @ block.w_o.double().T).to(torch.bfloat16), s.to(torch.bfloat16), S


@pytest.mark.parametrize("b,t,d,heads,keys,dk,dv", [(1, 1, 64, 2, 1, 32, 48), (2, 40, 256, 4, 2, 64, 64), (2, 100, 128, 4, 4, 40, 24),
                                                    (1, 300, 512, 6, 3, 128, 128), (4, 70, 200, 10, 5, 128, 128)])
def test_block_against_plain(cuda_dev, b, t, d, heads, keys, dk, dv):
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(b + t)
    x, stream = (torch.randn((b, t, d), generator=gen, device=cuda_dev).to(torch.bfloat16) for _ in range(2))
    state = 0.3 * torch.randn((b, heads, dk, dv), generator=gen, device=cuda_dev)
    block = example.DeltaBlock(d, heads, keys, dk, dv, cuda_dev, seed=t)
    out, kept, last = _plain_block(block, x, stream, state)
    got = block(x, stream, state)
    assert torch.equal(stream, kept)
    assert _apart(got, out) <= BOUND
    assert _apart(state, last) <= BOUND


def test_prompt_and_single_tokens_agree(cuda_dev):
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(3)
    blocks = [example.DeltaBlock(256, 4, 2, 64, 80, cuda_dev, seed) for seed in range(2)]
    x = torch.randn((2, 150, 256), generator=gen, device=cuda_dev).to(torch.bfloat16)
    whole_states = [k.new_state(2) for k in blocks]
    whole = example.run_blocks(blocks, x, whole_states)
    states = [k.new_state(2) for k in blocks]
    parts = [example.run_blocks(blocks, x[:, :130].contiguous(), states)]
    parts += [example.run_blocks(blocks, x[:, i:i + 1].contiguous(), states) for i in range(130, 150)]
    assert _apart(torch.cat(parts, 1), whole) <= 2 * BOUND
    for one, many in zip(states, whole_states):
        assert _apart(one, many) <= 2 * BOUND


def test_decoding_in_a_graph(cuda_dev):
    """A decode step captured once and replayed moves the state on as the calls do."""
    block = example.DeltaBlock(128, 4, 2, 64, 64, cuda_dev)
    x = torch.randn((2, 1, 128), device=cuda_dev).to(torch.bfloat16)
    state, token = block.new_state(2), x.clone()
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


def test_gradients_of_the_autograd_functions(cuda_dev):
    """The functions hand their operators' gradients on, each to its input."""
    gen = torch.Generator(device=cuda_dev)
    gen.manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, device=cuda_dev)  # noqa: E731
    x, res = r(12, 64).to(torch.bfloat16).requires_grad_(), r(12, 64).to(torch.bfloat16).requires_grad_()
    w, b = r(64).requires_grad_(), r(64).requires_grad_()
    dy, ds = r(12, 64).to(torch.bfloat16), r(12, 64).to(torch.bfloat16)
    y, s = example.LayerNorm.apply(x, res, w, b, 1e-5)
    got = torch.autograd.grad((y, s), (x, res, w, b), (dy, ds))
    _, mean, rstd, kept = g.layer_norm_fused(x.detach(), w.detach(), b.detach(), residual=res.detach(), stats=True)
    dx, dw, db = g.layer_norm_backward(dy, kept, w.detach(), mean, rstd, ds=ds)
    assert all(torch.equal(a, c) for a, c in zip(got, (dx, dx, dw, db)))
    y, _ = example.LayerNorm.apply(x, None, w, None, 1e-5)  # s unused: no gradient through it
    got = torch.autograd.grad(y, (x, w), dy)
    _, mean, rstd, _ = g.layer_norm_fused(x.detach(), w.detach(), stats=True)
    dx, dw, _ = g.layer_norm_backward(dy, x.detach(), w.detach(), mean, rstd)
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)

    q, k = (0.2 * r(1, 70, 1, 32)).to(torch.bfloat16).requires_grad_(), (0.2 * r(1, 70, 1, 32)).to(torch.bfloat16).requires_grad_()
    v = r(1, 70, 2, 16).to(torch.bfloat16).requires_grad_()
    gate, beta = (-r(1, 70, 2).abs()).requires_grad_(), torch.sigmoid(r(1, 70, 2)).requires_grad_()
    h0 = r(1, 2, 32, 16).requires_grad_()
    do, dstate = r(1, 70, 2, 16).to(torch.bfloat16), r(1, 2, 32, 16)
    leaves = (q, k, v, gate, beta, h0)
    o, last = example.GatedDelta.apply(q, k, v, gate, beta, 0.5, h0)
    got = torch.autograd.grad((o, last), leaves, (do, dstate))
    plain = [t.detach() for t in leaves]
    want = g.gated_delta_backward(do, *plain[:5], 0.5, h0=plain[5], dstate=dstate)
    assert all(torch.equal(a, c) for a, c in zip(got, want))
    o, _ = example.GatedDelta.apply(q, k, v, gate, beta, 0.5, None)
    assert len(torch.autograd.grad(o, leaves[:5], do)) == 5


def test_the_example_runs(cuda_dev):
    done = subprocess.run([sys.executable, _path, "--d", "256", "--heads", "4", "--keys", "2", "--size", "64", "--tokens", "96",
                           "--new", "4"], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr
    assert "decoded against" in done.stdout and "loss" in done.stdout
