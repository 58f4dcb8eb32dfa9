"""gated_delta() and its gradient where a size of 0 leaves outputs that are empty
sums: they are zeros, as the epilogue of 0 is for a product with k == 0."""
from __future__ import annotations

import pytest
import torch

from test_delta_norm_abi import P, _delta

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def test_outputs_of_empty_sums_are_not_passed_over(gemv_lib):
    """Without a GPU: the call goes on to the device (fake pointers are none of its),
    unless none of its outputs has an element; what is wrong with them is refused first."""
    g, L = gemv_lib, gemv_lib._lib_with_operators()
    refused = (g.GEMV_ERR_ARG, g.GEMV_ERR_ALIAS, g.GEMV_ERR_ALIGN, g.GEMV_ERR_DTYPE, g.GEMV_ERR_SCRATCH)
    cases = [(False, {"dk": 0}, (6,)), (True, {"dk": 0}, (10, 11, 12)), (True, {"dv": 0}, (8, 9, 11, 12)),
             (True, {"heads": 0}, (8, 9)), (True, {"dk": 0, "dv": 0}, (11, 12))]
    for back, shape, outs in cases:
        st = _delta(g, L, back, shape=shape)
        assert st != g.GEMV_OK and st not in refused, (back, shape)
        # (null outputs are left out, empty ones are never written)
        assert _delta(g, L, back, {i: None for i in outs}, shape=shape) == g.GEMV_OK
        for i in outs:
            assert _delta(g, L, back, {i: P[i] + 1}, shape=shape) == g.GEMV_ERR_ALIGN, (i, shape)
            assert _delta(g, L, back, strides={i: (0, 512, 64)}, shape=shape) == g.GEMV_ERR_ARG, (i, shape)
            assert _delta(g, L, back, strides={i: (-1, 8, 1)}, shape=shape) == g.GEMV_ERR_ARG, (i, shape)
        if back:
            assert _delta(g, L, back, {outs[0]: P[outs[1]]}, shape=shape) == g.GEMV_ERR_ALIAS, shape
    assert _delta(g, L, False, {6: P[2]}, shape={"dk": 0}) == g.GEMV_ERR_ALIAS
    assert _delta(g, L, True, {10: P[6]}, shape={"dk": 0}) == g.GEMV_ERR_ALIAS
    assert _delta(g, L, True, shape={"heads": 0, "heads_k": 65536}) == g.GEMV_ERR_ARG
    for back, shape in ((False, {"dv": 0}), (False, {"heads": 0}), (True, {"batch": 0}), (True, {"dk": 0, "steps": 0}),
                        (True, {"heads": 0, "heads_k": 0}), (True, {"heads": 0, "dk": 0})):
        assert _delta(g, L, back, shape=shape) == g.GEMV_OK, (back, shape)


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 70])
@pytest.mark.parametrize("dtype,gates", [(BF16, F32), (F16, F16)])
@pytest.mark.parametrize("hk,h,dk,dv", [(2, 4, 0, 24), (2, 4, 16, 0), (2, 0, 16, 24), (2, 4, 0, 0), (1, 1, 0, 1)])
def test_empty_sums_are_zero(cuda_dev, hk, h, dk, dv, dtype, gates, steps):
    """Into outputs that held something, dense and as columns of a matrix whose others stay."""
    import memory_bound_gemv_02_gb300 as g
    b = 3
    one = lambda *s, t=dtype: torch.ones(s, dtype=t, device=cuda_dev)  # noqa: E731
    q, k, v, do = one(b, steps, hk, dk), one(b, steps, hk, dk), one(b, steps, h, dv), one(b, steps, h, dv)
    gate, beta = -one(b, steps, h, t=gates), one(b, steps, h, t=gates)
    h0, dstate = one(b, h, dk, dv, t=F32), one(b, h, dk, dv, t=F32)
    o, state = g.gated_delta(q, k, v, gate, beta, 0.5, h0=h0, o=torch.full_like(v, 7.0))
    assert o.shape == v.shape and (o == 0).all() and state.numel() == 0
    names, like = ("dq", "dk", "dv", "dg", "dbeta"), (q, k, v, gate, beta)
    got = g.gated_delta_backward(do, q, k, v, gate, beta, 0.5, h0=h0, dstate=dstate,
                                 **{n: torch.full_like(t, 7.0) for n, t in zip(names, like)})
    for n, a, t in zip(names, got, like):
        assert a.shape == t.shape and (a == 0).all(), n
    wide = {n: torch.full((*t.shape[:2], 2 * t.shape[2] + 1, *t.shape[3:]), 7.0, dtype=t.dtype, device=cuda_dev)
            for n, t in zip((*names, "o"), (*like, v))}
    part = {n: w[:, :, 1::2] for n, w in wide.items()}
    g.gated_delta(q, k, v, gate, beta, 0.5, h0=h0, o=part.pop("o"))
    g.gated_delta_backward(do, q, k, v, gate, beta, 0.5, h0=h0, dstate=dstate, **part)
    for n, w in wide.items():
        assert (w[:, :, 1::2] == 0).all() and (w[:, :, ::2] == 7).all(), n


@pytest.mark.gpu
def test_empty_sums_in_a_graph(cuda_dev):
    import memory_bound_gemv_02_gb300 as g
    q, v = torch.ones((2, 30, 1, 0), dtype=BF16, device=cuda_dev), torch.ones((2, 30, 2, 40), dtype=BF16, device=cuda_dev)
    gate, o = torch.zeros((2, 30, 2), device=cuda_dev), torch.empty_like(v)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g.gated_delta(q, q, v, gate, gate, 1.0, o=o)
    o.fill_(5.0)
    graph.replay()
    assert (o == 0).all()
