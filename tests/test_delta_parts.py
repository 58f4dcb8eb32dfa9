"""The gradient of a sequence in parts, the last first, each with the state before it
and the gradient that the part behind it leaves: what bounds the workspace."""
from __future__ import annotations

import pytest
import torch

import delta_refs as ref
import memory_bound_gemv_02_gb300 as g
from operator_refs import check, half_ulp
from test_gated_delta_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("heads,dk,dv", [(2, 64, 40), (40, 128, 80)])
def test_gradient_in_parts(cuda_dev, heads, dk, dv, dtype):
    x, h0, do, dstate = make(cuda_dev, 2, 250, heads // 2, heads, dk, dv, dtype, resets=(120,))
    names = ("q", "k", "v", "g", "beta")
    want, tols = ref.backward(do, *(x[n] for n in names), x["scale"], h0, dstate)
    starts, state = [], h0
    ends = (0, 100, 107, 171, 250)
    for a, e in zip(ends, ends[1:]):
        starts.append(state)
        _, state = g.gated_delta(*(x[n][:, a:e] for n in names), x["scale"], h0=state)
    grads, behind = [], dstate
    whole = g.gated_delta_workspace(x["q"], x["k"], x["v"], do)
    for a, e, start in reversed(list(zip(ends, ends[1:], starts))):
        part = [x[n][:, a:e] for n in names]
        assert g.gated_delta_workspace(*part[:3], do[:, a:e]) < whole
        *got, behind = g.gated_delta_backward(do[:, a:e], *part, x["scale"], h0=start, dstate=behind)
        grads.insert(0, got)
    # as much error again from the states that the parts start from
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        a = torch.cat([p[i] for p in grads], 1)
        check(a, want[i], half_ulp(want[i], a.dtype) + 2 * tols[i] + 1e-30, name)
    check(behind, want[5], 2 * tols[5] + 1e-30, "dh0")
