"""gated_delta() and gated_delta_backward() against the rule step by step in float64."""
from __future__ import annotations

import threading

import pytest
import torch

import delta_refs as ref
import memory_bound_gemv_02_gb300 as g
from operator_refs import check, half_ulp

pytestmark = pytest.mark.gpu

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def make(dev, b, t, hk, h, dk, dv, dtype, gates=F32, seed=0, resets=()):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed + t + 10 * dk)
    r = lambda *s: torch.randn(s, generator=gen, device=dev)  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-9)  # noqa: E731
    x = {"q": unit(r(b, t, hk, dk)).to(dtype), "k": unit(r(b, t, hk, dk)).to(dtype), "v": r(b, t, h, dv).to(dtype),
         "g": (-r(b, t, h).abs() * 0.2).to(gates), "beta": torch.sigmoid(r(b, t, h)).to(gates)}
    for i in resets:
        x["g"][:, i] = float("-inf")
    x["scale"] = dk ** -0.5
    return x, r(b, h, dk, dv), r(b, t, h, dv).to(dtype), 0.3 * r(b, h, dk, dv)


def check_forward(x, h0, o, state, label=""):
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want, last, tol, tol_s = ref.forward(*args, x["scale"], h0)
    check(o, want, half_ulp(want, o.dtype) + tol, label + " o")
    check(state, last, tol_s + 1e-30, label + " state")


def check_backward(x, h0, do, dstate, got, label=""):
    args = [x[n] for n in ("q", "k", "v", "g", "beta")]
    want, tols = ref.backward(do, *args, x["scale"], h0, dstate)
    for name, a, w, tol in zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), got, want, tols):
        check(a, w, half_ulp(w, a.dtype) + tol + 1e-30, f"{label} {name}")


def run(x, h0=None, **kw):
    return g.gated_delta(x["q"], x["k"], x["v"], x["g"], x["beta"], x["scale"], h0=h0, **kw)


def run_back(x, do, h0=None, dstate=None, **kw):
    return g.gated_delta_backward(do, x["q"], x["k"], x["v"], x["g"], x["beta"], x["scale"], h0=h0, dstate=dstate, **kw)


SIZES = [  # batch, steps, heads of k, of v, dk, dv
    (1, 1, 1, 1, 1, 1), (2, 1, 2, 4, 128, 128), (3, 2, 1, 3, 17, 5), (1, 7, 2, 2, 256, 130), (2, 12, 1, 2, 64, 33), (2, 13, 2, 2, 72, 40),
    (1, 49, 1, 1, 128, 128), (2, 63, 2, 2, 64, 64), (1, 64, 1, 2, 96, 72), (1, 65, 2, 2, 128, 200), (2, 128, 1, 1, 256, 64),
    (1, 129, 1, 3, 40, 8), (1, 200, 2, 4, 100, 99), (1, 300, 1, 1, 255, 31), (1, 193, 1, 1, 1, 3)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,gates", [(BF16, F32), (F16, F16), (BF16, BF16), (F16, F32)])
def test_forward(cuda_dev, size, dtype, gates):
    x, h0, _, _ = make(cuda_dev, *size, dtype, gates)
    o, state = run(x, h0)
    check_forward(x, h0, o, state)
    o, state = run(x)
    check_forward(x, None, o, state, "from zero")


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype,gates", [(BF16, F32), (F16, F16)])
def test_backward(cuda_dev, size, dtype, gates):
    x, h0, do, dstate = make(cuda_dev, *size, dtype, gates)
    check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate))
    check_backward(x, None, do, None, run_back(x, do), "without states")


MANY = [  # enough heads for a CTA of wide columns each
    (4, 64, 2, 6, 128, 128), (4, 70, 6, 6, 128, 128), (2, 200, 10, 10, 100, 99), (5, 129, 5, 5, 72, 200),
    (4, 70, 5, 10, 128, 128), (5, 193, 8, 8, 100, 99), (8, 129, 3, 6, 65, 130), (3, 193, 4, 8, 65, 128), (20, 49, 1, 2, 128, 65), (4, 130, 3, 9, 64, 128), (3, 100, 8, 8, 256, 96)]


@pytest.mark.parametrize("size", MANY)
@pytest.mark.parametrize("dtype,gates", [(BF16, F32), (F16, F32), (BF16, BF16)])
def test_many_heads(cuda_dev, size, dtype, gates):
    x, h0, do, dstate = make(cuda_dev, *size, dtype, gates, resets=(size[1] // 3,))
    o, state = run(x, h0)
    check_forward(x, h0, o, state)
    check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate))
    o, state = run(x)
    check_forward(x, None, o, state, "from zero")


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 9, 16])
@pytest.mark.parametrize("dk", [40, 128, 200])
def test_gradients_of_shared_heads(cuda_dev, group, dk):
    x, h0, do, dstate = make(cuda_dev, 1, 100, 2, 2 * group, dk, 32, BF16)
    check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate))


@pytest.mark.parametrize("steps,resets", [(40, (0, 1, 39)), (200, (0,)), (200, (63, 64, 65)), (200, (128, 199)),
                                          (130, tuple(range(130))), (300, (17, 100, 101, 256))])
def test_new_documents(cuda_dev, steps, resets):
    """Nothing passes a new document, in either direction, not even a large state."""
    x, h0, do, dstate = make(cuda_dev, 2, steps, 1, 2, 64, 40, BF16, resets=resets)
    o, state = run(x, 1e4 * h0 if resets[0] == 0 else h0)
    start = resets[0]
    check_forward(x, None if start == 0 else h0, o, state)
    got = run_back(x, do, h0, dstate)
    check_backward(x, h0, do, dstate, got)
    assert (got[3][:, list(resets)] == 0).all()
    if start == 0:
        assert (got[5] == 0).all()


@pytest.mark.parametrize("steps", [20, 150])
@pytest.mark.parametrize("low", [-1e4, -88.0, torch.finfo(F32).min])
def test_decays_that_vanish(cuda_dev, steps, low):
    x, h0, do, dstate = make(cuda_dev, 1, steps, 1, 1, 32, 32, BF16)
    x["g"][:, steps // 2] = low
    o, state = run(x, h0)
    check_forward(x, h0, o, state)
    check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate))


@pytest.mark.parametrize("steps", [30, 200])
def test_strong_and_absent_decays(cuda_dev, steps):
    """Decays of exp(-60) step after step, whose sums pass any range, and none at all."""
    for level in (-60.0, -3.0, 0.0):
        x, h0, do, dstate = make(cuda_dev, 1, steps, 1, 2, 64, 64, BF16)
        x["g"].fill_(level)
        o, state = run(x, h0)
        check_forward(x, h0, o, state, f"g = {level}")
        check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate), f"g = {level}")


@pytest.mark.parametrize("heads", [1, 24])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("size", [1e6, 1e-6, 1e30, 0.0])
def test_states_beyond_their_inputs_range(cuda_dev, heads, dtype, size):
    """States (and gradients of the last) far above and below what fp16 holds; beta
    of 0 leaves v out where it would be lost beside them."""
    x, h0, do, dstate = make(cuda_dev, 1, 140, heads, heads, 64, 48, dtype)
    h0, dstate = h0 * size, dstate * size
    x["scale"] = min(1.0, 0.1 / size) if size else 1.0  # o within its type
    o, state = run(x, h0)
    check_forward(x, h0, o, state)
    x["scale"] = min(x["scale"], 1e-3)
    do = do * min(1.0, 1e3 * size) if size < 1 else do
    x["v"].zero_()
    dv_scale = 1.0 if size <= 1e3 else 1e3 / size  # dv and dk within theirs
    got = run_back(x, do, h0 * dv_scale, dstate * dv_scale)
    check_backward(x, h0 * dv_scale, do, dstate * dv_scale, got)


def test_heads_do_not_meet(cuda_dev):
    """A NaN in one head's v leaves the other heads' bits as they were, and what is not
    a step of the call is not read."""
    x, h0, do, dstate = make(cuda_dev, 2, 150, 2, 4, 64, 64, BF16)
    want = (*run(x, h0), *run_back(x, do, h0, dstate))
    y = {**x, "v": x["v"].clone()}
    y["v"][1, 70, 2] = float("nan")
    got = (*run(y, h0), *run_back(y, do, h0, dstate))
    for i, heads in ((0, 4), (1, 4), (4, 4), (5, 4), (6, 4), (7, 4)):  # o, state, dv, dg, dbeta, dh0
        a, b = (t[i] if i in (1, 7) else t[i].transpose(1, 2) for t in (got, want))
        keep = torch.ones((2, heads), dtype=torch.bool, device=cuda_dev)
        keep[1, 2] = False
        assert torch.equal(a[keep], b[keep]), i
    long = torch.full((2, 200, 2 * 128 + 256), float("nan"), dtype=BF16, device=cuda_dev)
    for n, at, heads in (("q", 0, 2), ("k", 128, 2), ("v", 256, 4)):
        part = long[:, :150, at:at + heads * 64].unflatten(2, (heads, 64))
        part.copy_(x[n])
        y[n] = part
    got = (*run(y, h0), *run_back(y, do, h0, dstate))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("steps", [30, 200])
def test_gates_at_their_ends(cuda_dev, steps):
    """beta of 0 (nothing written; its gradient is there), 1 with equal keys, and 2."""
    x, h0, do, dstate = make(cuda_dev, 1, steps, 1, 1, 48, 32, BF16)
    for beta, same in ((0.0, False), (1.0, True), (2.0, False)):
        x["beta"].fill_(beta)
        if same:
            x["k"].copy_(x["k"][:, :1].expand_as(x["k"]).clone())
        elif beta == 2.0:  # |k|^2 rounded to at most 1
            x["k"].copy_((x["k"].float() * 0.99).to(BF16))
        o, state = run(x, h0)
        check_forward(x, h0, o, state, f"beta {beta}")
        check_backward(x, h0, do, dstate, run_back(x, do, h0, dstate), f"beta {beta}")


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("steps", [5, 140])
def test_parts_of_one_projection(cuda_dev, dtype, steps):
    """q, k and v as columns of one matrix, (heads, steps) storage, shared rows, odd offsets;
    elements around the outputs stay."""
    b, hk, h, dk, dv = 2, 2, 4, 64, 32
    x, h0, do, dstate = make(cuda_dev, b, steps, hk, h, dk, dv, dtype)
    for shift in (0, 3):
        wide = torch.zeros((b, steps, 2 * hk * dk + h * dv + 11), dtype=dtype, device=cuda_dev)
        qv = wide[..., shift:shift + hk * dk].unflatten(2, (hk, dk))
        kv = wide[..., shift + hk * dk:shift + 2 * hk * dk].unflatten(2, (hk, dk))
        vv = wide[..., shift + 2 * hk * dk:shift + 2 * hk * dk + h * dv].unflatten(2, (h, dv))
        for view, name in ((qv, "q"), (kv, "k"), (vv, "v")):
            view.copy_(x[name])
        gates = torch.stack([x["g"], x["beta"]], dim=-1)
        y = {**x, "q": qv, "k": kv, "v": vv, "g": gates[..., 0], "beta": gates[..., 1]}
        out = torch.full((b, h, steps + 2, dv + shift), 7.0, dtype=dtype, device=cuda_dev)
        o = out[:, :, 1:steps + 1, shift:].transpose(1, 2)
        _, state = run(y, h0, o=o)
        check_forward(x, h0, o, state, f"shift {shift}")
        assert (out[:, :, 0] == 7).all() and (out[:, :, -1] == 7).all() and (out[..., :shift] == 7).all()
        grads = torch.full_like(wide, 7.0)
        dq = grads[..., shift:shift + hk * dk].unflatten(2, (hk, dk))
        dk_ = grads[..., shift + hk * dk:shift + 2 * hk * dk].unflatten(2, (hk, dk))
        dv_ = grads[..., shift + 2 * hk * dk:shift + 2 * hk * dk + h * dv].unflatten(2, (h, dv))
        got = run_back(y, do.transpose(1, 2).contiguous().transpose(1, 2), h0, dstate, dq=dq, dk=dk_, dv=dv_)
        check_backward(x, h0, do, dstate, got, f"shift {shift}")
        assert (grads[..., :shift] == 7).all() and (grads[..., shift + 2 * hk * dk + h * dv:] == 7).all()
    # one row of v and of the gates for all steps
    y = {**x, "v": x["v"][:, :1].expand_as(x["v"]), "g": x["g"][:, :1].expand_as(x["g"]), "beta": x["beta"][:1].expand_as(x["beta"])}
    o, state = run(y, h0)
    check_forward(y, h0, o, state, "expanded")
    check_backward(y, h0, do, dstate, run_back(y, do, h0, dstate), "expanded")


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_steps_continue_a_prompt(cuda_dev, dtype):
    """A prompt and then single tokens on a state updated in place, as the whole at once."""
    x, h0, _, _ = make(cuda_dev, 2, 150, 2, 4, 64, 64, dtype)
    want, last, tol, tol_s = ref.forward(*(x[n] for n in ("q", "k", "v", "g", "beta")), x["scale"], h0)
    state, outs = h0.clone(), []
    for a, e in ((0, 100), (100, 140), *((t, t + 1) for t in range(140, 150))):
        part = {n: x[n][:, a:e] if n != "scale" else x[n] for n in x}
        o, s = run(part, state, state=state)
        assert s is state
        outs.append(o)
    o = torch.cat(outs, 1)
    check(o, want, half_ulp(want, dtype) + 2 * tol, "o")
    check(state, last, 2 * tol_s, "state")


def test_in_place_gradient_of_the_state(cuda_dev):
    x, h0, do, dstate = make(cuda_dev, 1, 100, 1, 2, 64, 64, BF16)
    want = run_back(x, do, h0, dstate)
    kept = dstate.clone()
    got = run_back(x, do, h0, kept, dh0=kept)
    assert got[5] is kept and all(torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_to_do(cuda_dev):
    x, h0, do, dstate = make(cuda_dev, 2, 0, 1, 2, 16, 8, BF16)
    o, state = run(x, h0)
    assert o.shape == (2, 0, 2, 8) and torch.equal(state, h0)
    _, state = run(x)
    assert (state == 0).all()
    *_, dh0 = run_back(x, do, h0, dstate)
    assert torch.equal(dh0, dstate)
    *_, dh0 = run_back(x, do, h0)
    assert (dh0 == 0).all()
    for size in ((0, 70, 1, 1, 16, 8), (1, 70, 1, 1, 16, 0)):
        x, h0, do, dstate = make(cuda_dev, *size, BF16)
        run(x, h0)
        run_back(x, do, h0, dstate)


def test_repeats_bitwise_and_in_two_graphs(cuda_dev):
    """Calls on two streams at once and in two captured graphs, each with its workspace,
    give the same bits."""
    x, h0, do, dstate = make(cuda_dev, 2, 190, 2, 4, 128, 128, BF16)
    o, state = run(x, h0)
    grads = run_back(x, do, h0, dstate)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    results = []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                results.append((*run(x, h0), *run_back(x, do, h0, dstate)))
    torch.cuda.synchronize()
    for r in results:
        assert all(torch.equal(a, b) for a, b in zip(r, (o, state, *grads)))
    graphs = []
    for s in streams:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = (*run(x, h0), *run_back(x, do, h0, dstate))
        graphs.append((graph, out))
    for graph, out in graphs:
        for t in out:
            t.fill_(3)
    torch.cuda.synchronize()
    for (graph, _), s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, (o, state, *grads)))


def test_streams_and_threads(cuda_dev):
    """A stream of the caller's while other work is pending, and host threads at once."""
    x, h0, do, dstate = make(cuda_dev, 1, 130, 1, 2, 64, 64, BF16)
    want = (*run(x, h0), *run_back(x, do, h0, dstate))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)
    got = (*run(x, h0, stream=side), *run_back(x, do, h0, dstate, stream=side))
    side.synchronize()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(10):
                    got = (*run(x, h0), *run_back(x, do, h0, dstate))
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert not bad


def test_a_given_workspace(cuda_dev):
    x, h0, do, dstate = make(cuda_dev, 1, 130, 1, 2, 40, 24, F16)
    want = (*run(x, h0), *run_back(x, do, h0, dstate))
    for back in (False, True):
        size = g.gated_delta_workspace(x["q"], x["k"], x["v"], do if back else None)
        room = torch.full((size + 512,), 9, dtype=torch.uint8, device=cuda_dev)
        ws = room[256:256 + size]
        got = run_back(x, do, h0, dstate, workspace=ws) if back else run(x, h0, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want[2:] if back else want[:2]))
        assert (room[:256] == 9).all() and (room[256 + size:] == 9).all()
        with pytest.raises(g.GemvError) as e:
            (run_back(x, do, h0, dstate, workspace=ws[:-1]) if back else run(x, h0, workspace=ws[:-1]))
        assert e.value.status == g.GEMV_ERR_SCRATCH
    y, h0, _, _ = make(cuda_dev, 1, 12, 1, 2, 40, 24, F16)
    assert g.gated_delta_workspace(y["q"], y["k"], y["v"]) == 0


def test_refusals(cuda_dev):
    x, h0, do, dstate = make(cuda_dev, 1, 70, 2, 4, 32, 32, BF16)
    bad = [
        {**x, "q": x["q"].float()}, {**x, "k": x["k"].half()}, {**x, "v": x["v"].float()}, {**x, "beta": x["beta"].half()},
        {**x, "g": x["g"].double()}, {**x, "g": x["g"].bfloat16()}]
    for y in bad:
        with pytest.raises(TypeError):
            run(y, h0)
    for y in ({**x, "q": x["q"][:, :-1]}, {**x, "k": x["k"][..., :-1]}, {**x, "v": x["v"][:, :, :3]},
              {**x, "q": x["q"].transpose(2, 3).contiguous().transpose(2, 3)}, {**x, "g": x["g"][..., :-1]},
              {**x, "q": x["q"].cpu()}, {**x, "v": x["v"][0]}):
        with pytest.raises(ValueError):
            run(y, h0)
    with pytest.raises(ValueError):
        run(x, h0[:, :, :-1])
    with pytest.raises(ValueError):
        run(x, h0.transpose(2, 3))
    with pytest.raises(TypeError):
        run(x, h0.bfloat16())
    for kw in ({"o": x["v"]}, {"o": x["v"][:, :, :1].expand_as(x["v"])}):
        with pytest.raises(g.GemvError) as e:
            run(x, h0, **kw)
        assert e.value.status in (g.GEMV_ERR_ALIAS, g.GEMV_ERR_ARG)
    for kw in ({"dq": x["q"]}, {"dv": do}, {"dg": x["beta"]}, {"dh0": h0}):
        with pytest.raises(g.GemvError) as e:
            run_back(x, do, h0, dstate, **kw)
        assert e.value.status == g.GEMV_ERR_ALIAS
    y, h0, _, _ = make(cuda_dev, 1, 2, 1, 1, 257, 8, BF16)
    with pytest.raises(g.GemvError) as e:
        run(y, h0)
    assert e.value.status == g.GEMV_ERR_ARG


@pytest.mark.parametrize("size", [(4, 130, 10, 10, 128, 128)])
def test_a_wait_that_gives_up(cuda_dev, size):
    """Waits without a poll: NaN instead of a hang, a count, and nothing left behind."""
    x, h0, do, dstate = make(cuda_dev, *size, BF16)
    want = (*run(x, h0), *run_back(x, do, h0, dstate))
    torch.cuda.synchronize()
    g.gemv_wait_timeouts(reset=True)
    for back in (False, True):
        g.gemv_debug_wait_budget(0)
        got = run_back(x, do, h0, dstate) if back else run(x, h0)
        torch.cuda.synchronize()
        assert torch.isnan(got[-1]).all() and torch.isnan(got[0].float()).all()
        assert g.gemv_wait_timeouts(reset=True) > 0
    g.gemv_debug_wait_budget(-1)
    got = (*run(x, h0), *run_back(x, do, h0, dstate))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
