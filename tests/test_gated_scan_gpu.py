"""gated_scan and gated_scan_backward on the GPU against the recurrence walked
in float64, step by step."""
from __future__ import annotations

import pytest
import torch

import memory_bound_gemv_02_gb300 as g
import operator_refs as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float16, torch.bfloat16, torch.float32]
SHAPES = [(1, 1, 1), (1, 1, 64), (3, 1, 4096), (2, 2, 40), (1, 3, 7), (2, 17, 130), (1, 31, 64), (1, 33, 64),
          (3, 64, 72), (2, 100, 257), (1, 255, 96), (2, 511, 33), (1, 1025, 128), (5, 640, 64), (1, 4099, 24),
          (1, 9000, 65), (40, 300, 512)]


def _inputs(b, t, d, dtype, dev, seed, resets=True, lo=-1.5):
    x = ref.uniform((b, t, d), dtype, seed, dev)
    # decays between exp(lo) and 1, squared so that many are near 1
    gate = -ref.uniform((b, t, d), torch.float32, seed + 1, dev, 0, 1) ** 2 * -lo
    if resets and t > 3:
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed + 2)
        gate[torch.rand((b, t, d), generator=gen, device=dev) < 0.01] = float("-inf")
    return x, gate.to(dtype), ref.uniform((b, d), torch.float32, seed + 3, dev, -3, 3)


def _check_forward(x, gate, h0, h, state, label):
    torch.cuda.synchronize()
    h64, tol = ref.gated_scan(x, gate, h0)
    ref.check(h, h64, tol + ref.half_ulp(h64, h.dtype), f"{label} h")
    ref.check(state, h64[:, -1], tol[:, -1] + ref.half_ulp(h64[:, -1], torch.float32), f"{label} state")


def _check_backward(dh, gate, h, h0, dstate, dx, dg, dh0, label):
    torch.cuda.synchronize()
    rx, rg, r0, tx, tg, t0 = ref.gated_scan_backward(dh, gate, h, h0, dstate)
    ref.check(dx, rx, tx + ref.half_ulp(rx, dx.dtype), f"{label} dx")
    ref.check(dg, rg, tg + ref.half_ulp(rg, dg.dtype), f"{label} dg")
    ref.check(dh0, r0, t0 + ref.half_ulp(r0, torch.float32), f"{label} dh0")


@pytest.mark.parametrize("b,t,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_forward(cuda_dev, b, t, d, dtype):
    x, gate, h0 = _inputs(b, t, d, dtype, cuda_dev, t + d)
    h, state = g.gated_scan(x, gate, h0=h0)
    _check_forward(x, gate, h0, h, state, f"{b}x{t}x{d}")
    h, state = g.gated_scan(x, gate)
    _check_forward(x, gate, None, h, state, f"{b}x{t}x{d} from zero")


@pytest.mark.parametrize("b,t,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward(cuda_dev, b, t, d, dtype):
    x, gate, h0 = _inputs(b, t, d, dtype, cuda_dev, t + d)
    dh = ref.uniform((b, t, d), dtype, 7, cuda_dev)
    dstate = ref.uniform((b, d), torch.float32, 8, cuda_dev, -2, 2)
    h, _ = g.gated_scan(x, gate, h0=h0)
    _check_backward(dh, gate, h, h0, dstate, *g.gated_scan_backward(dh, gate, h, h0=h0, dstate=dstate), "full")
    _check_backward(dh, gate, h, None, None, *g.gated_scan_backward(dh, gate, h), "no carries")


def test_backward_against_differences(cuda_dev):
    """The gradient of sum(w h) + sum(v state) by central differences of the
    float64 recurrence: at a step of 1e-6 they are within 1e-7 of the derivative
    here (third derivatives of order 10, cancellation 1e-15 * 1e2 / 1e-6)."""
    b, t, d = 2, 37, 5
    x, gate, h0 = _inputs(b, t, d, torch.float32, cuda_dev, 5, resets=False)
    w, v = ref.uniform((b, t, d), torch.float32, 6, cuda_dev), ref.uniform((b, d), torch.float32, 7, cuda_dev)
    h, _ = g.gated_scan(x, gate, h0=h0)
    dx, dg, dh0 = g.gated_scan_backward(w, gate, h, h0=h0, dstate=v)

    def loss(x_, g_, h0_):
        hh = ref.gated_scan(x_, g_, h0_)[0]
        return float((hh * w.double()).sum() + (hh[:, -1] * v.double()).sum())

    args = [x.double(), gate.double(), h0.double()]
    for k, grad in enumerate((dx, dg, dh0)):
        for seed in range(4):
            direction = ref.uniform(args[k].shape, torch.float64, 60 + seed, cuda_dev)
            up, down = ([a + s * 1e-6 * direction if i == k else a for i, a in enumerate(args)] for s in (1, -1))
            want = (loss(*up) - loss(*down)) / 2e-6
            got = float((grad.double() * direction).sum())
            # fp32 gradients: each entry within 100 u of terms whose sum is below 400
            assert abs(got - want) <= 1e-7 * 100 + 100 * ref.U32 * 400, (k, got, want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [1, 5, 200])
def test_state_in_place(cuda_dev, dtype, t):
    x, gate, h0 = _inputs(3, t, 72, dtype, cuda_dev, 11)
    start = h0.clone()
    h, state = g.gated_scan(x, gate, h0=h0, state=h0)
    assert state is h0
    _check_forward(x, gate, start, h, state, "in place")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,t,d", [(2, 300, 64), (3, 77, 33), (2, 1, 64), (2, 2500, 48)])
def test_strided(cuda_dev, dtype, b, t, d):
    """Halves of one projection, (steps, batch, width) storage and odd offsets."""
    x, gate, h0 = _inputs(b, t, d, dtype, cuda_dev, 13)
    both = torch.cat([x, gate], dim=2)
    out = torch.full((b, t, 2 * d), 7.0, dtype=dtype, device=cuda_dev)
    h, state = g.gated_scan(both[:, :, :d], both[:, :, d:], h0=h0, h=out[:, :, d:])
    _check_forward(x, gate, h0, h, state, "halves")
    assert (out[:, :, :d] == 7).all()
    xt, gt = x.transpose(0, 1).contiguous().transpose(0, 1), gate.transpose(0, 1).contiguous().transpose(0, 1)
    ht = torch.empty((t, b, d), dtype=dtype, device=cuda_dev).transpose(0, 1)
    h2, state2 = g.gated_scan(xt, gt, h0=h0, h=ht)
    _check_forward(x, gate, h0, h2, state2, "steps first")
    # odd element offsets and a padded step stride
    pad = torch.zeros((b, t, d + 5), dtype=dtype, device=cuda_dev)
    pad[:, :, 3:3 + d] = x
    h3, state3 = g.gated_scan(pad[:, :, 3:3 + d], gate, h0=h0)
    _check_forward(x, gate, h0, h3, state3, "padded")
    dh = ref.uniform((b, t, d), dtype, 17, cuda_dev)
    grads = torch.full((b, t, 2 * d), 7.0, dtype=dtype, device=cuda_dev)
    dx, dg, dh0 = g.gated_scan_backward(dh, both[:, :, d:], h, h0=h0, dx=grads[:, :, :d], dg=grads[:, :, d:])
    _check_backward(dh, gate, h, h0, None, dx, dg, dh0, "halves")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t", [1, 700])
def test_expanded_inputs(cuda_dev, dtype, t):
    """One gate shared by all sequences (stride 0) and one row shared by all steps."""
    x, gate, h0 = _inputs(3, t, 64, dtype, cuda_dev, 19)
    shared = gate[:1].expand(3, t, 64)
    h, state = g.gated_scan(x, shared, h0=h0)
    _check_forward(x, shared, h0, h, state, "shared gate")
    row = x[:, :1].expand(3, t, 64)
    h, state = g.gated_scan(row, gate, h0=h0)
    _check_forward(row, gate, h0, h, state, "shared step")
    dx, dg, dh0 = g.gated_scan_backward(row, shared, h, h0=h0)
    _check_backward(row, shared, h, h0, None, dx, dg, dh0, "shared")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("t,cut", [(4, 2), (200, 100), (200, 128), (3000, 1111), (3000, 2048)])
def test_resets_hide_what_was_before(cuda_dev, dtype, t, cut):
    """NaN and infinities before a reset do not reach what follows, and the
    gradient of what follows does not reach back."""
    x, gate, h0 = _inputs(2, t, 64, dtype, cuda_dev, 23, resets=False)
    gate[:, cut] = float("-inf")
    clean_h, clean_state = g.gated_scan(x, gate, h0=h0)
    dirty = x.clone()
    dirty[:, cut - 1, ::3] = float("nan")
    dirty[:, 0, 1::3] = float("inf")
    h, state = g.gated_scan(dirty, gate, h0=torch.full_like(h0, float("inf")))
    assert torch.equal(h[:, cut:], clean_h[:, cut:]) and torch.equal(state, clean_state)
    _check_forward(dirty, gate, torch.full_like(h0, float("inf")), h, state, "dirty")
    dh = ref.uniform((2, t, 64), dtype, 29, cuda_dev)
    late = dh.clone()
    late[:, cut + 1:, ::2] = float("nan")
    dx0, dg0, _ = g.gated_scan_backward(dh, gate, clean_h, h0=h0)
    dx, dg, dh0 = g.gated_scan_backward(late, gate, clean_h, h0=h0)
    assert torch.equal(dx[:, :cut], dx0[:, :cut]) and torch.equal(dg[:, :cut], dg0[:, :cut])
    assert (dg[:, cut] == 0).all()
    # an infinite state before the reset leaves dg there at zero
    bad = clean_h.clone()
    bad[:, cut - 1] = float("inf")
    _, dg, _ = g.gated_scan_backward(dh, gate, bad, h0=h0)
    assert (dg[:, cut] == 0).all()


@pytest.mark.parametrize("t", [6, 400, 3000])
def test_infinite_states_are_carried(cuda_dev, t):
    """Without a reset an infinity stays, however small the decay's product gets;
    NaN spreads; nothing else turns into either."""
    x, gate, _ = _inputs(1, t, 64, torch.float32, cuda_dev, 31, resets=False, lo=-6.0)
    gate = gate - 1.0
    x[:, 1, 0] = float("inf")
    x[:, 1, 1] = float("nan")
    h, state = g.gated_scan(x, gate)
    torch.cuda.synchronize()
    assert torch.isinf(h[:, 1:, 0]).all() and torch.isinf(state[:, 0]).all()
    assert torch.isnan(h[:, 1:, 1]).all()
    _check_forward(x[:, :, 2:].contiguous(), gate[:, :, 2:].contiguous(), None, h[:, :, 2:], state[:, 2:], "others")


@pytest.mark.parametrize("dtype", TYPES)
def test_growth_and_zero_decay(cuda_dev, dtype):
    """Positive gates (growth) and gates whose exponential underflows to zero."""
    x, gate, h0 = _inputs(2, 130, 64, dtype, cuda_dev, 37, resets=False)
    gate[:, ::2] = 0.05
    gate[:, 40, 5:9] = -200.0
    h, state = g.gated_scan(x, gate, h0=h0)
    _check_forward(x, gate, h0, h, state, "growth")
    # growth without bound over a state of zeros stays zero
    zeros = torch.zeros((1, 2000, 64), dtype=dtype, device=cuda_dev)
    h, state = g.gated_scan(zeros, torch.full_like(zeros, 5.0))
    assert (h == 0).all() and (state == 0).all()


def test_empty(cuda_dev):
    h0 = ref.uniform((2, 8), torch.float32, 1, cuda_dev)
    none = torch.empty((2, 0, 8), device=cuda_dev)
    h, state = g.gated_scan(none, none, h0=h0)
    assert h.shape == (2, 0, 8) and torch.equal(state, h0)
    assert (g.gated_scan(none, none)[1] == 0).all()
    _, _, dh0 = g.gated_scan_backward(none, none, none, h0=h0, dstate=h0 + 1)
    assert torch.equal(dh0, h0 + 1)
    for shape in ((0, 4, 8), (2, 4, 0)):
        e = torch.empty(shape, device=cuda_dev)
        assert g.gated_scan(e, e)[0].shape == shape


def test_repeatable_and_on_a_stream(cuda_dev):
    x, gate, h0 = _inputs(2, 5000, 96, torch.bfloat16, cuda_dev, 41)
    dh = ref.uniform(x.shape, torch.bfloat16, 43, cuda_dev)
    h, state = g.gated_scan(x, gate, h0=h0)
    grads = g.gated_scan_backward(dh, gate, h, h0=h0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(s):
            h2, state2 = g.gated_scan(x, gate, h0=h0)
            grads2 = g.gated_scan_backward(dh, gate, h2, h0=h0)
        s.synchronize()
        assert torch.equal(h, h2) and torch.equal(state, state2)
        assert all(torch.equal(p, q) for p, q in zip(grads, grads2))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("b,t,d", [(2, 40, 96), (25, 12, 640), (1, 3000, 512), (2, 700, 65), (3, 300, 2048)])
def test_calls_back_to_back(cuda_dev, dtype, b, t, d):
    """Calls on two sets of inputs in turn, nothing waited for between them: every
    one gives what it gives alone, and no input changes."""
    sets = [_inputs(b, t, d, dtype, cuda_dev, 71 + 10 * i) for i in range(2)]
    dhs = [ref.uniform((b, t, d), dtype, 91 + i, cuda_dev) for i in range(2)]
    kept = [[v.clone() for v in s] for s in sets]
    alone = []
    for (x, gate, h0), dh in zip(sets, dhs):
        h, state = g.gated_scan(x, gate, h0=h0)
        torch.cuda.synchronize()
        grads = g.gated_scan_backward(dh, gate, h, h0=h0, dstate=state)
        torch.cuda.synchronize()
        alone.append((h, state, *grads))
    outs = [[torch.empty_like(v) for v in a] for a in alone]
    for i in (0, 1, 0, 1, 0):
        (x, gate, h0), (h, state, dx, dg, dh0) = sets[i], outs[i]
        g.gated_scan(x, gate, h0=h0, h=h, state=state)
        g.gated_scan_backward(dhs[i], gate, h, h0=h0, dstate=state, dx=dx, dg=dg, dh0=dh0)
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        assert all(torch.equal(p, q) for p, q in zip(a, o))
    assert all(torch.equal(p, q) for s, k in zip(sets, kept) for p, q in zip(s, k))


@pytest.mark.parametrize("b,t,d", [(2, 700, 64), (1, 5000, 512), (2, 700, 65), (40, 200, 512)])
def test_a_wait_that_gives_up(cuda_dev, b, t, d):
    """Waits for copies given no polls: the calls return, their outputs are NaN, the
    counter says so, and the next calls are right."""
    x, gate, h0 = _inputs(b, t, d, torch.bfloat16, cuda_dev, 53)
    dh = ref.uniform(x.shape, torch.bfloat16, 59, cuda_dev)
    torch.cuda.synchronize()
    g.gemv_wait_timeouts(reset=True)
    g.gemv_debug_wait_budget(0)
    h, _ = g.gated_scan(x, gate, h0=h0)
    torch.cuda.synchronize()
    assert torch.isnan(h).all() and g.gemv_wait_timeouts(reset=True) > 0
    h, state = g.gated_scan(x, gate, h0=h0)
    _check_forward(x, gate, h0, h, state, "after")
    g.gemv_debug_wait_budget(0)
    dx, dg, _ = g.gated_scan_backward(dh, gate, h, h0=h0)
    torch.cuda.synchronize()
    assert torch.isnan(dx).all() and torch.isnan(dg).all() and g.gemv_wait_timeouts(reset=True) > 0
    _check_backward(dh, gate, h, h0, None, *g.gated_scan_backward(dh, gate, h, h0=h0), "after")
    assert g.gemv_wait_timeouts() == 0


def test_refusals(cuda_dev):
    x, gate, h0 = _inputs(2, 6, 16, torch.bfloat16, cuda_dev, 47)
    with pytest.raises(TypeError):
        g.gated_scan(x, gate.float())
    with pytest.raises(TypeError):
        g.gated_scan(x, gate, h0=h0.half())
    with pytest.raises(TypeError):
        g.gated_scan(x.double(), gate.double())
    with pytest.raises(ValueError):
        g.gated_scan(x, gate[:, :5])
    with pytest.raises(ValueError):
        g.gated_scan(x.transpose(1, 2), gate.transpose(1, 2))
    with pytest.raises(ValueError):
        g.gated_scan(x.cpu(), gate.cpu())
    with pytest.raises(ValueError):
        g.gated_scan(x, gate, h0=h0[:, :8])
    for kw in ({"h": x}, {"h": gate}):
        with pytest.raises(g.GemvError) as e:
            g.gated_scan(x, gate, **kw)
        assert e.value.status == g.GEMV_ERR_ALIAS
    with pytest.raises(g.GemvError) as e:  # an output whose rows coincide
        g.gated_scan(x, gate, h=torch.empty((2, 1, 16), dtype=torch.bfloat16, device=cuda_dev).expand(2, 6, 16))
    assert e.value.status == g.GEMV_ERR_ARG
    both = torch.empty((2, 6, 16), dtype=torch.bfloat16, device=cuda_dev)
    with pytest.raises(g.GemvError) as e:
        g.gated_scan_backward(x, gate, x.clone(), dx=both, dg=both)
    assert e.value.status == g.GEMV_ERR_ALIAS
