"""Cases of the layer operators around the matrix-vector product: the residual
addition with a root-mean-square norm and an 8-bit output, the matrix product
of several vectors with its epilogue, and the gated linear recurrence over a
sequence with its gradient.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end) or, where ``own`` is set, through the package's entry points; ``exact``
computes the same outputs from the definitions in float64.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6


def listed():
    return [
        # one decoded token's residual stream, quantised for the next projection: pure latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16", "residual": True, "eight": True},
        # a prompt of 8192 tokens, residual added, 8-bit output with its row scales
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "d": 7168, "dtype": "bf16", "residual": True, "eight": True},
        # rows of odd length (no row but the first is 16-byte aligned), 16-bit output, no residual
        {"name": "norm_odd_rows", "op": "norm", "rows": 1001, "d": 7169, "dtype": "f16", "residual": False, "eight": False},
        # one token through a square projection: the weights' stream, latency counts
        {"name": "gemm_one_token", "op": "gemm", "m": 1, "n": 4096, "k": 4096, "dtype": "bf16", "bias": True,
         "act": "silu", "residual": True},
        # sixteen sequences decoded together on 8-bit weights and activations
        {"name": "gemm_decode_16", "op": "gemm", "m": 16, "n": 14336, "k": 4096, "dtype": "e4m3", "bias": False,
         "act": "silu", "residual": False},
        # a ragged batch over a matrix whose rows are nowhere aligned
        {"name": "gemm_ragged", "op": "gemm", "m": 77, "n": 4099, "k": 7169, "dtype": "f16", "bias": True,
         "act": "relu", "residual": False},
        # a prompt through the wide projection, 16-bit
        {"name": "gemm_prompt", "op": "gemm", "m": 8192, "n": 14336, "k": 4096, "dtype": "bf16", "bias": True,
         "act": "silu", "residual": False},
        # the same prompt back to the residual stream, 8-bit operands
        {"name": "gemm_prompt_8bit", "op": "gemm", "m": 8192, "n": 4096, "k": 14336, "dtype": "e4m3", "bias": False,
         "act": "none", "residual": True},
        # one decoded token for 64 sequences: the recurrence's single step
        {"name": "scan_one_token", "op": "scan", "b": 64, "t": 1, "d": 4096, "dtype": "bf16", "backward": False},
        # a batch of prompts, forward
        {"name": "scan_prompts", "op": "scan", "b": 4, "t": 8192, "d": 4096, "dtype": "bf16", "backward": False},
        # the same batch's gradient
        {"name": "scan_prompts_grad", "op": "scan", "b": 4, "t": 8192, "d": 4096, "dtype": "bf16", "backward": True},
        # one long document over few channels: the sequence itself has to be split; odd length and width
        {"name": "scan_long_grad", "op": "scan", "b": 1, "t": 65537, "d": 1001, "dtype": "f16", "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _align(rng, v):
    """Half of the sizes are multiples of 64, as models choose them; the rest are left as drawn."""
    return max(64, v // 64 * 64) if v > 64 and rng.random() < 0.5 else v


def draw(rng):
    op = rng.choice(["norm", "gemm", "gemm", "scan", "scan"])
    if op == "norm":
        d = _align(rng, _log_int(rng, 64, 16384))
        rows = _log_int(rng, 1, min(65536, 8192 * 7168 // d))
        return {"op": op, "rows": rows, "d": d, "dtype": rng.choice(["f16", "bf16", "bf16", "f32"]),
                "residual": rng.random() < 0.7, "eight": rng.random() < 0.6}
    if op == "gemm":
        n, k = _align(rng, _log_int(rng, 128, 18433)), _align(rng, _log_int(rng, 128, 16384))
        m = _log_int(rng, 1, min(8192, 8192 * 14336 * 4096 // (n * k)))
        return {"op": op, "m": m, "n": n, "k": k, "dtype": rng.choice(["f16", "bf16", "e4m3"]),
                "bias": rng.random() < 0.5, "act": rng.choice(["none", "relu", "silu", "log_sigmoid"]),
                "residual": rng.random() < 0.4}
    d = _align(rng, _log_int(rng, 64, 8192))
    b = _log_int(rng, 1, 64)
    t = 1 if rng.random() < 0.15 else _log_int(rng, 2, min(65537, 4 * 8192 * 4096 // (b * d)))
    return {"op": op, "b": b, "t": t, "d": d, "dtype": rng.choice(["f16", "bf16", "bf16", "f32"]),
            "backward": t > 1 and rng.random() < 0.5}


def _quantise_rows(x):
    scale = x.abs().amax(dim=1) / E4M3_MAX
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    td = TYPES[case["dtype"]]

    def normal(*shape, sigma=1.0, mean=0.0):
        return torch.randn(shape, generator=gen, device=dev) * sigma + mean

    s = {"case": case}
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        s["x"] = normal(rows, d).to(td)
        s["weight"] = normal(d, sigma=0.1, mean=1.0).to(td)
        # the residual stream of a deep model: several times an increment's size
        s["residual"] = normal(rows, d, sigma=4.0).to(td) if case["residual"] else None
        s["y"] = torch.empty((rows, d), device=dev, dtype=torch.float8_e4m3fn if case["eight"] else td)
        s["scale"] = torch.empty(rows, device=dev) if case["eight"] else None
        s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
    elif case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        od = torch.bfloat16 if case["dtype"] == "e4m3" else td
        B, A = normal(n, k, sigma=0.02), normal(m, k)
        s["scale_a"] = s["scale_b"] = None
        if case["dtype"] == "e4m3":
            s["B"], s["scale_b"] = _quantise_rows(B)
            s["A"], s["scale_a"] = _quantise_rows(A)
        else:
            s["B"], s["A"] = B.to(td), A.to(td)
        s["bias"] = normal(n, sigma=0.1) if case["bias"] else None
        s["residual"] = normal(m, n).to(od) if case["residual"] else None
        s["c"] = torch.empty((m, n), device=dev, dtype=od)
    else:
        b, t, d = case["b"], case["t"], case["d"]
        # the log of a sigmoid gate whose half-lives run from one step to some hundreds
        z = normal(b, t, d, sigma=1.0) + torch.linspace(0.0, 6.0, d, device=dev)
        g = -torch.log1p(torch.exp(-z))
        if t > 64:  # packed documents: nothing is carried into the first token of each
            starts = torch.rand((b, t, 1), generator=gen, device=dev) < 1.0 / 2048
            g = torch.where(starts, float("-inf"), g)
        s["g"] = g.to(td)
        s["h0"] = normal(b, d)
        if case["backward"]:
            s["dh"] = normal(b, t, d).to(td)
            s["h"] = normal(b, t, d).to(td)  # the states that the forward pass kept
            s["dstate"] = normal(b, d)
            s["dx"], s["dg"] = torch.empty_like(s["dh"]), torch.empty_like(s["dh"])
            s["dh0"] = torch.empty_like(s["h0"])
        else:
            s["x"] = normal(b, t, d).to(td)
            s["h"], s["state"] = torch.empty_like(s["x"]), torch.empty_like(s["h0"])
    return s


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "gemm": _plain_gemm, "scan": _plain_scan}[op](state)
    import memory_bound_gemv_02_gb300 as g
    if op == "norm":
        y, scale, res = g.rms_norm_fused(state["x"], state["weight"], residual=state["residual"], eps=EPS,
                                         eight_bit=state["case"]["eight"], y=state["y"], scale=state["scale"],
                                         residual_out=state["residual_out"])
        return {"y": y, "scale": scale, "residual": res}
    if op == "gemm":
        return {"c": g.gemm_fused(state["B"], state["A"], state["c"], scale_a=state["scale_a"],
                                  scale_b=state["scale_b"], bias=state["bias"], activation=state["case"]["act"],
                                  residual=state["residual"])}
    if state["case"]["backward"]:
        dx, dg, dh0 = g.gated_scan_backward(state["dh"], state["g"], state["h"], h0=state["h0"],
                                            dstate=state["dstate"], dx=state["dx"], dg=state["dg"], dh0=state["dh0"])
        return {"dx": dx, "dg": dg, "dh0": dh0}
    h, last = g.gated_scan(state["x"], state["g"], h0=state["h0"], h=state["h"], state=state["state"])
    return {"h": h, "state": last}


# ------------------------------------------------------------ plain forms --

def _plain_norm(state):
    x, td = state["x"].float(), state["x"].dtype
    s = x if state["residual"] is None else x + state["residual"].float()
    t = s * state["weight"].float()
    rstd = torch.rsqrt((s * s).mean(dim=1, keepdim=True) + EPS)
    y = t * rstd
    out = {"y": y.to(td), "scale": None, "residual": None if state["residual"] is None else s.to(td)}
    if state["case"]["eight"]:
        peak = y.abs().amax(dim=1, keepdim=True)
        scale = torch.where(peak == 0, torch.ones_like(peak), peak / E4M3_MAX)
        out["y"], out["scale"] = (y / scale).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), scale[:, 0]
    return out


def _plain_act(y, act):
    if act == "relu":
        return torch.clamp(y, min=0.0)
    if act == "silu":
        return y / (1.0 + torch.exp(-y))
    if act == "log_sigmoid":
        return torch.clamp(y, max=0.0) - torch.log1p(torch.exp(-y.abs()))
    return y


def _plain_gemm(state):
    y = torch.matmul(state["A"].float(), state["B"].float().t())
    if state["scale_a"] is not None:
        y = y * state["scale_a"][:, None] * state["scale_b"][None, :]
    if state["bias"] is not None:
        y = y + state["bias"]
    y = _plain_act(y, state["case"]["act"])
    if state["residual"] is not None:
        y = y + state["residual"].float()
    return {"c": y.to(state["c"].dtype)}


def _doubled(a, h):
    """h_t = a_t h_{t-1} + h_t along dim 1, by doubling the span that each step covers."""
    span = 1
    while span < h.shape[1]:
        h = torch.cat([h[:, :span], h[:, span:] + a[:, span:] * h[:, :-span]], dim=1)
        a = torch.cat([a[:, :span], a[:, span:] * a[:, :-span]], dim=1)
        span *= 2
    return h


def _plain_scan(state):
    g, h0, td = state["g"].float(), state["h0"], state["g"].dtype
    a = torch.exp(g)
    if not state["case"]["backward"]:
        x = state["x"].float()
        x[:, 0] += a[:, 0] * h0
        h = _doubled(a, x)
        return {"h": h.to(td), "state": h[:, -1].clone()}
    dh = state["dh"].float()
    dh[:, -1] += state["dstate"]
    # the gradient of h_t gathers dh_s from s = t on, decayed by a_{t+1} .. a_s: the same recurrence, reversed
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], dim=1)
    d = _doubled(later.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([h0[:, None], state["h"][:, :-1].float()], dim=1)
    return {"dx": d.to(td), "dg": (d * a * before).to(td), "dh0": d[:, 0] * a[:, 0]}


# ------------------------------------------------------------ definitions --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        v = s["x"].double()
        if s["residual"] is not None:
            v += s["residual"].double()
        y = v / (v.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS).sqrt() * s["weight"].double()
        res = v if s["residual"] is not None else None
        if not case["eight"]:
            return {"y": y, "scale": None, "residual": res}
        scale = y.abs().max(dim=1).values / E4M3_MAX
        return {"y": y / scale[:, None], "scale": scale, "residual": res}
    if case["op"] == "gemm":
        B, A = s["B"].double(), s["A"].double()
        if s["scale_a"] is not None:
            A *= s["scale_a"].double()[:, None]
            B *= s["scale_b"].double()[:, None]
        y = torch.einsum("mk,nk->mn", A, B)
        if s["bias"] is not None:
            y += s["bias"].double()
        if case["act"] == "relu":
            y = torch.where(y > 0, y, 0.0)
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        elif case["act"] == "log_sigmoid":
            y = -torch.logaddexp(-y, torch.zeros_like(y))
        if s["residual"] is not None:
            y += s["residual"].double()
        return {"c": y}
    b, t, d = case["b"], case["t"], case["d"]
    decay = s["g"].double().exp()
    if not case["backward"]:
        h = s["h0"].double()
        out = s["x"].double()
        for i in range(t):
            h = torch.addcmul(out[:, i], decay[:, i], h)
            out[:, i] = h
        return {"h": out, "state": h}
    dx = s["dh"].double()
    dg = torch.empty_like(dx)
    carry = s["dstate"].double()
    for i in range(t - 1, -1, -1):
        total = dx[:, i] + carry
        dx[:, i] = total
        carry = total * decay[:, i]
        dg[:, i] = carry * (s["h"][:, i - 1].double() if i else s["h0"].double())
    return {"dx": dx, "dg": dg, "dh0": carry}


# ------------------------------------------------------------------- work --

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "norm":
        cells = case["rows"] * case["d"]
        per = es * (3 if case["residual"] else 1) + (1 if case["eight"] else es)
        return {"bytes": cells * per + case["d"] * es + (4 * case["rows"] if case["eight"] else 0),
                "flops": 6 * cells}
    if case["op"] == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        oe = 2
        b = (m + n) * k * es + m * n * oe * (2 if case["residual"] else 1)
        b += (4 * n if case["bias"] else 0) + (4 * (m + n) if case["dtype"] == "e4m3" else 0)
        return {"bytes": b, "flops": 2 * m * n * k}
    cells, chans = case["b"] * case["t"] * case["d"], case["b"] * case["d"]
    if case["backward"]:  # dh, g and h in, dx and dg out; h0, dstate and dh0
        return {"bytes": 5 * es * cells + 12 * chans, "flops": 5 * cells}
    return {"bytes": 3 * es * cells + 8 * chans, "flops": 3 * cells}  # x and g in, h out; h0 and the last state
