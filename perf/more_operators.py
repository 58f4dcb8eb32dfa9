"""Cases of the layer norm with its gradient and of the gated delta rule: single
tokens, prompts and its gradient.

The layer norm, per row:

    s = x + residual,   y = (s - mean(s)) * rstd * weight + bias,   rstd = 1 / sqrt(var(s) + eps)

The gated delta rule, per sequence and head, on a state S (dk, dv):

    S_t = exp(g_t) S_{t-1} + k_t d_t^T,   d_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),   o_t = scale S_t^T q_t

Heads of q and k are shared by consecutive heads of v, g, beta and o.

``run`` computes a case in plain torch operations (fp32, rounded once at the
end) or, where ``own`` is set, through the package's entry points; ``exact``
computes the same outputs from the definitions in float64.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5
CHUNK = 64


def listed():
    return [
        # one decoded token's residual stream: pure latency
        {"name": "norm_one_token", "op": "norm", "rows": 1, "d": 4096, "dtype": "bf16", "residual": True,
         "backward": False},
        # a prompt of 8192 tokens, residual added, statistics kept for the gradient
        {"name": "norm_prompt", "op": "norm", "rows": 8192, "d": 7168, "dtype": "bf16", "residual": True,
         "backward": False},
        # every head's output of a prompt by itself: many short rows
        {"name": "norm_heads", "op": "norm", "rows": 131072, "d": 128, "dtype": "f32", "residual": False,
         "backward": False},
        # the prompt's gradient, with the weight's and the bias's, added to the residual stream's
        {"name": "norm_prompt_grad", "op": "norm", "rows": 8192, "d": 7168, "dtype": "bf16", "residual": True,
         "backward": True},
        # rows of odd length (no row but the first is 16-byte aligned)
        {"name": "norm_odd_grad", "op": "norm", "rows": 1001, "d": 7169, "dtype": "f16", "residual": False,
         "backward": True},
        # one stream's next token: latency
        {"name": "delta_one_stream", "op": "delta", "b": 1, "t": 1, "hk": 16, "h": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "gates": "f32", "backward": False},
        # 64 streams decoded together, two heads of v for each of k: the states' traffic
        {"name": "delta_one_token", "op": "delta", "b": 64, "t": 1, "hk": 16, "h": 32, "dk": 128, "dv": 128,
         "dtype": "bf16", "gates": "f32", "backward": False},
        # seven drafted tokens of 16 streams checked at once
        {"name": "delta_drafted", "op": "delta", "b": 16, "t": 7, "hk": 16, "h": 32, "dk": 128, "dv": 128,
         "dtype": "bf16", "gates": "bf16", "backward": False},
        # a batch of prompts
        {"name": "delta_prompts", "op": "delta", "b": 4, "t": 8192, "hk": 16, "h": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "gates": "f32", "backward": False},
        # one long document over few heads, odd length
        {"name": "delta_long", "op": "delta", "b": 1, "t": 65537, "hk": 4, "h": 8, "dk": 128, "dv": 128,
         "dtype": "f16", "gates": "f32", "backward": False},
        # the prompts' gradient, heads of k shared
        {"name": "delta_prompts_grad", "op": "delta", "b": 4, "t": 8192, "hk": 8, "h": 16, "dk": 128, "dv": 128,
         "dtype": "bf16", "gates": "f32", "backward": True},
        # a small model's gradient: odd length, head sizes that fill no tile
        {"name": "delta_ragged_grad", "op": "delta", "b": 3, "t": 1001, "hk": 6, "h": 6, "dk": 96, "dv": 72,
         "dtype": "f16", "gates": "f16", "backward": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _align(rng, v, step=64):
    """Half of the sizes are multiples of ``step``, as models choose them; the rest are left as drawn."""
    return max(step, v // step * step) if v > step and rng.random() < 0.5 else v


def draw(rng):
    if rng.random() < 0.4:
        d = _align(rng, _log_int(rng, 64, 16384))
        return {"op": "norm", "rows": _log_int(rng, 1, min(131072, 8192 * 7168 // d)), "d": d,
                "dtype": rng.choice(["f16", "bf16", "bf16", "f32"]), "residual": rng.random() < 0.6,
                "backward": rng.random() < 0.5}
    dk, dv = _align(rng, rng.randint(16, 256), 32), _align(rng, rng.randint(16, 256), 32)
    hk = _log_int(rng, 1, 16)
    h = hk * rng.choice([1, 1, 2, 4])
    b = _log_int(rng, 1, 64)
    dtype = rng.choice(["f16", "bf16", "bf16"])
    gates = rng.choice(["f32", dtype])
    backward = rng.random() < 0.4
    per_token = h * max(dk, 64) * max(dv, 64)
    most = 4 * 8192 * 16 * 128 * 128 // (b * per_token)
    if backward or rng.random() < 0.6:
        t = _log_int(rng, 2, max(2, min(8192 if backward else 65537, most)))
    else:
        t = 1
    return {"op": "delta", "b": b, "t": t, "hk": hk, "h": h, "dk": dk, "dv": dv, "dtype": dtype, "gates": gates,
            "backward": backward}


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
        s["weight"] = normal(d, sigma=0.1, mean=1.0).to(td)
        # rows whose mean is not zero, on a residual stream several times an increment's size
        off = normal(rows, 1, sigma=0.5)
        if case["backward"]:
            v = (normal(rows, d, sigma=4.0) + off).to(td)
            s["s"], s["dy"] = v, normal(rows, d).to(td)
            f = v.float()
            s["mean"] = f.mean(dim=1)
            s["rstd"] = torch.rsqrt((f - s["mean"][:, None]).square().mean(dim=1) + EPS)
            s["ds"] = normal(rows, d).to(td) if case["residual"] else None
            s["dx"] = torch.empty_like(v)
            s["dweight"], s["dbias"] = torch.empty(d, device=dev), torch.empty(d, device=dev)
        else:
            s["x"] = (normal(rows, d) + off).to(td)
            s["bias"] = normal(d, sigma=0.1).to(td)
            s["residual"] = normal(rows, d, sigma=4.0).to(td) if case["residual"] else None
            s["y"] = torch.empty_like(s["x"])
            s["mean"], s["rstd"] = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
            s["residual_out"] = torch.empty_like(s["x"]) if case["residual"] else None
        return s
    b, t, hk, h, dk, dv = (case[n] for n in ("b", "t", "hk", "h", "dk", "dv"))
    tg = TYPES[case["gates"]]
    unit = lambda v: (v / v.square().sum(dim=-1, keepdim=True).sqrt()).to(td)  # noqa: E731
    s["q"], s["k"] = unit(normal(b, t, hk, dk)), unit(normal(b, t, hk, dk))
    s["v"] = normal(b, t, h, dv).to(td)
    # the log of a gate whose half-lives run from a few steps to some hundreds, over the heads
    z = normal(b, t, h) + torch.linspace(1.0, 6.0, h, device=dev)
    g = -torch.log1p(torch.exp(-z))
    if t > 64:  # packed documents: nothing is carried into the first token of each
        starts = torch.rand((b, t, 1), generator=gen, device=dev) < 1.0 / 2048
        g = torch.where(starts, float("-inf"), g)
    s["g"] = g.to(tg)
    s["beta"] = torch.sigmoid(normal(b, t, h)).to(tg)
    s["h0"] = normal(b, h, dk, dv, sigma=0.3)
    s["scale"] = dk ** -0.5
    if case["backward"]:
        s["do"] = normal(b, t, h, dv).to(td)
        s["dstate"] = normal(b, h, dk, dv, sigma=0.1)
        for name in ("q", "k", "v", "g", "beta", "h0"):
            s["d" + name] = torch.empty_like(s[name])
    else:
        s["o"], s["state"] = torch.empty_like(s["v"]), torch.empty_like(s["h0"])
    return s


def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "norm":
            return _plain_norm_backward(state) if case["backward"] else _plain_norm(state)
        return _plain_delta(state)
    import memory_bound_gemv_02_gb300 as g
    if case["op"] == "norm":
        if case["backward"]:
            dx, dw, db = g.layer_norm_backward(state["dy"], state["s"], state["weight"], state["mean"], state["rstd"],
                                               ds=state["ds"], dx=state["dx"], dweight=state["dweight"],
                                               dbias=state["dbias"])
            return {"dx": dx, "dweight": dw, "dbias": db}
        y, mean, rstd, res = g.layer_norm_fused(state["x"], state["weight"], state["bias"], residual=state["residual"],
                                                eps=EPS, y=state["y"], mean=state["mean"], rstd=state["rstd"],
                                                residual_out=state["residual_out"])
        return {"y": y, "mean": mean, "rstd": rstd, "residual": res}
    args = [state[n] for n in ("q", "k", "v", "g", "beta")]
    if case["backward"]:
        grads = g.gated_delta_backward(state["do"], *args, scale=state["scale"], h0=state["h0"],
                                       dstate=state["dstate"], dq=state["dq"], dk=state["dk"], dv=state["dv"],
                                       dg=state["dg"], dbeta=state["dbeta"], dh0=state["dh0"])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads))
    o, last = g.gated_delta(*args, scale=state["scale"], h0=state["h0"], o=state["o"], state=state["state"])
    return {"o": o, "state": last}


# ------------------------------------------------------------ plain forms --

def _plain_norm(state):
    x, td = state["x"].float(), state["x"].dtype
    s = x if state["residual"] is None else x + state["residual"].float()
    mean = s.mean(dim=1, keepdim=True)
    rstd = torch.rsqrt((s - mean).square().mean(dim=1, keepdim=True) + EPS)
    y = (s - mean) * rstd * state["weight"].float() + state["bias"].float()
    return {"y": y.to(td), "mean": mean[:, 0], "rstd": rstd[:, 0],
            "residual": None if state["residual"] is None else s.to(td)}


def _plain_norm_backward(state):
    dy, rstd = state["dy"].float(), state["rstd"][:, None]
    xh = (state["s"].float() - state["mean"][:, None]) * rstd
    t = dy * state["weight"].float()
    dx = (t - t.mean(dim=1, keepdim=True) - xh * (t * xh).mean(dim=1, keepdim=True)) * rstd
    if state["ds"] is not None:
        dx = dx + state["ds"].float()
    return {"dx": dx.to(state["s"].dtype), "dweight": (dy * xh).sum(dim=0), "dbias": dy.sum(dim=0)}


def _chunks(x, n):
    """(b, t, h, ...) as (b, h, n, CHUNK, ...) in fp32, zeros behind the last step."""
    b, t, h = x.shape[:3]
    x = torch.cat([x.float(), torch.zeros((b, n * CHUNK - t, *x.shape[2:]), device=x.device)], dim=1)
    return x.view(b, n, CHUNK, *x.shape[2:]).movedim(3, 1)


def _steps(x, t):
    """The reverse of ``_chunks``."""
    x = x.movedim(1, 3)
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :t]


def _plain_delta(state):
    """Chunks of 64 steps: within one, (I + A) D = beta (V - decay K S) for all steps
    at once; the state is carried from chunk to chunk."""
    case = state["case"]
    b, t, hk, h, scale = case["b"], case["t"], case["hk"], case["h"], state["scale"]
    n = (t + CHUNK - 1) // CHUNK
    shared = lambda x: x.repeat_interleave(h // hk, dim=2)  # noqa: E731
    q, k = _chunks(shared(state["q"]), n), _chunks(shared(state["k"]), n)
    v, beta = _chunks(state["v"], n), _chunks(state["beta"], n)
    g = _chunks(state["g"], n).double()
    # decays from step j to step i >= j (and from the chunk's start, to its end), 0 across a new document
    new = g < -1e3
    total = torch.where(new, 0.0, g).cumsum(dim=-1)
    docs = new.cumsum(dim=-1)
    lower = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=q.device).tril()
    reach = lower & (docs[..., :, None] == docs[..., None, :])
    decay = torch.where(reach, (total[..., :, None] - total[..., None, :]).float(), float("-inf")).exp()
    first = torch.where(docs == 0, total.float().exp(), 0.0)
    last = decay[..., -1, :]
    kk, qk = k @ k.mT, q @ k.mT
    A = beta[..., None] * (decay * kk).tril(-1)
    T = torch.zeros_like(A)  # (I + A)^-1, row by row
    for i in range(CHUNK):
        T[..., i, :] = -(A[..., i, None, :i] @ T[..., :i, :])[..., 0, :]
        T[..., i, i] += 1.0
    P = scale * decay * qk
    S = state["h0"].clone()
    starts, D = [], torch.empty_like(v)
    for c in range(n):
        starts.append(S)
        R = beta[:, :, c, :, None] * (v[:, :, c] - first[:, :, c, :, None] * (k[:, :, c] @ S))
        D[:, :, c] = T[:, :, c] @ R
        S = first[:, :, c, -1, None, None] * S + (last[:, :, c, :, None] * k[:, :, c]).mT @ D[:, :, c]
    S0 = torch.stack(starts, dim=2)
    td, tg = state["v"].dtype, state["g"].dtype
    if not case["backward"]:
        o = scale * first[..., None] * (q @ S0) + P @ D
        return {"o": _steps(o, t).to(td), "state": S}
    do = _chunks(state["do"], n)
    dS = state["dstate"].clone()
    ends, dR = [], torch.empty_like(v)
    for c in range(n - 1, -1, -1):
        ends.insert(0, dS)
        dD = P[:, :, c].mT @ do[:, :, c] + last[:, :, c, :, None] * (k[:, :, c] @ dS)
        dR[:, :, c] = T[:, :, c].mT @ dD
        dS = first[:, :, c, -1, None, None] * dS + (scale * first[:, :, c, :, None] * q[:, :, c]).mT @ do[:, :, c] \
            - ((beta * first)[:, :, c, :, None] * k[:, :, c]).mT @ dR[:, :, c]
    dS1 = torch.stack(ends, dim=2)
    dP = scale * decay * (do @ D.mT)
    M = -(decay * (dR @ D.mT)).tril(-1)
    dq0 = scale * first[..., None] * (do @ S0.mT)
    x0 = -first[..., None] * (dR @ S0.mT)
    y0 = last[..., None] * (D @ dS1.mT)
    X = x0 + M @ k
    M = beta[..., None] * M
    dq = dq0 + dP @ k
    dk = beta[..., None] * X + M.mT @ k + dP.mT @ q + y0
    dbeta = (dR * v).sum(dim=-1) + (k * X).sum(dim=-1)
    # a decay's gradient: what is carried over its step, from before it to behind it
    W = (dP * qk + M * kk).tril(-1)
    behind = W.flip(-2).cumsum(dim=-2).flip(-2).tril(-1).sum(dim=-1)  # W[i, j] for j < step <= i
    ahead = ((q * dq0).sum(dim=-1) + beta * (k * x0).sum(dim=-1)).flip(-1).cumsum(dim=-1).flip(-1)
    ky = (k * y0).sum(dim=-1)
    before = torch.cat([torch.zeros_like(ky[..., :1]), ky[..., :-1].cumsum(dim=-1)], dim=-1)
    whole = first[..., -1] * (S0 * dS1).sum(dim=(-2, -1))
    dg = torch.where(new, 0.0, behind + ahead + before + whole[..., None])
    fold = lambda x: _steps(x, t).unflatten(2, (hk, h // hk)).sum(dim=3).to(td)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dk), "dv": _steps(beta[..., None] * dR, t).to(td),
            "dg": _steps(dg, t).to(tg), "dbeta": _steps(dbeta, t).to(tg), "dh0": dS}


# ------------------------------------------------------------ definitions --

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        if case["backward"]:
            dy, w = s["dy"].double(), s["weight"].double()
            rstd = s["rstd"].double()
            xh = torch.einsum("rd,r->rd", s["s"].double() - s["mean"].double().unsqueeze(1), rstd)
            u = dy * w
            a, c = u.sum(dim=1) / case["d"], torch.einsum("rd,rd->r", u, xh) / case["d"]
            dx = rstd.unsqueeze(1) * (u - a.unsqueeze(1) - c.unsqueeze(1) * xh)
            if s["ds"] is not None:
                dx += s["ds"].double()
            return {"dx": dx, "dweight": torch.einsum("rd,rd->d", dy, xh), "dbias": dy.sum(dim=0)}
        v = s["x"].double()
        if s["residual"] is not None:
            v += s["residual"].double()
        mean = v.sum(dim=1) / case["d"]
        c = v - mean.unsqueeze(1)
        rstd = 1.0 / (c.pow(2).sum(dim=1) / case["d"] + EPS).sqrt()
        y = torch.addcmul(s["bias"].double(), c * rstd.unsqueeze(1), s["weight"].double())
        return {"y": y, "mean": mean, "rstd": rstd, "residual": None if s["residual"] is None else v}
    return _exact_delta_backward(s) if case["backward"] else _exact_delta(s)


def _per_head(s, names):
    """(t, b * h, ...) in float64, heads of q and k repeated."""
    case, out = s["case"], []
    for name in names:
        x = s[name].double()
        if name in ("q", "k"):
            x = x[:, :, torch.arange(case["h"], device=x.device) // (case["h"] // case["hk"])]
        out.append(x.transpose(0, 1).flatten(1, 2).contiguous())
    return out


def _advance(S, q, k, v, a, beta):
    """One step of (heads, dk, dv) states: the new states, the corrections and what they correct."""
    S = S * a[:, None, None]
    e = v - torch.bmm(k[:, None], S)[:, 0]
    d = beta[:, None] * e
    return torch.baddbmm(S, k[:, :, None], d[:, None]), d, e


def _exact_delta(s):
    case = s["case"]
    q, k, v, g, beta = _per_head(s, ("q", "k", "v", "g", "beta"))
    a = g.exp()
    S = s["h0"].double().flatten(0, 1)
    o = torch.empty_like(v)
    for i in range(case["t"]):
        S, _, _ = _advance(S, q[i], k[i], v[i], a[i], beta[i])
        o[i] = torch.bmm(q[i][:, None], S)[:, 0]
    o = (o * s["scale"]).unflatten(1, (case["b"], case["h"])).transpose(0, 1)
    return {"o": o, "state": S.view(s["h0"].shape)}


def _exact_delta_backward(s):
    """Step by step in reverse, the states of each run of steps recomputed from its first."""
    case, scale = s["case"], s["scale"]
    q, k, v, g, beta, do = _per_head(s, ("q", "k", "v", "g", "beta", "do"))
    a = g.exp()
    span = max(1, int(math.sqrt(case["t"])))
    S = s["h0"].double().flatten(0, 1)
    kept = {}
    for i in range(case["t"]):
        if i % span == 0:
            kept[i] = S
        S, _, _ = _advance(S, q[i], k[i], v[i], a[i], beta[i])
    dq, dk, dv, dg, dbeta = (torch.empty_like(x) for x in (q, k, v, g, beta))
    dS = s["dstate"].double().flatten(0, 1)
    for start in sorted(kept, reverse=True):
        states, ds, es = [kept[start]], [], []
        for i in range(start, min(start + span, case["t"])):
            new, d, e = _advance(states[-1], q[i], k[i], v[i], a[i], beta[i])
            states.append(new), ds.append(d), es.append(e)
        for i in range(min(start + span, case["t"]) - 1, start - 1, -1):
            old, d, e = states[i - start], ds[i - start], es[i - start]
            dq[i] = scale * torch.bmm(states[i - start + 1], do[i][:, :, None])[:, :, 0]
            dS = torch.baddbmm(dS, q[i][:, :, None] * scale, do[i][:, None])
            dd = torch.bmm(k[i][:, None], dS)[:, 0]
            dbeta[i] = (dd * e).sum(dim=1)
            dv[i] = beta[i][:, None] * dd
            # the prediction a S^T k is taken from v
            back = torch.bmm(old, dv[i][:, :, None])[:, :, 0]
            dk[i] = torch.bmm(dS, d[:, :, None])[:, :, 0] - a[i][:, None] * back
            dg[i] = a[i] * ((dS * old).sum(dim=(1, 2)) - (k[i] * back).sum(dim=1))
            dS = a[i][:, None, None] * torch.baddbmm(dS, k[i][:, :, None], dv[i][:, None], alpha=-1.0)
    b, h, hk = case["b"], case["h"], case["hk"]
    whole = lambda x: x.unflatten(1, (b, h)).transpose(0, 1)  # noqa: E731
    fold = lambda x: whole(x).unflatten(2, (hk, h // hk)).sum(dim=3)  # noqa: E731
    return {"dq": fold(dq), "dk": fold(dk), "dv": whole(dv), "dg": whole(dg), "dbeta": whole(dbeta),
            "dh0": dS.view(s["h0"].shape)}


# ------------------------------------------------------------------- work --

def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "norm":
        rows, d = case["rows"], case["d"]
        extra = (1 if case["backward"] else 2) if case["residual"] else 0  # ds in; or the residual in and out
        if case["backward"]:  # dy and s in, dx out; the weight in, its gradient and the bias's out, the statistics
            return {"bytes": rows * d * es * (3 + extra) + d * (es + 8) + 8 * rows, "flops": 12 * rows * d}
        return {"bytes": rows * d * es * (2 + extra) + 2 * d * es + 8 * rows, "flops": 8 * rows * d}
    b, t, hk, h, dk, dv = (case[n] for n in ("b", "t", "hk", "h", "dk", "dv"))
    gates, state = 2 * b * t * h * BYTES[case["gates"]], 4 * b * h * dk * dv
    qk, vo = b * t * hk * dk * es, b * t * h * dv * es
    if case["backward"]:  # all inputs, do and dstate in; a gradient of each input out
        # the states again (4 of dk x dv per step), dq, dS's two updates, the corrections', dk's two parts, the decay's
        return {"bytes": 4 * qk + 3 * vo + 2 * gates + 3 * state, "flops": 18 * b * t * h * dk * dv}
    return {"bytes": 2 * qk + 2 * vo + gates + 2 * state, "flops": 6 * b * t * h * dk * dv}
