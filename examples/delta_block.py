"""A gated delta-rule block made of the package's operators.

    s       = x + stream                                (stream keeps s)
    y       = layer_norm(s)
    q, k, v = y W_q^T, y W_k^T, y W_v^T                 per head, q and k of unit length
    g, beta = log(sigmoid(y W_g^T + b_g)), sigmoid(y W_b^T)
    S_t     = exp(g_t) S_{t-1} + k_t (beta_t (v_t - exp(g_t) S_{t-1}^T k_t))^T
    o_t     = S_t^T q_t / sqrt(d_k)
    out     = layer_norm(o, per head) W_o^T

``DeltaBlock`` runs it on a prompt of many tokens and on single tokens, with the
state updated in place; ``LayerNorm`` and ``GatedDelta`` are the norm and the rule
with their gradients as torch.autograd.Functions.

    python examples/delta_block.py [--d 1024 --heads 8 --keys 4 --batch 2 --tokens 512]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_gemv_02_gb300 as g300  # noqa: E402


class DeltaBlock:
    """``heads`` heads of size ``dv`` whose keys and queries (``keys`` heads of size
    ``dk``) are shared by neighbours."""

    def __init__(self, d, heads, keys, dk, dv, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weights(rows, cols):
            return (torch.randn((rows, cols), generator=gen, device=device) / cols ** 0.5).to(torch.bfloat16)

        self.d, self.heads, self.keys, self.dk, self.dv = d, heads, keys, dk, dv
        self.norm = 1 + 0.1 * torch.randn(d, generator=gen, device=device)
        self.shift = 0.1 * torch.randn(d, generator=gen, device=device)
        # q, k and v of a token side by side; g and beta likewise
        self.w_qkv = weights(2 * keys * dk + heads * dv, d)
        self.w_g, self.w_b = weights(heads, d), weights(heads, d)
        self.b_g = torch.linspace(1.0, 5.0, heads, device=device)  # half-lives of two steps to a hundred
        self.w_o = weights(d, heads * dv)
        self.unit = torch.full((dk,), dk ** -0.5, device=device)  # a norm of unit length
        self.norm_o = torch.ones(dv, device=device)

    def new_state(self, batch):
        return torch.zeros((batch, self.heads, self.dk, self.dv), device=self.w_o.device)

    def __call__(self, x, stream, state, last=False):
        """x and stream: (batch, tokens, d) bfloat16, contiguous; stream becomes
        stream + x and state moves on by the tokens, both in place.  Returns the
        block's output, or, for the ``last`` block, the stream with it."""
        b, t, d = x.shape
        rows = stream.view(b * t, d)
        y, _, _, _ = g300.layer_norm_fused(x.view(b * t, d), self.norm, self.shift, residual=rows, residual_out=rows)
        qkv = g300.gemm_fused(self.w_qkv, y)
        wide = self.keys * self.dk
        # q and k of unit length, in place of what they were
        units = qkv[:, :2 * wide].reshape(-1, self.dk)
        units, _, _ = g300.rms_norm_fused(units, self.unit)
        units = units.view(b, t, 2, self.keys, self.dk)
        v = qkv[:, 2 * wide:].view(b, t, self.heads, self.dv)
        g = g300.gemm_fused(self.w_g, y, bias=self.b_g, activation="log_sigmoid", out_dtype=torch.float32)
        beta = g300.gemm_fused(self.w_b, y, activation="sigmoid", out_dtype=torch.float32)
        o, _ = g300.gated_delta(units[:, :, 0], units[:, :, 1], v, g.view(b, t, -1), beta.view(b, t, -1),
                                scale=self.dk ** -0.5, h0=state, state=state)
        o, _, _, _ = g300.layer_norm_fused(o.view(-1, self.dv), self.norm_o)
        return g300.gemm_fused(self.w_o, o.view(b * t, -1), residual=rows if last else None).view(b, t, d)


def run_blocks(blocks, x, states):
    """A stack of blocks over x (batch, tokens, d); states advance in place."""
    stream = torch.zeros_like(x)
    for i, block in enumerate(blocks):
        x = block(x, stream, states[i], last=i == len(blocks) - 1)
    return x


class LayerNorm(torch.autograd.Function):
    """y, s = layer_norm(x + residual), x + residual with their gradients; rows
    (rows, d), residual may be None (s is x then)."""

    @staticmethod
    def forward(ctx, x, residual, weight, bias, eps):
        y, mean, rstd, s = g300.layer_norm_fused(x, weight, bias, residual=residual, eps=eps, stats=True)
        ctx.save_for_backward(x if s is None else s, weight, bias, mean, rstd)
        ctx.with_residual = residual is not None
        if s is None:
            s = x.view_as(x)
        return y, s

    @staticmethod
    def backward(ctx, dy, ds):
        s, weight, bias, mean, rstd = ctx.saved_tensors
        dx, dw, db = g300.layer_norm_backward(dy.contiguous(), s, weight, mean, rstd, ds=ds.contiguous())
        return (dx, dx if ctx.with_residual else None, None if weight is None else dw.to(weight.dtype),
                None if bias is None else db.to(bias.dtype), None)


class GatedDelta(torch.autograd.Function):
    """o, last state = gated_delta(q, k, v, g, beta, scale, h0) with their gradients;
    h0 may be None (zero)."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale, h0):
        o, state = g300.gated_delta(q, k, v, g, beta, scale, h0=h0)
        ctx.save_for_backward(q, k, v, g, beta, h0)
        ctx.scale = scale
        return o, state

    @staticmethod
    def backward(ctx, do, dstate):
        q, k, v, g, beta, h0 = ctx.saved_tensors
        *grads, dh0 = g300.gated_delta_backward(do.contiguous(), q, k, v, g, beta, ctx.scale, h0=h0,
                                                dstate=dstate.contiguous())
        return (*grads, None, None if h0 is None else dh0)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--d", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--keys", type=int, default=4)
    ap.add_argument("--size", type=int, default=128, help="of a head")
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--new", type=int, default=64, help="tokens decoded one at a time")
    args = ap.parse_args()
    dev = torch.device("cuda", 0)
    blocks = [DeltaBlock(args.d, args.heads, args.keys, args.size, args.size, dev, seed) for seed in range(2)]
    x = torch.randn((args.batch, args.tokens + args.new, args.d), device=dev).to(torch.bfloat16)

    whole = run_blocks(blocks, x, [b.new_state(args.batch) for b in blocks])
    states = [b.new_state(args.batch) for b in blocks]
    run_blocks(blocks, x[:, :args.tokens].contiguous(), states)
    torch.cuda.synchronize()
    start = time.perf_counter()
    decoded = [run_blocks(blocks, x[:, t:t + 1].contiguous(), states)
               for t in range(args.tokens, args.tokens + args.new)]
    torch.cuda.synchronize()
    took = time.perf_counter() - start
    decoded, want = torch.cat(decoded, 1).float(), whole[:, args.tokens:].float()
    print(f"decoded against the whole prompt: {((decoded - want).norm() / want.norm()).item():.2e} of the norm apart, "
          f"{took / args.new * 1e6:.0f} us per token for {len(blocks)} blocks")

    # gradient descent through the norm and the rule: keys, values and gates fitted to a target
    shape = (args.batch, args.tokens)
    rows = torch.randn((args.batch * args.tokens, args.d), device=dev).to(torch.bfloat16)
    leaves = {"w": torch.ones(args.d, device=dev), "b": torch.zeros(args.d, device=dev),
              "w_k": torch.randn((args.d, args.keys * args.size), device=dev) / args.d ** 0.5,
              "w_v": torch.randn((args.d, args.heads * args.size), device=dev) / args.d ** 0.5,
              "g": torch.full((args.heads,), -0.1, device=dev)}
    target = torch.randn((*shape, args.heads, args.size), device=dev).cumsum(1) / args.tokens ** 0.5
    losses = []
    for _ in range(20):
        p = {n: t.requires_grad_() for n, t in leaves.items()}
        y, _ = LayerNorm.apply(rows, None, p["w"], p["b"], 1e-5)
        k = torch.nn.functional.normalize((y.float() @ p["w_k"]).view(*shape, args.keys, args.size), dim=-1)
        v = (y.float() @ p["w_v"]).view(*shape, args.heads, args.size)
        g = p["g"].expand(*shape, args.heads).contiguous()
        o, _ = GatedDelta.apply(k.to(torch.bfloat16), k.to(torch.bfloat16), v.to(torch.bfloat16), g,
                                torch.full_like(g, 0.5), args.size ** -0.5, None)
        loss = (o.float() - target).square().mean()
        losses.append(loss.item())
        grads = torch.autograd.grad(loss, list(p.values()))
        with torch.no_grad():
            leaves = {n: (t - 200 * d / (1 + d.norm() * 200)).detach() for (n, t), d in zip(p.items(), grads)}
            leaves["g"].clamp_(max=-0.01)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
