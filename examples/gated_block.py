"""A gated recurrent block made of the package's operators.

    s   = x + stream                          (stream keeps s)
    y   = rms_norm(s) in 8 bits, one scale per token
    u   = y W_u^T + b_u                       8-bit weights, one scale per row
    g   = log(sigmoid(y W_g^T + b_g))         the gate, as a log decay
    h_t = exp(g_t) h_{t-1} + u_t
    out = h W_o^T

``GatedBlock`` runs it on a prompt of many tokens and on single tokens, with the
recurrent state updated in place; ``GatedScan`` is the recurrence with its
gradient as a torch.autograd.Function.

    python examples/gated_block.py [--d 1024 --width 2048 --batch 2 --tokens 512]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_bound_gemv_02_gb300 as g300  # noqa: E402


def eight_bit_rows(w):
    """(weights in 8 bits, fp32 scale per row): the largest of a row becomes 448."""
    scale = w.float().abs().amax(1).clamp_min(1e-30) / 448
    return (w.float() / scale[:, None]).to(torch.float8_e4m3fn), scale


class GatedBlock:
    def __init__(self, d, width, device, seed=0):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def weights(rows, cols):
            return torch.randn((rows, cols), generator=gen, device=device) / cols ** 0.5

        self.norm = 1 + 0.1 * torch.randn(d, generator=gen, device=device)
        self.w_u, self.s_u = eight_bit_rows(weights(width, d))
        self.w_g, self.s_g = eight_bit_rows(weights(width, d))
        self.w_o = weights(d, width).to(torch.bfloat16)
        self.b_u = torch.zeros(width, device=device)
        self.b_g = torch.full((width,), 2.0, device=device)  # decays around 0.88

    def new_state(self, batch):
        return torch.zeros((batch, self.b_u.shape[0]), device=self.b_u.device)

    def __call__(self, x, stream, state, last=False):
        """x and stream: (batch, tokens, d) bfloat16, contiguous; stream becomes
        stream + x and state moves on by the tokens, both in place.  Returns the block's
        output, or, for the ``last`` block, the stream with it."""
        b, t, d = x.shape
        rows = stream.view(b * t, d)
        y, scale, _ = g300.rms_norm_fused(x.view(b * t, d), self.norm, residual=rows, eight_bit=True,
                                          residual_out=rows)
        u = g300.gemm_fused(self.w_u, y, scale_a=scale, scale_b=self.s_u, bias=self.b_u)
        g = g300.gemm_fused(self.w_g, y, scale_a=scale, scale_b=self.s_g, bias=self.b_g, activation="log_sigmoid")
        h, _ = g300.gated_scan(u.view(b, t, -1), g.view(b, t, -1), h0=state, state=state)
        return g300.gemm_fused(self.w_o, h.view(b * t, -1), residual=rows if last else None).view(b, t, d)


def run_blocks(blocks, x, states):
    """A stack of blocks over x (batch, tokens, d); states advance in place."""
    stream = torch.zeros_like(x)
    for i, block in enumerate(blocks):
        x = block(x, stream, states[i], last=i == len(blocks) - 1)
    return x


class GatedScan(torch.autograd.Function):
    """h = gated_scan(x, g, h0) with its gradient; returns (h, last state).  h0 may be None (zero)."""

    @staticmethod
    def forward(ctx, x, g, h0):
        h, state = g300.gated_scan(x, g, h0=h0)
        ctx.save_for_backward(g, h, h0)
        return h, state

    @staticmethod
    def backward(ctx, dh, dstate):
        g, h, h0 = ctx.saved_tensors
        dx, dg, dh0 = g300.gated_scan_backward(dh.contiguous(), g, h, h0=h0, dstate=dstate.contiguous())
        return dx, dg, None if h0 is None else dh0


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--d", type=int, default=1024)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--batch", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--new", type=int, default=64, help="tokens decoded one at a time")
    args = ap.parse_args()
    dev = torch.device("cuda", 0)
    blocks = [GatedBlock(args.d, args.width, dev, seed) for seed in range(2)]
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

    # gradient descent through the recurrence: inputs and gates fitted to a target
    shape = (args.batch, args.tokens, args.width)
    u = (0.1 * torch.randn(shape, device=dev)).requires_grad_()
    g = torch.full(shape, -0.5, device=dev, requires_grad=True)
    h0 = torch.zeros((args.batch, args.width), device=dev, requires_grad=True)
    target = torch.randn(shape, device=dev).cumsum(1) / args.tokens ** 0.5
    losses = []
    for _ in range(50):
        h, _ = GatedScan.apply(u, g, h0)
        loss = (h - target).square().mean()
        losses.append(loss.item())
        du, dg, dh0 = torch.autograd.grad(loss, (u, g, h0))
        with torch.no_grad():
            for p, dp in ((u, du), (g, dg), (h0, dh0)):
                p -= 0.002 * h.numel() * dp
            g.clamp_(max=-0.1)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
