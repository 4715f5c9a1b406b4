"""A pre-norm gated feed-forward block on the block-128 FP8 operators.

    r   = x + residual                      (mxfp4_fp8_rmsnorm: the sum, its RMS
    q   = FP8(rmsnorm(r) * w)                norm and the quantization in one pass)
    h   = FP8(act(q Wg^T) * (q Wu^T))       (mxfp4_fp8_gated)
    out = h Wd^T                            (mxfp4_fp8_gemm)

FeedForward.decode() serves single tokens: three calls, nothing but the weights
read from memory once serve() has laid those out.  FeedForward.train() is the
same block under autograd:

    d(out) -> FP8 along its rows and along the tokens
    dh  = d(out) Wd,  dWd = d(out)^T h      (mxfp4_fp8_gemm)
    dy, dWg, dWu                            (mxfp4_fp8_gated_backward, which also
                                             gives h along the tokens)
    dx, dw                                  (mxfp4_fp8_rmsnorm_backward, with the
                                             residual's own gradient added)

Run:  python examples/fp8_feed_forward.py   (needs the GPU library)
"""
from __future__ import annotations

import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import microscaling_fp4_quantized_block_amd as mx  # noqa: E402


class _Block(torch.autograd.Function):
    """(out, r) of bf16 x and residual [tokens, width] and the bf16 weights, with FP8 products both ways."""

    @staticmethod
    def forward(ctx, x, residual, norm, gate, up, down, act, eps):
        q, r, y, rstd = mx.mxfp4_fp8_rmsnorm(x, norm, eps, residual=residual, train=True)
        h, g, u = mx.mxfp4_fp8_gated(q, mx.mxfp4_fp8_quantize_pair(gate, up), act=act, train=True)
        out = mx.mxfp4_fp8_gemm(h, mx.mxfp4_fp8_quantize(down, block_rows=128))
        ctx.save_for_backward(r, y, rstd, norm, gate, up, down, g, u)
        ctx.act = act
        return out, r

    @staticmethod
    def backward(ctx, dout, dr):
        r, y, rstd, norm, gate, up, down, g, u = ctx.saved_tensors
        dout = dout.contiguous()
        dh = mx.mxfp4_fp8_gemm(mx.mxfp4_fp8_quantize(dout), mx.mxfp4_fp8_quantize(down, axis=0, block_rows=128))
        dy, dgate, dup, ht = mx.mxfp4_fp8_gated_backward(
            dh, g, u, mx.mxfp4_fp8_quantize_pair(gate, up, axis=0), mx.mxfp4_fp8_quantize(y, axis=0), act=ctx.act,
            dtype=torch.bfloat16, want_ht=True)
        ddown = mx.mxfp4_fp8_gemm(mx.mxfp4_fp8_quantize(dout, axis=0), ht)
        dx, dnorm = mx.mxfp4_fp8_rmsnorm_backward(dy, r, norm, rstd, dres=dr.contiguous())
        return dx, dx, dnorm.to(torch.bfloat16), dgate, dup, ddown, None, None


class FeedForward:
    def __init__(self, width: int, hidden: int, act: str = "silu", eps: float = 1e-6, device="cuda", seed: int = 0):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=g, device=device) * cols ** -0.5
            return w.to(torch.bfloat16).requires_grad_()

        self.norm = torch.ones(width, dtype=torch.bfloat16, device=device).requires_grad_()
        self.gate, self.up, self.down = weight(hidden, width), weight(hidden, width), weight(width, hidden)
        self.act, self.eps = act, eps

    def parameters(self):
        return [self.norm, self.gate, self.up, self.down]

    def train(self, x, residual):
        """(out, r), differentiable in x, residual and the weights."""
        return _Block.apply(x, residual, self.norm, self.gate, self.up, self.down, self.act, self.eps)

    @torch.no_grad()
    def serve(self):
        """The products' weights as they are now, laid out in FP8: what a program keeps between decode() calls for as
        long as it does not change them."""
        return (mx.mxfp4_fp8_quantize_pair(self.gate, self.up), mx.mxfp4_fp8_quantize(self.down, block_rows=128))

    @torch.no_grad()
    def decode(self, x, residual, served=None):
        """(out, r); residual is overwritten with r.  served: the weights of serve(); without them the weights are laid
        out in the call."""
        pair, down = served or self.serve()
        q, r = mx.mxfp4_fp8_rmsnorm(x, self.norm, self.eps, residual=residual, sum_out=residual)
        return mx.mxfp4_fp8_gemm(mx.mxfp4_fp8_gated(q, pair, act=self.act), down), r


def main():
    torch.manual_seed(0)
    tokens, width, hidden = 512, 768, 2048
    block, target = FeedForward(width, hidden), FeedForward(width, hidden, seed=1)
    x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
    res = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
    want = target.decode(x, res.clone())[0].float()
    for step in range(31):
        out, _ = block.train(x, res)
        loss = (out.float() - want).square().mean()
        loss.backward()
        with torch.no_grad():
            for p in block.parameters():   # steps of 1 % of each weight's own size
                p -= 0.01 * p.norm() / p.grad.norm() * p.grad
                p.grad = None
        if step % 10 == 0:
            print(f"training step {step:3d}  loss {loss.item():.4f}")

    block = FeedForward(4096, 14336)
    x = torch.randn(1, 4096, device="cuda").to(torch.bfloat16)
    res = torch.zeros(1, 4096, dtype=torch.bfloat16, device="cuda")
    served = block.serve()
    block.decode(x, res, served)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.decode(x, res, served)
    for _ in range(10):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(200):
        graph.replay()
    torch.cuda.synchronize()
    print(f"one token through a 4096 x 14336 block: {(time.perf_counter() - t) / 200 * 1e6:.1f} us (graph replay)")


if __name__ == "__main__":
    main()
